// Launchers of the router kernels (router.hip).
#pragma once

#include "common.hpp"

namespace ep {

constexpr int32_t kMaxGroups = 64;

struct RouterArgs {
  const void *logits;
  int dtype;                                      // ep_float_t
  int64_t T;
  int32_t E, k, score;                            // score: ep_score_t
  const float *bias;
  int32_t groups, keep, top, renorm;
  float scale;
};

hipError_t launch_router(const RouterArgs &a, void *idx, int idx64, float *weights, hipStream_t s);

hipError_t launch_router_backward(const RouterArgs &a, const void *idx, int idx64, const float *grad_weights,
                                  void *grad_logits, hipStream_t s);

}  // namespace ep
