// Launchers and size helpers of the routed low-rank adapters (lora.hip).
#pragma once

#include "common.hpp"

namespace ep {

constexpr int32_t kMaxRank = 128;
constexpr int kLoraSplits = 8;                    // most shares of a down product's reduction axis

struct LoraWs {                                   // byte offsets of the workspace sub-arrays
  size_t part, u, bt, at, total;
};
// part: partial down products [splits][T][R]; backward also keeps u [T][R]
// and the transposes of B ([N][R][out]) and A ([N][in][R]).
__host__ inline LoraWs lora_ws(int64_t T, int64_t in, int64_t out, int64_t R, int64_t N, int backward) {
  LoraWs w;
  w.part = 0;
  w.u = align_up((size_t)(kLoraSplits * T * R) * 4, kWsAlign);
  w.bt = w.u + (backward ? align_up((size_t)(T * R) * 4, kWsAlign) : 0);
  w.at = w.bt + (backward ? align_up((size_t)(N * R * out) * 2, kWsAlign) : 0);
  w.total = w.at + (backward ? align_up((size_t)(N * R * in) * 2, kWsAlign) : 0);
  return w;
}

struct LoraArgs {
  ep_handle_t h;
  const void *x;
  int32_t in, out_features, rank;
  const void *a, *b;
  const float *scale;
  const void *base;
  void *out;
  float *down;
  char *ws;
};
hipError_t launch_lora(const LoraArgs &p, hipStream_t s);

struct LoraGradArgs {
  ep_handle_t h;
  const void *grad_out, *x;
  int32_t in, out_features, rank;
  const void *a, *b;
  const float *scale;
  const float *down;
  const void *grad_base;
  void *grad_x;
  float *grad_a, *grad_b;
  char *ws;
};
hipError_t launch_lora_backward(const LoraGradArgs &p, hipStream_t s);

}  // namespace ep
