// Launchers and workspace of the gated feed-forward block (ffn.hip) and the
// block-scaled product (gmm_b128.hip).
#pragma once

#include "common.hpp"

namespace ep {

struct FfnWs {             // byte offsets of the workspace's parts
  size_t a;                // bf16 [rows, I]: the down product's operand
  size_t d;                // bf16 [rows, 2I]: gradient of gate and up rows (backward)
  size_t total;
};
__host__ inline FfnWs ffn_ws(int64_t rows, int32_t inter, int backward) {
  FfnWs w;
  w.a = 0;
  w.d = align_up((size_t)rows * inter * 2, kWsAlign);
  w.total = w.d + (backward ? align_up((size_t)rows * inter * 4, kWsAlign) : 0);
  if (w.total == 0) w.total = kWsAlign;
  return w;
}

struct FfnArgs {
  ep_handle_t h;
  const int64_t *recv_count;
  int32_t hidden, inter, act;
  const void *x, *w1, *w2;
  int32_t ck_quant;        // EP_QUANT_NONE or EP_QUANT_FP8_B128
  void *ck;                // checkpoint, or NULL
  char *ws;
  void *out;
};
struct FfnGradArgs {
  FfnArgs f;               // out unused
  const void *grad_out;
  void *grad_x, *grad_w1, *grad_w2;
};
hipError_t launch_ffn(const FfnArgs &p, hipStream_t s);
hipError_t launch_ffn_backward(const FfnGradArgs &p, hipStream_t s);

struct GmmB128Args {
  ep_handle_t h;
  const int64_t *recv_count;
  const char *a;
  int32_t a_quant, k, n;
  const void *w;
  const float *w_scales;
  int32_t transposed, act; // act: EP_ACT_NONE, or the gate's
  int32_t out_quant;
  char *out;
};
hipError_t launch_gmm_b128(const GmmB128Args &p, hipStream_t s);

}  // namespace ep
