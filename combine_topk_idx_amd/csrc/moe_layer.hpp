// Launchers and size helpers of the few-token expert layer (moe_layer.hip).
#pragma once

#include "common.hpp"

namespace ep {

constexpr int64_t kLayerMaxPairs = 2048;          // (token, j) pairs of one call

// Bytes of one packed 32-row x 64-wide weight fragment.
__host__ __device__ constexpr int fragment_bytes(int quant) {
  return quant == EP_QUANT_NONE ? 4096 : quant == EP_QUANT_MXFP8 ? 2048 : 1024;
}

struct LayerWs {                                  // byte offsets of the workspace sub-arrays
  size_t act, y, done, heads, lists, total;
};
__host__ inline LayerWs layer_ws(int64_t T, int32_t k, int32_t E, int32_t hidden, int32_t inter) {
  const size_t P = (size_t)T * k, used = P < (size_t)E ? P : (size_t)E;
  LayerWs w;
  w.act = 0;
  w.y = w.act + align_up(P * inter * 2, kWsAlign);
  w.done = w.y + align_up(P * hidden * 4, kWsAlign);
  w.heads = w.done + align_up((size_t)(hidden / 32) * 4, kWsAlign);
  w.lists = w.heads + align_up(used * 16, kWsAlign);
  w.total = w.lists + align_up(used * P * 2, kWsAlign);
  return w;
}

struct LayerArgs {
  const void *x;
  int64_t T;
  int32_t k, E, hidden, inter, quant;
  const void *idx;
  int idx64;
  const float *weights;
  const uint8_t *w1, *w1_scales, *w2, *w2_scales;
  char *ws;
  void *out;
};

hipError_t launch_moe_layer(const LayerArgs &a, hipStream_t s);

hipError_t launch_pack_ex(const void *w, const void *scales, int quant, int E, int N, int K, int gate_up, void *pw,
                          void *pscales, hipStream_t s);

}  // namespace ep
