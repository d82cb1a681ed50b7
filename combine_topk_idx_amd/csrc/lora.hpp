// Launchers and size helpers of the routed low-rank adapters (lora.hip).
#pragma once

#include "common.hpp"

namespace ep {

constexpr int32_t kMaxRank = 128;
constexpr int kLoraSplits = 4;                    // most shares of a down product's reduction axis
constexpr int64_t kLoraSplitRows = 16384;         // and the most rows it is split for

// Tokens of a piece of an adapter's gradient: its R x C partial sums then
// have at most a sixteenth of the bytes of the token rows read for them.
constexpr int outer_chunk(int R) { return R <= 8 ? 256 : 32 * R; }

// The rows a workspace is sized for: the layout's, or its tokens if they are
// more (blocks with a small capacity).
__host__ inline int64_t lora_rows(const ep_handle_t &h) {
  return h.max_rows > h.num_tokens ? h.max_rows : h.num_tokens;
}

// The up product's operand holds, for each row and step of 16 ranks, 16 high
// then 16 low bf16 parts; ranks are filled up with zeros to the steps its
// kernel is built for (1, 2, 3, 4, 6 or 8).
__host__ __device__ constexpr int operand_ranks(int R) {
  const int steps = (R + 15) / 16;
  return 16 * (steps <= 4 ? steps : steps <= 6 ? 6 : 8);
}

// Whether the work of a call fits the launches of its kernels: grids of fewer
// than 2^32 threads (a larger one is not refused by the runtime but cut to 32
// bits) and row numbers that a tile added to them leaves within 32 bits.
bool lora_fits(const ep_handle_t &h, int32_t in, int32_t out, int32_t R, int backward);

struct LoraWs {                                   // byte offsets of the workspace sub-arrays
  size_t operand, part, u, bt, at, outer, total;
};
// For `rows` rows (lora_rows): the up product's operand, 4 bytes a rank and
// row, and the down product's partial sums; backward also keeps u [T][R],
// the transposes of B ([N][R][out]) and A ([N][in][R]), and the partial
// gradients of the adapters with several pieces (an adapter of n rows has at
// most 2 n / chunk of them).
__host__ inline LoraWs lora_ws(int64_t rows, int64_t in, int64_t out, int64_t R, int64_t N, int backward) {
  LoraWs w;
  const int64_t chunk = outer_chunk((int)R), slots = rows <= chunk ? 0 : 2 * rows / chunk + 1;
  w.operand = 0;
  w.part = align_up((size_t)(rows * operand_ranks((int)R)) * 4, kWsAlign);
  w.u = w.part + align_up((size_t)(rows <= kLoraSplitRows ? kLoraSplits * rows * R : 0) * 4, kWsAlign);
  w.bt = w.u + (backward ? align_up((size_t)(rows * R) * 4, kWsAlign) : 0);
  w.at = w.bt + (backward ? align_up((size_t)(N * R * out) * 2, kWsAlign) : 0);
  w.outer = w.at + (backward ? align_up((size_t)(N * R * in) * 2, kWsAlign) : 0);
  w.total = w.outer + (backward ? align_up((size_t)(slots * R * (in > out ? in : out)) * 4, kWsAlign) : 0);
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
