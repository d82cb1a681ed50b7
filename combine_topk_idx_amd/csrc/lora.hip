// Low-rank adapters of many requests, grouped by a routing layout of the
// adapter ids, for gfx950: forward and every gradient.
//
// What is computed, for token t with adapter e (rank R):
//   v_t   = A_e x_t                            (R x in)
//   out_t = base_t + s_e B_e v_t               (out x R)
//   u_t   = s_e B_e^T dy_t
//   dx_t  = dbase_t + A_e^T u_t
//   dA_e  = sum_t u_t x_t^T,   dB_e = s_e sum_t dy_t v_t^T
//
// R is small against in and out, so every product streams rows of tokens
// once and the bytes of x, base, out and their gradients bound the time.  The
// layout gives each adapter's tokens as one run of rows; a work item is up
// to 32 of them.
//   down   (v, u): a workgroup takes an item, its waves share the reduction
//          axis and their sums are added through LDS.  It leaves v in float32
//          for the caller and, times the scale, cut into bf16 high and low
//          parts (16 significant bits) in the operand order of
//   up     (out, dx): a workgroup takes 64 (32) rows and a block of columns, whose
//          part of B (A) it holds in registers.
//   outer  (dA, dB): a workgroup takes an adapter and a block of columns and
//          walks the adapter's rows, its waves sharing them out; the float32
//          factor is cut into three bf16 parts (24 bits), so the products are
//          those of the float32 values.
// All sums are float32 and in a fixed order.  Infinities give what the
// products above give: parts of zero and ranks that fill up a step meet none.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "formats.hpp"
#include "lora.hpp"
#include "ring.hpp"

namespace ep {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kTile = 32;                         // rows of a down product's work item
constexpr int kPer = kMaxExperts / kWave;         // adapters per lane of a search, at most

struct Item {
  int expert, row0, n;                            // expert -1: none; rows [row0, row0 + n)
  int pieces, slot;                               // the adapter's items; partial slot of its first one
};

// The `item`-th work item: every adapter's block of rows cut into pieces of
// `tile`, in adapter order; with `empty` an adapter without rows has one item
// of none.  Slots count the pieces of the adapters that have several.  Every
// wave searches by itself (no LDS, no barrier): a lane takes one adapter, or
// kPer of them where there are more than 64.
template <int PER>
__device__ __forceinline__ Item find_item_per(const int *__restrict__ offsets, int N, int tile, bool empty, int item) {
  const int lane = threadIdx.x & (kWave - 1);
  int start[PER + 1], mine = 0, split = 0;
#pragma unroll
  for (int i = 0; i <= PER; ++i) start[i] = offsets[min(lane * PER + i, N)];
  int pieces[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int rows = start[i + 1] - start[i];
    pieces[i] = (rows + tile - 1) / tile;
    if (empty && lane * PER + i < N) pieces[i] = max(pieces[i], 1);
    mine += pieces[i];
    split += pieces[i] > 1 ? pieces[i] : 0;
  }
  int upto = mine, slots = split;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(upto, d), q = __shfl_up(slots, d);
    if (lane >= d) { upto += o; slots += q; }
  }
  Item it;
  it.expert = -1;
  const uint64_t past = __ballot(upto > item);
  if (past == 0) return it;                       // uniform
  const int owner = __builtin_ffsll((long long)past) - 1;
  int at = item - (upto - mine), slot = slots - split, e = -1, row0 = 0, n = 0, pc = 0, sl = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e < 0 && at < pieces[i]) {
      e = lane * PER + i;
      row0 = start[i] + at * tile;
      n = min(tile, start[i + 1] - row0);
      pc = pieces[i];
      sl = slot + at;
    }
    at -= pieces[i];
    slot += pieces[i] > 1 ? pieces[i] : 0;
  }
  it.expert = __builtin_amdgcn_readlane(e, owner);
  it.row0 = __builtin_amdgcn_readlane(row0, owner);
  it.n = __builtin_amdgcn_readlane(n, owner);
  it.pieces = __builtin_amdgcn_readlane(pc, owner);
  it.slot = __builtin_amdgcn_readlane(sl, owner);
  return it;
}
__device__ __forceinline__ Item find_item(const int *__restrict__ offsets, int N, int tile, bool empty, int item) {
  return N <= kWave ? find_item_per<1>(offsets, N, tile, empty, item)
                    : find_item_per<kPer>(offsets, N, tile, empty, item);
}

// Operands of the 16 x 16 x 32 step: lane (c = l % 16, g = l / 16) holds K
// [8 g, 8 g + 8) of row / column c; its sums are column c, rows 4 g + i.
__device__ __forceinline__ f32x4 mfma(const bf16x8 &a, const bf16x8 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The largest bf16.  Factors are held to it before they are rounded to their
// high part, so that a value near the largest float keeps a finite one and an
// infinity leaves infinity as its rest (its own high part would leave inf - inf).
constexpr float kLargest = 3.38953139e38f;
__device__ __forceinline__ float high_of(float x) { return __builtin_amdgcn_fmed3f(x, -kLargest, kLargest); }

// Two floats as bf16 parts: a word of the high ones and one of what they leave.
__device__ __forceinline__ u32x2 split2(float x, float y) {
  const uint32_t hi = pack_bf16x2(high_of(x), high_of(y));
  return {hi, pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi))};
}

// Down product: v[r] = sum over i of w[e][r][i] rows[t][i], t the token of the
// layout's row.  MF: 16-row blocks of the rank; W: waves.
//
// A wave takes every W-th 64-wide step.  In the matrix cores' operand order 16
// consecutive lanes hold 16 rows, and a load in that order makes one cache
// access a lane (16 bytes a clock and CU, which bounded the kernel); so eight
// lanes read a row's 128-byte line, and the order is changed through LDS the
// wave has to itself (no barrier).  Chunk q of row r lies at place q ^ (r & 7)
// of its line there: reads of 8 rows fall in distinct banks.
template <int MF, int W>
__global__ __launch_bounds__(W *kWave) void down_kernel(const int *__restrict__ offsets,
                                                        const int *__restrict__ row_src, int N,
                                                        const uint16_t *__restrict__ rows, int K,
                                                        const uint16_t *__restrict__ w, int R,
                                                        const float *__restrict__ scale, int scaled,
                                                        float *__restrict__ sum, uint16_t *__restrict__ operand,
                                                        int splits, int64_t max_rows, float *__restrict__ part) {
  constexpr int kLines = 32 + 16 * MF;            // rows of a step: the tokens', then w's
  constexpr int kLoads = kLines / 8;
  constexpr int kRing = MF <= 4 ? 2 : 1;          // steps in flight
  constexpr int kStage = W * kLines * 8, kSums = 4 * W * kWave;
  __shared__ __attribute__((aligned(16))) u32x4 s_mem[kStage > kSums ? kStage : kSums];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int unit = blockIdx.x, split = unit % splits;
  const Item it = find_item(offsets, N, kTile, false, unit / splits);
  if (it.expert < 0) return;                      // uniform
  // token of row `lane` of the tile; rows past the tile and of padding: -1
  const int src = (lane & 31) < it.n ? row_src[it.row0 + (lane & 31)] : -1;
  const int first = __builtin_amdgcn_readfirstlane(src);
  if (first < 0) return;                          // uniform: a tile of padding
  // load i: line 8 i + lane / 8, chunk lane % 8
  const uint16_t *line[kLoads];
  int chunk = lane & 7;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * i + (lane >> 3);
    if (i < 4) {
      const int t = __shfl(src, r & 31);
      line[i] = rows + (size_t)(t < 0 ? first : t) * K + chunk * 8;
    } else {
      line[i] = w + ((size_t)it.expert * R + min(r - 32, R - 1)) * K + chunk * 8;
    }
  }
  u32x4 *mine = s_mem + wv * kLines * 8;
  const int all = K / 64, s_lo = (int)((int64_t)all * split / splits);   // this split's steps
  const int steps = (int)((int64_t)all * (split + 1) / splits) - s_lo;
  f32x4 acc[MF][2];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int h = 0; h < 2; ++h) acc[f][h] = f32x4{};
  u32x4 in[kRing][kLoads];
  auto load = [&](int q, int s) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) in[q][i] = *(const u32x4 *)(line[i] + (s_lo + s) * 64);
    keep_loads();
  };
  // the line's chunks [0, 4 M) are multiplied
  auto multiply = [&](int q, int M) {
    wave_lds_fence();                             // the step before has been read
#pragma unroll
    for (int i = 0; i < kLoads; ++i) mine[(8 * i + (lane >> 3)) * 8 + (chunk ^ (lane >> 3))] = in[q][i];
    wave_lds_fence();
    auto operand_at = [&](int row, int m) {
      return __builtin_bit_cast(bf16x8, mine[row * 8 + ((m * 4 + g) ^ (row & 7))]);
    };
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m >= M) break;                          // uniform
      const bf16x8 x0 = operand_at(c, m), x1 = operand_at(16 + c, m);
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const bf16x8 a = operand_at(32 + 16 * f + c, m);
        acc[f][0] = mfma(a, x0, acc[f][0]);
        acc[f][1] = mfma(a, x1, acc[f][1]);
      }
    }
  };
  if (wv < steps) {                               // uniform
#pragma unroll
    for (int q = 0; q < kRing; ++q) load(q, min(wv + q * W, steps - 1));
    // whole rings without a condition in them (a load whose value only a
    // branch uses is moved into that branch), then the rest
    int s = wv;
    for (; s + (kRing - 1) * W < steps; s += kRing * W) {
#pragma unroll
      for (int q = 0; q < kRing; ++q) {
        multiply(q, 2);
        load(q, min(s + (q + kRing) * W, steps - 1));   // past the end: never used
      }
    }
#pragma unroll
    for (int q = 0; q < kRing - 1; ++q)
      if (s + q * W < steps) multiply(q, 2);      // uniform
  }
  if (K % 64 != 0 && split == splits - 1 && wv == W - 1) {   // uniform: the last 32, twice in the line
#pragma unroll
    for (int i = 0; i < kLoads; ++i) in[0][i] = *(const u32x4 *)(line[i] + all * 64 - (chunk & 4) * 8);
    multiply(0, 1);
  }
  __syncthreads();                                // the stages become the sums
  f32x4 *s_tile = (f32x4 *)s_mem;                 // [tile of a round][wave][lane]
  // a lane holds token c of half h, ranks 16 f + 4 g + i; waves 0..3 add up
  // one of four (f, h) tiles each
  const float sc = scale ? scale[it.expert] : 1.0f;
  const int r16 = operand_ranks(R);
#pragma unroll
  for (int f0 = 0; f0 < MF; f0 += 2) {
    if (f0 > 0) __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (f0 + (q >> 1) < MF) s_tile[(q * W + wv) * kWave + lane] = acc[f0 + (q >> 1) < MF ? f0 + (q >> 1) : 0][q & 1];
    __syncthreads();
    const int f = f0 + (wv >> 1), h = wv & 1;
    if (wv < 4 && f * 16 < r16) {                 // uniform
      f32x4 v = s_tile[wv * W * kWave + lane];
#pragma unroll
      for (int q = 1; q < W; ++q) v += s_tile[(wv * W + q) * kWave + lane];
      const int r = f * 16 + 4 * g, row = h * 16 + c, t = __shfl(src, row);
      if (t >= 0 && splits > 1) {
        if (r < R) *(f32x4 *)(part + ((size_t)split * max_rows + it.row0 + row) * R + r) = v;
      } else if (t >= 0) {
        if (r >= R) v = f32x4{};                  // ranks that fill up the operand
        const f32x4 by = v * sc;
        if (r < R) *(f32x4 *)(sum + (size_t)t * R + r) = scaled ? by : v;
        uint16_t *to = operand + (size_t)(it.row0 + row) * 2 * r16 + f * 32 + 4 * g;
        const u32x2 xy = split2(by.x, by.y), zw = split2(by.z, by.w);
        *(u32x2 *)to = u32x2{xy.x, zw.x};
        *(u32x2 *)(to + 16) = u32x2{xy.y, zw.y};
      }
    }
  }
}

// x as bf16 parts: each the rounding of what the ones before it leave.  SAFE:
// beyond the largest bf16 too, an infinity in the last part (as in split2).
template <bool SAFE>
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8 &hi, bf16x8 &mid, bf16x8 &lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (__bf16)(SAFE ? high_of(v[i]) : v[i]);
    const float rest = v[i] - (float)hi[i];
    mid[i] = (__bf16)(SAFE ? high_of(rest) : rest);
    lo[i] = (__bf16)(rest - (float)mid[i]);
  }
}

// Infinities (and NaN) of bf16 operands become +-1: an infinity times a lower
// part of zero would be NaN, and what it makes of the highest part is the whole
// product (a lower part that is itself infinite has the highest one's sign).
__device__ __forceinline__ bf16x8 finite_only(const bf16x8 &v) {
  u32x4 d = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((d[j] & 0x7f80u) == 0x7f80u) d[j] = (d[j] & 0xffff8000u) | 0x3f80u;
    if ((d[j] & 0x7f800000u) == 0x7f800000u) d[j] = (d[j] & 0x8000ffffu) | 0x3f800000u;
  }
  return __builtin_bit_cast(bf16x8, d);
}

// Whether the 16 bytes hold an infinity (or NaN); `top` carries it on.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void look(const u32x4 &d, u16x2 &top) {
#pragma unroll
  for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, d[j] & 0x7fff7fffu));
}
__device__ __forceinline__ bool not_finite(const u16x2 &top) { return max(top.x, top.y) >= 0x7f80; }

// The up product's w in the lanes that hold the low parts, without infinities.
template <int NT, int RS>
__device__ __forceinline__ void drop_infinities(bf16x8 (&w)[NT][RS], bool low) {
#pragma unroll
  for (int o = 0; o < NT; ++o)
#pragma unroll
    for (int k = 0; k < RS; ++k)
      if (low) w[o][k] = finite_only(w[o][k]);
}

// Up product: out[t] = base[t] + w[e] (s v[t]) of up to 16 STEPS rows over a
// block of columns.  The 32-wide K of a matrix-core step holds 16 ranks' high parts,
// then their low parts, against the same w twice (RS steps).  A wave takes
// 16 NT columns in NT tiles, lane c the columns NT c + o of tile o, so that
// base and out move as runs of 16 lanes; it holds their w in registers and
// walks the rows 16 at a time, the base of all of them loaded beforehand.  The
// first `rest` workgroups copy the rows of the tokens without an adapter,
// each wave those of rest_tokens tokens.  Bound by base and out: 8192 tokens of
// rank 16, out 7168, 51 us (4.6 TB/s); with w read again for every 16 rows 70.
template <int NT>
struct Run;
template <>
struct Run<4> { typedef u32x2 type; };
template <>
struct Run<8> { typedef u32x4 type; };

// What the up product reads of the down product: its operand, or where the
// reduction axis was split over workgroups the shares' sums, which it adds
// up and cuts itself (the first column block leaves the sum for the caller).
struct Down {
  const uint16_t *operand;
  const float *part;
  int splits, scaled;
  int64_t max_rows;
  const float *scale;
  float *sum;
};

template <int RS, int NT, int STEPS, bool PART>
__device__ __forceinline__ void up_rows(int src, const Item &it, int from_row, int n, const Down &down, int R, bool leave,
                                        bf16x8 (&wv16)[NT][RS], const uint16_t *base, uint16_t *out, int C, int col,
                                        bool on) {
  typedef typename Run<NT>::type Cols;
  const int lane = threadIdx.x & (kWave - 1), c = lane & 15, g = lane >> 4;
  int tok[STEPS][4];
  Cols bv[STEPS][4];
  bf16x8 v[STEPS][RS];
  // unconditional loads (rows and columns out of range: ones in range, never
  // used), so that they stay in flight together
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tok[s][i] = __shfl(src, from_row + 16 * s + 4 * g + i);
      bv[s][i] = Cols{};
    }
  if (base) {                                     // uniform
    const uint16_t *from = base + min(col, C - NT);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) bv[s][i] = *(const Cols *)(from + (size_t)max(tok[s][i], 0) * C);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int k = 0; k < RS; ++k) {
      const int row = from_row + 16 * s + c;
      const size_t at = it.row0 + min(row, n - 1);
      if constexpr (!PART) {
        v[s][k] = *(const bf16x8 *)(down.operand + at * 2 * operand_ranks(R) + k * 32 + g * 8);
      } else {
        // lanes g and g + 2 hold the high and the low parts of the same ranks
        const int r = k * 16 + (g & 1) * 8, t = __shfl(src, row);
        const float sc = down.scale ? down.scale[it.expert] : 1.0f;
        const float *from = down.part + at * R + min(r, R - 8);
        f32x4 p0 = {}, p1 = {};
        for (int q = 0; q < down.splits; ++q) {
          p0 += *(const f32x4 *)(from + (size_t)q * down.max_rows * R);
          p1 += *(const f32x4 *)(from + (size_t)q * down.max_rows * R + 4);
        }
        if (leave && g < 2 && t >= 0 && r < R) {
          const float by = down.scaled ? sc : 1.0f;
          *(f32x4 *)(down.sum + (size_t)t * R + r) = p0 * by;
          *(f32x4 *)(down.sum + (size_t)t * R + r + 4) = p1 * by;
        }
        u32x4 part;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 &p = i < 2 ? p0 : p1;
          const u32x2 two = split2(r < R ? p[2 * (i & 1)] * sc : 0.0f, r < R ? p[2 * (i & 1) + 1] * sc : 0.0f);
          part[i] = g < 2 ? two.x : two.y;
        }
        v[s][k] = __builtin_bit_cast(bf16x8, part);
      }
    }
  if constexpr (RS == 1 && !PART) {
    // w as it was loaded; here, where every load is on its way
    if (R == 8) {                                 // uniform
#pragma unroll
      for (int o = 0; o < NT; ++o)
        if (g & 1) wv16[o][0] = bf16x8{};
    }
    u16x2 top = {};
#pragma unroll
    for (int o = 0; o < NT; ++o) look(__builtin_bit_cast(u32x4, wv16[o][0]), top);
    if (__builtin_expect(__any(not_finite(top)), 0)) drop_infinities(wv16, g >= 2);   // uniform
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    f32x4 acc[NT];
#pragma unroll
    for (int o = 0; o < NT; ++o) {
      acc[o] = f32x4{};
#pragma unroll
      for (int k = 0; k < RS; ++k) acc[o] = mfma(v[s][k], wv16[o][k], acc[o]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Cols o;
#pragma unroll
      for (int q = 0; q < NT / 2; ++q)
        o[q] = pack_bf16x2(bf16_lo(bv[s][i][q]) + acc[2 * q][i], bf16_hi(bv[s][i][q]) + acc[2 * q + 1][i]);
      if (on && tok[s][i] >= 0) *(Cols *)(out + (size_t)tok[s][i] * C + col) = o;
    }
  }
}

template <int RS, int NT, int STEPS, bool PART>
__global__ __launch_bounds__(kThreads) void up_kernel(const int *__restrict__ offsets, const int *__restrict__ row_src,
                                                      const int *__restrict__ slot, int N,
                                                      Down down, int64_t T, const uint16_t *__restrict__ w, int R,
                                                      const uint16_t *base, uint16_t *out, int C, int blocks, int rest,
                                                      int rest_tokens) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  if ((int)blockIdx.x < rest) {                   // uniform
    const int vecs = C / 8;
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wv) * rest_tokens;
    uint64_t without = __ballot(lane < rest_tokens && t0 + lane < T && slot[min(t0 + lane, T - 1)] < 0);
    for (; without; without &= without - 1) {     // uniform
      const int64_t t = t0 + __builtin_ffsll((long long)without) - 1;
      const u32x4 *from = (const u32x4 *)base + t * vecs;
      u32x4 *to = (u32x4 *)out + t * vecs;
#pragma unroll 4
      for (int i = lane; i < vecs; i += kWave) to[i] = base ? from[i] : u32x4{};
    }
    return;
  }
  const int unit = blockIdx.x - rest;
  const int block0 = unit % blocks * kWaves * 16 * NT, first = block0 + wv * 16 * NT;
  const Item it = find_item(offsets, N, 16 * STEPS, false, unit / blocks);
  if (it.expert < 0) return;                      // uniform
  const int src = lane < it.n ? row_src[it.row0 + lane] : -1;
  const int col = first + NT * c;
  bf16x8 wv16[NT][RS];                            // ranks past R: zeros, as in the operand
  bool bad = false;                               // w holds an infinity
  if constexpr (RS == 1 && !PART) {
    // little of w and 64 rows to use it: read in the operand order, beside the base
    if (first >= C) return;                       // uniform
#pragma unroll
    for (int o = 0; o < NT; ++o)
      wv16[o][0] = *(const bf16x8 *)(w + ((size_t)it.expert * C + min(col + o, C - 1)) * R + min((g & 1) * 8, R - 8));
  } else {
    // The workgroup's columns of w are one run of memory, read as it lies (16
    // bytes a thread: unit u) and turned to the operand order through LDS,
    // where the units of a line of 8 lie exchanged by their lane's number, so
    // that reads of 8 lanes fall in distinct banks.  4099 tokens at rank 64:
    // 17 us, against 21 in the operand order (an access a lane); 8192 at rank
    // 16: 54 against 51, the base waiting behind it.
    constexpr int kUnits = kWaves * 16 * NT * 2 * RS, kLoads = kUnits / kThreads;
    // Unit kUnits holds zeros, for ranks past R.
    __shared__ __attribute__((aligned(16))) u32x4 s_w[kUnits + 1];
    __shared__ int s_bad[kWaves];                 // the wave saw an infinity
    const int per = R / 8, lane_units = NT * per; // units of a column, of a lane's columns
    auto place = [&](int u) { return lane_units % 8 == 0 ? u ^ (u / lane_units & 7) : u; };
    const u32x4 *from = (const u32x4 *)(w + ((size_t)it.expert * C + block0) * R);
    const int here = min(kWaves * 16 * NT, C - block0) * per;
    u32x4 in[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) in[i] = from[min(i * kThreads + tid, here - 1)];
    u16x2 top = {};
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      look(in[i], top);
      if (i * kThreads + tid < here) s_w[place(i * kThreads + tid)] = in[i];
    }
    const bool saw = __any(not_finite(top));
    if (lane == 0) s_bad[wv] = saw;
    if (tid == 0) s_w[kUnits] = u32x4{};
    __syncthreads();
    if (first >= C) return;                       // uniform
    bad = __builtin_amdgcn_readfirstlane(s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3]);
#pragma unroll
    for (int o = 0; o < NT; ++o)
#pragma unroll
      for (int k = 0; k < RS; ++k) {
        const int q = 2 * k + (g & 1), u = (min(col + o, C - 1) - block0) * per + q;
        wv16[o][k] = __builtin_bit_cast(bf16x8, s_w[q < per ? place(u) : kUnits]);
      }
  }
  // rows of padding come last in a block: none from the first on
  const int n = __popcll(__ballot(src >= 0));
  if (n == 0) return;                             // uniform
  if (PART || n <= 16 || __builtin_expect(bad, 0)) {
    if (__builtin_expect(bad, 0)) drop_infinities(wv16, g >= 2);   // uniform
    for (int r = 0; r < n; r += 16)
      up_rows<RS, NT, 1, PART>(src, it, r, n, down, R, first == 0, wv16, base, out, C, col, col < C);
  } else {
    up_rows<RS, NT, STEPS, PART>(src, it, 0, n, down, R, first == 0, wv16, base, out, C, col, col < C);
  }
}

// dst[n][j][i] = src[n][i][j] of two stacks of matrices, in 64 x 64 tiles read
// and written in 16-byte chunks (rows and columns are multiples of 8), for the
// adapters with rows only.  A tile's rows are 33 words apart in LDS: a chunk's
// 8 rows read down a column by 64 lanes fall in distinct banks.  38 adapters
// of rank 64, half of them in use, 5888 + 3392 wide: 9.6 us; 32 x 32 tiles of
// 2-byte accesses over all of them took 32.
struct Transpose {
  const uint16_t *src;
  int rows, cols;
  uint16_t *dst;
};
constexpr int kTurn = 64;
__global__ __launch_bounds__(256) void transpose_kernel(const int *__restrict__ offsets, Transpose a, Transpose b,
                                                        int tiles_a) {
  __shared__ uint32_t tile[kTurn * 33];
  const Transpose &m = (int)blockIdx.x < tiles_a ? a : b;
  const int at = (int)blockIdx.x < tiles_a ? blockIdx.x : blockIdx.x - tiles_a;
  const int rows = m.rows, cols = m.cols;
  const int tr = (rows + kTurn - 1) / kTurn, tc = (cols + kTurn - 1) / kTurn;
  const int n = at / (tr * tc), in = at % (tr * tc);
  if (offsets[n] == offsets[n + 1]) return;       // uniform; nothing reads it
  const int i0 = in / tc * kTurn, j0 = in % tc * kTurn;
  const uint16_t *s = m.src + (size_t)n * rows * cols;
  uint16_t *d = m.dst + (size_t)n * rows * cols;
  const int q = threadIdx.x & 7, y = threadIdx.x >> 3;   // chunk of a line, line
  for (int i = y; i < kTurn; i += 32)
    if (i0 + i < rows && j0 + 8 * q < cols) {
      const u32x4 v = *(const u32x4 *)(s + (size_t)(i0 + i) * cols + j0 + 8 * q);
#pragma unroll
      for (int k = 0; k < 4; ++k) tile[i * 33 + 4 * q + k] = v[k];
    }
  __syncthreads();
  const uint16_t *half = (const uint16_t *)tile;
  for (int j = y; j < kTurn; j += 32)
    if (j0 + j < cols && i0 + 8 * q < rows) {
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = half[(8 * q + 2 * k) * 66 + j] | (uint32_t)half[(8 * q + 2 * k + 1) * 66 + j] << 16;
      *(u32x4 *)(d + (size_t)(j0 + j) * rows + i0 + 8 * q) = v;
    }
}

// Outer products: grad[e][r][c] (or [c][r] if T_OUT) = by * sum over the
// adapter's tokens of p[t][r] q[t][c], for a piece of `chunk` tokens and 16 NT
// columns.  MF: 16-row blocks of the rank.  A step takes 32 tokens, lane (c, g)
// the tokens 8 g .. 8 g + 7: their columns NT c + o for tile o (16 lanes read
// 16 NT consecutive columns) and their ranks 16 f + c, turned to the matrix
// cores' token-major operands in registers.  Bound by q's bytes: 8192 tokens
// of rank 16, 7168 columns, 25 us with q in the last-level cache, 36 us from
// memory (3.2 TB/s).  An adapter of one piece is done; the pieces of the others go to `part` (a slot of R x C each), which
// outer_sum_kernel adds up.  Registers for two waves a SIMD up to 64 ranks: the
// second pass for infinities would take the second wave away (30 tokens of 38
// adapters of rank 64, forward and gradients, 110 us against 90).
template <int MF, int NT, bool T_OUT>
__global__ __launch_bounds__(kThreads, MF <= 4 ? 2 : 1) void outer_kernel(const int *__restrict__ offsets,
                                                         const int *__restrict__ row_src, int N, int chunk,
                                                         const float *__restrict__ p, int R,
                                                         const uint16_t *__restrict__ q, int C,
                                                         const float *__restrict__ scale, float *__restrict__ grad,
                                                         float *__restrict__ part, int blocks) {
  typedef typename Run<NT>::type Cols;
  constexpr int kRing = MF <= 4 ? 2 : 1;          // steps of 32 tokens in flight
  constexpr int kMine = NT / kWaves;              // tiles a wave adds up
  __shared__ __attribute__((aligned(16))) f32x4 s_tile[NT * kWaves * kWave];   // [tile][wave][lane]
  extern __shared__ __attribute__((aligned(16))) int s_src[];   // the piece's tokens, padded with -1
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int c0 = (blockIdx.x % blocks) * 16 * NT;
  const Item it = find_item(offsets, N, chunk, true, blockIdx.x / blocks);
  if (it.expert < 0) return;                      // uniform
  if (it.n == 0) {                                // uniform: zeros, in whole lines
    const int here = min(16 * NT, C - c0);
    float *to = grad + (size_t)it.expert * R * C;
    if constexpr (T_OUT) {
      for (int i = tid; i < here * R / 4; i += kThreads) *(f32x4 *)(to + (size_t)c0 * R + i * 4) = f32x4{};
    } else {
      const int quads = here / 4;
      for (int i = tid; i < R * quads; i += kThreads)
        *(f32x4 *)(to + (size_t)(i / quads) * C + c0 + i % quads * 4) = f32x4{};
    }
    return;
  }
  const int padded = (it.n + 31) / 32 * 32;
  for (int i = tid; i < padded; i += kThreads) s_src[i] = i < it.n ? row_src[it.row0 + i] : -1;
  __syncthreads();
  const int col = min(c0 + NT * c, C - NT);
  f32x4 acc[MF][NT];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int o = 0; o < NT; ++o) acc[f][o] = f32x4{};
  Cols qv[kRing][8];
  float pv[kRing][MF][8];
  auto load = [&](int k, int t0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // rows of padding: token 0's, taken out below (the loads stay
      // unconditional, so that they are in flight together)
      const size_t t = (size_t)max(s_src[t0 + g * 8 + i], 0);
      qv[k][i] = *(const Cols *)(q + t * C + col);
#pragma unroll
      for (int f = 0; f < MF; ++f) pv[k][f][i] = p[t * R + min(f * 16 + c, R - 1)];
    }
    keep_loads();
  };
  auto multiply = [&](int k, int t0, auto safe) {
    constexpr bool kSafe = decltype(safe)::value;
    bf16x8 b[NT];
    const int *src = s_src + t0 + g * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool on = src[i] >= 0;
#pragma unroll
      for (int o = 0; o < NT; ++o)
        b[o][i] = __builtin_bit_cast(__bf16, (uint16_t)(on ? qv[k][i][o >> 1] >> (16 * (o & 1)) : 0u));
#pragma unroll
      for (int f = 0; f < MF; ++f) pv[k][f][i] = on ? pv[k][f][i] : 0.0f;
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      bf16x8 a0, a1, a2;
      split3<kSafe>(pv[k][f], a0, a1, a2);
#pragma unroll
      for (int o = 0; o < NT; ++o) {
        const bf16x8 rest = kSafe ? finite_only(b[o]) : b[o];
        acc[f][o] = mfma(a0, b[o], mfma(a1, rest, mfma(a2, rest, acc[f][o])));
      }
    }
  };
  constexpr std::false_type kFast{};
  constexpr int kStep = kWaves * 32;
  if (wv * 32 < padded) {                         // uniform
    const int last = padded - 32;
#pragma unroll
    for (int k = 0; k < kRing; ++k) load(k, min(wv * 32 + k * kStep, last));
    int t0 = wv * 32;
    for (; t0 + (kRing - 1) * kStep < padded; t0 += kRing * kStep) {
#pragma unroll
      for (int k = 0; k < kRing; ++k) {
        multiply(k, t0 + k * kStep, kFast);
        load(k, min(t0 + (k + kRing) * kStep, last));   // past the end: never used
      }
    }
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k)
      if (t0 + k * kStep < padded) multiply(k, t0 + k * kStep, kFast);   // uniform
    // A sum is NaN where an infinity, or a factor past the largest bf16, met
    // the factor's lower parts: only then the wave's steps once more, with
    // infinities against the highest part alone.
    bool nan = false;
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int o = 0; o < NT; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= acc[f][o][i] != acc[f][o][i];
    if (__builtin_expect(__any(nan), 0)) {        // uniform
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int o = 0; o < NT; ++o) acc[f][o] = f32x4{};
      for (t0 = wv * 32; t0 < padded; t0 += kStep) {
        load(0, t0);
        multiply(0, t0, std::true_type{});
      }
    }
  }
  const float by = scale ? scale[it.expert] : 1.0f;
  float *to = it.pieces > 1 ? part + (size_t)it.slot * R * C : grad + (size_t)it.expert * R * C;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    if (f > 0) __syncthreads();
    // ranks 16 f + 4 g + 0..3 of columns c0 + NT c + o
    const int r = f * 16 + 4 * g;
    if constexpr (T_OUT) {                        // a wave takes tiles
#pragma unroll
      for (int o = 0; o < NT; ++o) s_tile[(o * kWaves + wv) * kWave + lane] = acc[f][o];
      __syncthreads();
      const int o0 = wv * kMine, cc = c0 + NT * c + o0;
      f32x4 v[kMine];
#pragma unroll
      for (int d = 0; d < kMine; ++d) {
        v[d] = s_tile[(o0 + d) * kWaves * kWave + lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v[d] += s_tile[((o0 + d) * kWaves + k) * kWave + lane];
        v[d] *= by;
      }
      if (r < R && cc < C) {
#pragma unroll
        for (int d = 0; d < kMine; ++d) *(f32x4 *)(to + (size_t)(cc + d) * R + r) = v[d];
      }
    } else {                                      // a wave takes every fourth rank: NT columns in a row a lane
      float *s_sum = (float *)s_tile;             // [tile][wave][rank of four][lane]
#pragma unroll
      for (int o = 0; o < NT; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_sum[((o * kWaves + wv) * 4 + i) * kWave + lane] = acc[f][o][i];
      __syncthreads();
      f32x4 v[NT / 4];
#pragma unroll
      for (int o = 0; o < NT; ++o) {
        float x = s_sum[(o * kWaves * 4 + wv) * kWave + lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) x += s_sum[((o * kWaves + k) * 4 + wv) * kWave + lane];
        v[o / 4][o % 4] = x * by;
      }
      if (r < R && c0 + NT * c < C) {
#pragma unroll
        for (int d = 0; d < NT / 4; ++d) *(f32x4 *)(to + (size_t)(r + wv) * C + c0 + NT * c + 4 * d) = v[d];
      }
    }
  }
}

// grad[e] = the sum of the adapter's pieces in order, where it has several.
__global__ __launch_bounds__(256) void outer_sum_kernel(const int *__restrict__ offsets, int N, int chunk, int64_t quads,
                                                        const f32x4 *__restrict__ part, f32x4 *__restrict__ grad,
                                                        int blocks) {
  const int e = blockIdx.x / blocks;
  const int pieces = (offsets[e + 1] - offsets[e] + chunk - 1) / chunk;
  if (pieces <= 1) return;                        // uniform
  int slot = 0;
  for (int i = 0; i < e; ++i) {
    const int other = (offsets[i + 1] - offsets[i] + chunk - 1) / chunk;
    slot += other > 1 ? other : 0;
  }
  for (int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x; i < quads; i += (int64_t)blocks * 256) {
    f32x4 v = part[slot * quads + i];
    for (int k = 1; k < pieces; ++k) v += part[(slot + k) * quads + i];
    grad[e * quads + i] = v;
  }
}

// Zeros for the gradients of a call without tokens.
constexpr int kZeroBlocks = 2048;                 // eight workgroups a CU, each then walks on
__global__ __launch_bounds__(256) void zero_kernel(f32x4 *__restrict__ a, int64_t na, f32x4 *__restrict__ b, int64_t nb) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < na + nb; i += (int64_t)gridDim.x * 256)
    (i < na ? a + i : b + (i - na))[0] = f32x4{};
}

// Work items of a layout, at most: its rows in whole tiles and one partial
// tile per adapter (and no more than one per row).
int64_t items_upper(const ep_handle_t &h, int tile) {
  const int64_t rows = h.max_rows, whole = rows / tile + h.num_experts;
  return rows < whole ? rows : whole;
}

// Shares of a down product's axis.  Split where the tiles leave CUs idle, to
// about two workgroups a CU with eight steps each.  The up product then adds
// up the shares of its rows' ranks in every column block, so shares x rows x
// rank stays a third of the axis at most.  Measured (us, a whole call in 1, 2,
// 4, 8 shares): 16 tokens of 8 adapters, 4096 wide, rank 128 33, 28, 27, 31;
// rank 64 18.8, 17.1, 16.5, 17.4; 128 tokens of 16, 7168 wide, rank 32 20.9,
// 17.8, 17.0, 18.6; rank 64 28, 24, 25, 30; 128 of 8, 4096 wide, rank 128 35,
// 35, 38, 51; 600 of 8 39, 54, 67, 99.  From about half a tile a CU on whole:
// 4099 tokens at rank 64 (136 tiles) 24 + 19, 19 + 38 in two.
int down_splits(const ep_handle_t &h, int K, int R) {
  const int64_t items = items_upper(h, kTile);
  int s = 1;
  if (lora_rows(h) > kLoraSplitRows || items > 128) return s;
  const int64_t rows = (h.num_tokens + h.num_experts - 1) / h.num_experts, mine = rows < kTile ? rows : kTile;
  while (s < kLoraSplits && items * s * 2 <= 512 && K / 64 >= 2 * s * 8 && 2 * s * mine * R * 3 <= K) s *= 2;
  return s;
}

hipError_t run_down(const ep_handle_t &h, const void *rows, int K, const void *w, int R, const Down &down, void *operand,
                    void *part, hipStream_t s) {
  const dim3 grid((unsigned)(items_upper(h, kTile) * down.splits));
  const int mf = (R + 15) / 16;
#define EP_DOWN(MF, W)                                                                                         \
  hipLaunchKernelGGL((down_kernel<MF, W>), grid, dim3(W * kWave), 0, s, h.offsets, h.row_src, h.num_experts,   \
                     (const uint16_t *)rows, K, (const uint16_t *)w, R, down.scale, down.scaled, down.sum,     \
                     (uint16_t *)operand, down.splits, h.max_rows, (float *)part)
  if (mf == 1) EP_DOWN(1, 8);
  else if (mf == 2) EP_DOWN(2, 8);
  else if (mf <= 4) EP_DOWN(4, 8);
  else EP_DOWN(8, 4);                             // LDS: 20 KB a wave
#undef EP_DOWN
  return hipGetLastError();
}

// The up product's tiles (see the switch below): columns and rows of a workgroup.
int up_blocks(int C, int R) {
  const int cols = kWaves * 16 * (operand_ranks(R) <= 32 ? 8 : 4);
  return (C + cols - 1) / cols;
}
// Tokens a wave looks at for the rows without an adapter: 256 workgroups, then more tokens.
int64_t tokens_looked_at(const ep_handle_t &h) {
  const int64_t per = h.num_tokens / (256 * kWaves) + 1;
  return per < kWave ? per : kWave;
}
int64_t up_rest(const ep_handle_t &h, bool copies) {
  const int64_t tokens = kWaves * tokens_looked_at(h);
  return copies ? (h.num_tokens + tokens - 1) / tokens : 0;
}
int64_t up_units(const ep_handle_t &h, int C, int R, bool copies) {
  return items_upper(h, operand_ranks(R) <= 32 ? 64 : 32) * up_blocks(C, R) + up_rest(h, copies);
}

hipError_t run_up(const ep_handle_t &h, const Down &down, const void *w, int R, const void *base, void *out, int C,
                  hipStream_t s) {
  const int rs = operand_ranks(R) / 16;
  const int64_t rest_tokens = tokens_looked_at(h), rest = up_rest(h, out != base);
  const int blocks = up_blocks(C, R);
  const dim3 grid((unsigned)up_units(h, C, R, out != base)), block(kThreads);
#define EP_UP_PART(RS, NT, STEPS, PART)                                                                        \
  hipLaunchKernelGGL((up_kernel<RS, NT, STEPS, PART>), grid, block, 0, s, h.offsets, h.row_src, h.slot,        \
                     h.num_experts, down, h.num_tokens, (const uint16_t *)w, R, (const uint16_t *)base,        \
                     (uint16_t *)out, C, blocks, (int)rest, (int)rest_tokens)
#define EP_UP(RS, NT, STEPS)                     \
  if (down.splits > 1) EP_UP_PART(RS, NT, STEPS, true); \
  else EP_UP_PART(RS, NT, STEPS, false)
  switch (rs) {
    case 1: EP_UP(1, 8, 4); break;
    case 2: EP_UP(2, 8, 4); break;
    case 3: EP_UP(3, 4, 2); break;
    case 4: EP_UP(4, 4, 2); break;
    case 6: EP_UP(6, 4, 2); break;
    default: EP_UP(8, 4, 2); break;
  }
#undef EP_UP
#undef EP_UP_PART
  return hipGetLastError();
}

// Column blocks of the outer products, and their workgroups at most.
int outer_blocks(int C, int R) {
  const int cols = 16 * (R <= 32 ? 8 : 4);
  return (C + cols - 1) / cols;
}
int64_t outer_units(const ep_handle_t &h, int C, int R) {
  return (h.max_rows / outer_chunk(R) + h.num_experts) * outer_blocks(C, R);
}

template <bool T_OUT>
hipError_t run_outer(const ep_handle_t &h, const float *p, int R, const void *q, int C, const float *scale, float *grad,
                     float *part, hipStream_t s) {
  const int chunk = outer_chunk(R), mf = (R + 15) / 16, blocks = outer_blocks(C, R);
  const dim3 grid((unsigned)outer_units(h, C, R)), block(kThreads);
  const size_t lds = (size_t)chunk * 4;
#define EP_OUTER(MF, NT)                                                                                      \
  hipLaunchKernelGGL((outer_kernel<MF, NT, T_OUT>), grid, block, lds, s, h.offsets, h.row_src, h.num_experts, chunk, p, \
                     R, (const uint16_t *)q, C, scale, grad, part, blocks)
  if (mf == 1) EP_OUTER(1, 8);
  else if (mf == 2) EP_OUTER(2, 8);
  else if (mf <= 4) EP_OUTER(4, 4);
  else EP_OUTER(8, 4);
#undef EP_OUTER
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || h.max_rows <= chunk) return e;
  const int64_t quads = (int64_t)R * C / 4;
  const int sum_blocks = (int)((quads + 255) / 256);
  hipLaunchKernelGGL(outer_sum_kernel, dim3((unsigned)((int64_t)h.num_experts * sum_blocks)), dim3(256), 0, s, h.offsets,
                     h.num_experts, chunk, quads, (const f32x4 *)part, (f32x4 *)grad, sum_blocks);
  return hipGetLastError();
}

}  // namespace

bool lora_fits(const ep_handle_t &h, int32_t in, int32_t out, int32_t R, int backward) {
  const int64_t chunk = outer_chunk(R), most = (int64_t)UINT32_MAX / kThreads;
  const int64_t most_down = (int64_t)UINT32_MAX / (8 * kWave);   // its largest workgroup; shares: up to 512 workgroups only
  if (h.max_rows > INT32_MAX - (chunk > 64 ? chunk : 64) || items_upper(h, kTile) > most_down) return false;
  if (up_units(h, out, R, true) > most) return false;
  return !backward || (up_units(h, in, R, true) <= most && outer_units(h, in, R) <= most && outer_units(h, out, R) <= most);
}

hipError_t launch_lora(const LoraArgs &p, hipStream_t s) {
  if (p.h.num_tokens == 0) return hipSuccess;
  const LoraWs ws = lora_ws(lora_rows(p.h), p.in, p.out_features, p.rank, p.h.num_experts, 0);
  char *operand = p.ws + ws.operand, *part = p.ws + ws.part;
  const Down down{(const uint16_t *)operand, (const float *)part, down_splits(p.h, p.in, p.rank), 0, p.h.max_rows, p.scale, p.down};
  hipError_t e = run_down(p.h, p.x, p.in, p.a, p.rank, down, operand, part, s);
  if (e == hipSuccess) e = run_up(p.h, down, p.b, p.rank, p.base, p.out, p.out_features, s);
  return e;
}

hipError_t launch_lora_backward(const LoraGradArgs &p, hipStream_t s) {
  const int N = p.h.num_experts, R = p.rank;
  const LoraWs ws = lora_ws(lora_rows(p.h), p.in, p.out_features, R, N, 1);
  char *operand = p.ws + ws.operand, *part = p.ws + ws.part;
  float *u = (float *)(p.ws + ws.u), *outer = (float *)(p.ws + ws.outer);
  uint16_t *bt = (uint16_t *)(p.ws + ws.bt), *at = (uint16_t *)(p.ws + ws.at);
  if (p.h.num_tokens == 0) {
    // the layout is not asked: blocks of a fixed capacity hold rows of padding
    // also without tokens, and there is no token whose row could stand for them
    const int64_t quads_a = (int64_t)N * R * p.in / 4, quads_b = (int64_t)N * R * p.out_features / 4;
    const int64_t blocks = (quads_a + quads_b + 255) / 256;
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(blocks < kZeroBlocks ? blocks : kZeroBlocks)), dim3(256), 0, s,
                       (f32x4 *)p.grad_a, quads_a, (f32x4 *)p.grad_b, quads_b);
    return hipGetLastError();
  }
  hipError_t e = hipSuccess;
  const Transpose tb{(const uint16_t *)p.b, p.out_features, R, bt}, ta{(const uint16_t *)p.a, R, p.in, at};
  auto turns = [](int n) { return (int64_t)((n + kTurn - 1) / kTurn); };
  const int64_t tiles_b = N * turns(R) * turns(p.out_features), tiles_a = N * turns(R) * turns(p.in);
  hipLaunchKernelGGL(transpose_kernel, dim3((unsigned)(tiles_a + tiles_b)), dim3(256), 0, s, p.h.offsets, tb, ta,
                     (int)tiles_b);
  e = hipGetLastError();
  const Down down{(const uint16_t *)operand, (const float *)part, down_splits(p.h, p.out_features, R), 1, p.h.max_rows, p.scale,
                  u};
  if (e == hipSuccess) e = run_down(p.h, p.grad_out, p.out_features, bt, R, down, operand, part, s);
  // grad_out once more while the last-level cache may still hold it
  if (e == hipSuccess) e = run_outer<true>(p.h, p.down, R, p.grad_out, p.out_features, p.scale, p.grad_b, outer, s);
  if (e == hipSuccess) e = run_up(p.h, down, at, R, p.grad_base, p.grad_x, p.in, s);
  if (e == hipSuccess) e = run_outer<false>(p.h, u, R, p.x, p.in, nullptr, p.grad_a, outer, s);
  return e;
}

}  // namespace ep
