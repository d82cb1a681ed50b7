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
//   down   (v, u): a workgroup takes an item and a share of the reduction
//          axis, split again over its waves; the shares' partial sums go to the
//          workspace in float32 and are added in a fixed order by the reader.
//   up     (out, dx): a workgroup takes an item and a block of columns.  The
//          float32 v is cut into bf16 high and low parts (16 significant bits)
//          for the matrix cores.
//   outer  (dA, dB): a workgroup takes an adapter and a block of columns and
//          walks the adapter's rows, its waves sharing them out; the float32
//          factor is cut into three bf16 parts (24 bits), so the products are
//          those of the float32 values.
// All sums are float32 and in a fixed order.
#include "common.hpp"
#include "formats.hpp"
#include "lora.hpp"

namespace ep {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kTile = 32;                         // rows of a work item

struct Item {
  int expert, row0, n;                            // expert -1: none; n rows, 1 .. kTile
};

// The `item`-th work item: every adapter's block cut into tiles of kTile
// rows, in adapter order.  Rows past an adapter's tokens (padded blocks) have
// row_src -1; a tile that starts on one is empty (n = 0).
__device__ __forceinline__ Item find_item(const int *__restrict__ offsets, int N, int item) {
  __shared__ int s_wave[kWaves];
  __shared__ Item s_found;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
  const int rows = tid < N ? offsets[tid + 1] - offsets[tid] : 0;   // kMaxExperts == kThreads
  const int mine = (rows + kTile - 1) / kTile;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == kWave - 1) s_wave[wv] = upto;
  if (tid == 0) s_found.expert = -1;
  __syncthreads();
  for (int w = 0; w < wv; ++w) upto += s_wave[w];
  const int at = item - (upto - mine);
  if (at >= 0 && at < mine) {
    s_found.expert = tid;
    s_found.row0 = offsets[tid] + at * kTile;
    s_found.n = min(kTile, rows - at * kTile);
  }
  __syncthreads();
  Item it;
  it.expert = __builtin_amdgcn_readfirstlane(s_found.expert);
  it.row0 = __builtin_amdgcn_readfirstlane(s_found.row0);
  it.n = __builtin_amdgcn_readfirstlane(s_found.n);
  return it;
}
static_assert(kMaxExperts == kThreads, "one adapter per thread");

__device__ __forceinline__ v16f mfma(const bf16x8 &a, const bf16x8 &b, const v16f &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Down product: part[split][t][r] = sum over this split's share of
// w[e][r][i] rows[t][i].  MF: 32-row blocks of the rank.
template <int MF>
__global__ __launch_bounds__(kThreads) void down_kernel(const int *__restrict__ offsets,
                                                        const int *__restrict__ row_src, int N,
                                                        const uint16_t *__restrict__ rows, int K,
                                                        const uint16_t *__restrict__ w, int R, int splits, int64_t T,
                                                        float *__restrict__ part) {
  __shared__ __attribute__((aligned(16))) float s_tile[kWaves * 16 * kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave, c = lane & 31, g = lane >> 5;
  const int split = blockIdx.x % splits;
  const Item it = find_item(offsets, N, blockIdx.x / splits);
  if (it.expert < 0) return;                      // uniform
  const int first = row_src[it.row0];
  if (first < 0) return;                          // uniform: a tile of padding
  const int own = c < it.n ? row_src[it.row0 + c] : -1;
  const uint16_t *x = rows + (size_t)(own < 0 ? first : own) * K + g * 16;
  const uint16_t *a[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) a[f] = w + ((size_t)it.expert * R + min(f * 32 + c, R - 1)) * K + g * 16;
  const int steps = K / 32, parts = splits * kWaves, me = split * kWaves + wv;
  const int s0 = (int)((int64_t)steps * me / parts), s1 = (int)((int64_t)steps * (me + 1) / parts);
  v16f acc[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) acc[f] = v16f{};
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const bf16x8 b0 = *(const bf16x8 *)(x + s * 32), b1 = *(const bf16x8 *)(x + s * 32 + 8);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      acc[f] = mfma(*(const bf16x8 *)(a[f] + s * 32), b0, acc[f]);
      acc[f] = mfma(*(const bf16x8 *)(a[f] + s * 32 + 8), b1, acc[f]);
    }
  }
  // lane (c, g) holds token c, ranks 8 b + 4 g + i of each 32-row block
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    if (f > 0) __syncthreads();
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *(f32x4 *)(s_tile + ((wv * 4 + b) * kWave + lane) * 4) =
          f32x4{acc[f][4 * b], acc[f][4 * b + 1], acc[f][4 * b + 2], acc[f][4 * b + 3]};
    __syncthreads();
    if (tid < 4 * kWave) {
      const int b = tid / kWave;
      f32x4 v = *(const f32x4 *)(s_tile + (b * kWave + lane) * 4);
#pragma unroll
      for (int q = 1; q < kWaves; ++q) v += *(const f32x4 *)(s_tile + ((q * 4 + b) * kWave + lane) * 4);
      const int r = f * 32 + 8 * b + 4 * g;
      if (own >= 0 && r < R) *(f32x4 *)(part + ((size_t)split * T + own) * R + r) = v;
    }
  }
}

// x as bf16 parts x0 + x1 + x2 (each the rounding of what is left)
__device__ __forceinline__ void split2(const float (&v)[8], bf16x8 &hi, bf16x8 &lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (__bf16)v[i];
    lo[i] = (__bf16)(v[i] - (float)hi[i]);
  }
}
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8 &hi, bf16x8 &mid, bf16x8 &lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (__bf16)v[i];
    const float rest = v[i] - (float)hi[i];
    mid[i] = (__bf16)rest;
    lo[i] = (__bf16)(rest - (float)mid[i]);
  }
}

// Up product: out[t] = base[t] + w[e] (s v[t]) over a block of kUpCols
// columns; v[t] is the sum of the splits' partials, and the first column block
// leaves it (times s if `scaled`) in `sum`.  RS: 16-rank steps.
constexpr int kUpCols = 512;                      // columns of a workgroup: two 32-column tiles per wave
template <int RS>
__global__ __launch_bounds__(kThreads) void up_kernel(const int *__restrict__ offsets, const int *__restrict__ row_src,
                                                      int N, const float *__restrict__ part, int splits, int64_t T,
                                                      const uint16_t *__restrict__ w, int R,
                                                      const float *__restrict__ scale, const uint16_t *base,
                                                      uint16_t *out, int C, float *__restrict__ sum, int scaled,
                                                      int blocks) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave, c = lane & 31, g = lane >> 5;
  const int blk = blockIdx.x % blocks;
  const Item it = find_item(offsets, N, blockIdx.x / blocks);
  if (it.expert < 0) return;                      // uniform
  const int own = c < it.n ? row_src[it.row0 + c] : -1;
  const float sc = scale ? scale[it.expert] : 1.0f;
  bf16x8 hi[RS], lo[RS];
#pragma unroll
  for (int k = 0; k < RS; ++k) {
    const int r = k * 16 + g * 8;
    float v[8] = {};
    if (own >= 0 && r < R) {
      for (int q = 0; q < splits; ++q) {
        const f32x4 *from = (const f32x4 *)(part + ((size_t)q * T + own) * R + r);
        const f32x4 p0 = from[0], p1 = from[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] += p0[i]; v[4 + i] += p1[i]; }
      }
      if (blk == 0 && wv == 0) {
        const float by = scaled ? sc : 1.0f;
        f32x4 *to = (f32x4 *)(sum + (size_t)own * R + r);
        to[0] = f32x4{v[0] * by, v[1] * by, v[2] * by, v[3] * by};
        to[1] = f32x4{v[4] * by, v[5] * by, v[6] * by, v[7] * by};
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= sc;
    split2(v, hi[k], lo[k]);
  }
  // a tile's A row m = 8 b + 4 g' + i is column 16 g' + 4 b + i, so that a
  // lane's 16 sums are 16 consecutive columns of its token
  const int col_of = 16 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);
  for (int c0 = blk * kUpCols + wv * 32; c0 < min(C, (blk + 1) * kUpCols); c0 += kWaves * 32) {
    v16f acc = {};
    const uint16_t *row = w + ((size_t)it.expert * C + c0 + col_of) * R;
#pragma unroll
    for (int k = 0; k < RS; ++k) {
      const int r = min(k * 16 + g * 8, R - 8);   // ranks past R meet zeros in hi and lo
      const bf16x8 a = *(const bf16x8 *)(row + r);
      acc = mfma(a, lo[k], acc);
      acc = mfma(a, hi[k], acc);
    }
    if (own < 0) continue;
    const size_t at = (size_t)own * C + c0 + 16 * g;
    u32x4 b0 = {}, b1 = {};
    if (base) {
      b0 = *(const u32x4 *)(base + at);
      b1 = *(const u32x4 *)(base + at + 8);
    }
    u32x4 o0, o1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o0[i] = pack_bf16x2(bf16_lo(b0[i]) + acc[2 * i], bf16_hi(b0[i]) + acc[2 * i + 1]);
      o1[i] = pack_bf16x2(bf16_lo(b1[i]) + acc[8 + 2 * i], bf16_hi(b1[i]) + acc[8 + 2 * i + 1]);
    }
    *(u32x4 *)(out + at) = o0;
    *(u32x4 *)(out + at + 8) = o1;
  }
}

// out[t] = base[t] (or zeros) for the tokens without an adapter
__global__ __launch_bounds__(256) void rest_kernel(const int *__restrict__ slot, int64_t T, const u32x4 *base,
                                                   u32x4 *out, int vecs) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    if (slot[t] >= 0) continue;                   // uniform
    for (int i = threadIdx.x; i < vecs; i += blockDim.x) out[t * vecs + i] = base ? base[t * vecs + i] : u32x4{};
  }
}

// dst[n][j][i] = src[n][i][j], in 32 x 32 tiles
__global__ __launch_bounds__(256) void transpose_kernel(const uint16_t *__restrict__ src, int rows, int cols,
                                                        uint16_t *__restrict__ dst) {
  __shared__ uint16_t tile[32][33];
  const int tr = (rows + 31) / 32, tc = (cols + 31) / 32;
  const int n = blockIdx.x / (tr * tc), in = blockIdx.x % (tr * tc);
  const int i0 = in / tc * 32, j0 = in % tc * 32;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const uint16_t *s = src + (size_t)n * rows * cols;
  uint16_t *d = dst + (size_t)n * rows * cols;
  for (int i = y; i < 32; i += 8)
    if (i0 + i < rows && j0 + x < cols) tile[i][x] = s[(size_t)(i0 + i) * cols + j0 + x];
  __syncthreads();
  for (int j = y; j < 32; j += 8)
    if (j0 + j < cols && i0 + x < rows) d[(size_t)(j0 + j) * rows + i0 + x] = tile[x][j];
}

// Outer products: grad[e][r][c] (or [c][r] if T_OUT) = by * sum over the
// adapter's tokens of p[t][r] q[t][c], for a block of 64 columns.  The
// columns are taken in pairs: lane c of the even tile holds column 2 c, of
// the odd one 2 c + 1, so that a lane's four bytes of a row feed both.
template <int MF, bool T_OUT>
__global__ __launch_bounds__(kThreads) void outer_kernel(const int *__restrict__ offsets,
                                                         const int *__restrict__ row_src,
                                                         const float *__restrict__ p, int R,
                                                         const uint16_t *__restrict__ q, int C,
                                                         const float *__restrict__ scale, float *__restrict__ grad,
                                                         int blocks) {
  __shared__ __attribute__((aligned(16))) float s_tile[kWaves * 2 * 16 * kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave, c = lane & 31, g = lane >> 5;
  const int e = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * 64;
  const int lo = offsets[e], hi = offsets[e + 1];
  const int col = min(c0 + 2 * c, C - 2);
  v16f acc[MF][2];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int o = 0; o < 2; ++o) acc[f][o] = v16f{};
  for (int row = lo + wv * 16; row < hi; row += kWaves * 16) {
    bf16x8 even, odd;
    int own[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = row + g * 8 + i;
      own[i] = at < hi ? row_src[at] : -1;
      const uint32_t v = own[i] >= 0 ? *(const uint32_t *)(q + (size_t)own[i] * C + col) : 0u;
      even[i] = __builtin_bit_cast(__bf16, (uint16_t)(v & 0xffffu));
      odd[i] = __builtin_bit_cast(__bf16, (uint16_t)(v >> 16));
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int r = min(f * 32 + c, R - 1);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = own[i] >= 0 ? p[(size_t)own[i] * R + r] : 0.0f;
      bf16x8 a0, a1, a2;
      split3(v, a0, a1, a2);
      acc[f][0] = mfma(a0, even, mfma(a1, even, mfma(a2, even, acc[f][0])));
      acc[f][1] = mfma(a0, odd, mfma(a1, odd, mfma(a2, odd, acc[f][1])));
    }
  }
  const float by = scale ? scale[e] : 1.0f;
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    if (f > 0) __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *(f32x4 *)(s_tile + (((wv * 2 + o) * 4 + b) * kWave + lane) * 4) =
            f32x4{acc[f][o][4 * b], acc[f][o][4 * b + 1], acc[f][o][4 * b + 2], acc[f][o][4 * b + 3]};
    __syncthreads();
    // thread: quad (o, b) of a lane; ranks f * 32 + 8 b + 4 g + 0..3 of column c0 + 2 c + o
    const int o = tid / (4 * kWave), b = tid / kWave % 4;
    f32x4 v = *(const f32x4 *)(s_tile + ((o * 4 + b) * kWave + lane) * 4);
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += *(const f32x4 *)(s_tile + (((k * 2 + o) * 4 + b) * kWave + lane) * 4);
    v *= by;
    const int r = f * 32 + 8 * b + 4 * g, cc = c0 + 2 * c + o;
    if (r < R && cc < C) {
      if constexpr (T_OUT) {
        *(f32x4 *)(grad + ((size_t)e * C + cc) * R + r) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) grad[((size_t)e * R + r + i) * C + cc] = v[i];
      }
    }
  }
}
static_assert(kThreads == 2 * 4 * kWave, "one quad per thread");

// Work items of a layout, at most: its rows in whole tiles and one partial
// tile per adapter (and no more than one per row).
int64_t items_upper(const ep_handle_t &h) {
  const int64_t rows = h.max_rows, whole = rows / kTile + h.num_experts;
  return rows < whole ? rows : whole;
}

// Shares of a down product's axis: enough workgroups for two per CU, each
// wave with at least four 32-wide steps.
int down_splits(int64_t items, int K) {
  int s = 1;
  while (s < kLoraSplits && items * s < 512 && K / 32 >= 2 * s * kWaves * 4) s *= 2;
  return s;
}

hipError_t run_down(const ep_handle_t &h, const void *rows, int K, const void *w, int R, int splits, float *part,
                    hipStream_t s) {
  const dim3 grid((unsigned)(items_upper(h) * splits)), block(kThreads);
  const int mf = (R + 31) / 32;
#define EP_DOWN(MF)                                                                                            \
  hipLaunchKernelGGL(down_kernel<MF>, grid, block, 0, s, h.offsets, h.row_src, h.num_experts,                  \
                     (const uint16_t *)rows, K, (const uint16_t *)w, R, splits, h.num_tokens, part)
  if (mf == 1) EP_DOWN(1);
  else if (mf == 2) EP_DOWN(2);
  else if (mf == 3) EP_DOWN(3);
  else EP_DOWN(4);
#undef EP_DOWN
  return hipGetLastError();
}

hipError_t run_up(const ep_handle_t &h, const float *part, int splits, const void *w, int R, const float *scale,
                  const void *base, void *out, int C, float *sum, int scaled, hipStream_t s) {
  const int blocks = (C + kUpCols - 1) / kUpCols;
  const dim3 grid((unsigned)(items_upper(h) * blocks)), block(kThreads);
  const int rs = (R + 15) / 16;
#define EP_UP(RS)                                                                                              \
  hipLaunchKernelGGL(up_kernel<RS>, grid, block, 0, s, h.offsets, h.row_src, h.num_experts, part, splits,      \
                     h.num_tokens, (const uint16_t *)w, R, scale, (const uint16_t *)base, (uint16_t *)out, C, sum, \
                     scaled, blocks)
  if (rs == 1) EP_UP(1);
  else if (rs == 2) EP_UP(2);
  else if (rs <= 4) EP_UP(4);
  else EP_UP(8);
#undef EP_UP
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || out == base) return e;
  const int64_t b = h.num_tokens < 1024 ? h.num_tokens : 1024;
  hipLaunchKernelGGL(rest_kernel, dim3((unsigned)b), dim3(256), 0, s, h.slot, h.num_tokens, (const u32x4 *)base,
                     (u32x4 *)out, C / 8);
  return hipGetLastError();
}

template <bool T_OUT>
hipError_t run_outer(const ep_handle_t &h, const float *p, int R, const void *q, int C, const float *scale, float *grad,
                     hipStream_t s) {
  const int blocks = (C + 63) / 64;
  const dim3 grid((unsigned)((int64_t)h.num_experts * blocks)), block(kThreads);
  const int mf = (R + 31) / 32;
#define EP_OUTER(MF)                                                                                          \
  hipLaunchKernelGGL((outer_kernel<MF, T_OUT>), grid, block, 0, s, h.offsets, h.row_src, p, R,                \
                     (const uint16_t *)q, C, scale, grad, blocks)
  if (mf == 1) EP_OUTER(1);
  else if (mf == 2) EP_OUTER(2);
  else if (mf == 3) EP_OUTER(3);
  else EP_OUTER(4);
#undef EP_OUTER
  return hipGetLastError();
}

hipError_t run_transpose(const void *src, int N, int rows, int cols, void *dst, hipStream_t s) {
  const int64_t tiles = (int64_t)N * ((rows + 31) / 32) * ((cols + 31) / 32);
  hipLaunchKernelGGL(transpose_kernel, dim3((unsigned)tiles), dim3(256), 0, s, (const uint16_t *)src, rows, cols,
                     (uint16_t *)dst);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs &p, hipStream_t s) {
  if (p.h.num_tokens == 0) return hipSuccess;
  const LoraWs ws = lora_ws(p.h.num_tokens, p.in, p.out_features, p.rank, p.h.num_experts, 0);
  float *part = (float *)(p.ws + ws.part);
  const int splits = down_splits(items_upper(p.h), p.in);
  hipError_t e = run_down(p.h, p.x, p.in, p.a, p.rank, splits, part, s);
  if (e == hipSuccess)
    e = run_up(p.h, part, splits, p.b, p.rank, p.scale, p.base, p.out, p.out_features, p.down, 0, s);
  return e;
}

hipError_t launch_lora_backward(const LoraGradArgs &p, hipStream_t s) {
  const LoraWs ws = lora_ws(p.h.num_tokens, p.in, p.out_features, p.rank, p.h.num_experts, 1);
  float *part = (float *)(p.ws + ws.part), *u = (float *)(p.ws + ws.u);
  char *bt = p.ws + ws.bt, *at = p.ws + ws.at;
  hipError_t e = hipSuccess;
  if (p.h.num_tokens > 0) {
    const int splits = down_splits(items_upper(p.h), p.out_features);
    e = run_transpose(p.b, p.h.num_experts, p.out_features, p.rank, bt, s);
    if (e == hipSuccess) e = run_transpose(p.a, p.h.num_experts, p.rank, p.in, at, s);
    if (e == hipSuccess) e = run_down(p.h, p.grad_out, p.out_features, bt, p.rank, splits, part, s);
    if (e == hipSuccess) e = run_up(p.h, part, splits, at, p.rank, p.scale, p.grad_base, p.grad_x, p.in, u, 1, s);
  }
  if (e == hipSuccess) e = run_outer<false>(p.h, u, p.rank, p.x, p.in, nullptr, p.grad_a, s);
  if (e == hipSuccess) e = run_outer<true>(p.h, p.down, p.rank, p.grad_out, p.out_features, p.scale, p.grad_b, s);
  return e;
}

}  // namespace ep
