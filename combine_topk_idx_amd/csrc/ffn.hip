// Gated feed-forward block over expert rows, forward and backward (bf16):
//   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a W2^T
//   da = dy W2,  dg = da u act'(g),  du = da act(g)
//   dx = [dg du] W1,  dW1 = [dg du]^T x,  dW2 = dy^T a
// Every product runs on the core of gemm_core.hpp: both projections, the
// activation, the product of the two and the checkpoint in one launch; the
// activation's gradient in the epilogue of dy W2.
#include "ffn.hpp"
#include "gemm_core.hpp"

namespace ep {

namespace {

using namespace gemm;

enum Mode { kUp, kDown, kGradX, kGradAct };
enum Checkpoint { kCkNone, kCkBf16, kCkFp8 };             // uniform over a launch

struct RowArgs {
  const int *offsets;
  const int64_t *recv_count;
  int E;
  const char *r;           // [rows, k] bf16
  const char *c;           // weights [E, ...] bf16
  int k, n;                // reduction length and output columns (kUp, kGradAct: I)
  char *out;               // kUp: a; kGradAct: a; else the rows [rows, n]
  int act, ck_form;        // ep_act_t, Checkpoint
  char *ck;                // checkpoint data
  float *ck_scales;
  char *d;                 // kGradAct: [rows, 2I]
};

// The product over k of a tile: acc[c][r] += C fragment c . R fragment r.
template <class S, bool CSTR, bool RSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product(Acc &acc, const Source &c, const Source &r, int steps,
                                        int64_t k_all, lds_u8 *lds, int wave, int lane) {
  typedef Loader<S::BN, CSTR, 2, S::kWaves, SPLIT> LC;
  typedef Loader<S::BM, RSTR, 2, S::kWaves, false> LR;
  constexpr int kLoads = LC::kLoads + LR::kLoads, N = S::kStages;
  constexpr int kCStride = SPLIT ? S::BN / 2 : 32;
  LC lc;
  LR lr;
  lc.init(wave, lane, c);
  lr.init(wave, lane, r);
  Reader<S::BN, CSTR, 2, S::CF> rc;
  Reader<S::BM, RSTR, 2, S::RF> rr;
  const int wn = wave % S::WN, wm = wave / S::WN;
  rc.init(lane, SPLIT ? wn * 32 : wn * S::CF * 32, [](int f) { return f * kCStride; });
  rr.init(lane, wm * S::RF * 32, [](int f) { return f * 32; });
#pragma unroll
  for (int i = 0; i < S::CF; ++i)
#pragma unroll
    for (int j = 0; j < S::RF; ++j) acc[i][j] = v16f{};
  auto fetch = [&](int t) {
    lds_u8 *at = lds + (t % N) * S::kStage;
    lc.load(at, c, t, k_all - (int64_t)t * 64);
    lr.load(at + S::BN * kKBytes, r, t, k_all - (int64_t)t * 64);
  };
  // Fragments are read one k step of 16 ahead, across the stages' borders: the
  // waves meet before the last step's matrix instructions, which then cover
  // the first reads of the next stage.
  bf16x8 fc[2][S::CF], fr[2][S::RF];
  auto read = [&](int t, int s, int to) {
    const lds_u8 *tc = lds + (t % N) * S::kStage, *tr = tc + S::BN * kKBytes;
#pragma unroll
    for (int i = 0; i < S::CF; ++i) fc[to][i] = rc.bf16(tc, i, i * kCStride, s);
#pragma unroll
    for (int j = 0; j < S::RF; ++j) fr[to][j] = rr.bf16(tr, j, j * 32, s);
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int j = 0; j < S::RF; ++j)
#pragma unroll
      for (int i = 0; i < S::CF; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[from][i], fr[from][j], acc[i][j], 0, 0, 0);
  };
  // stage t is there and no wave reads stage t - 1 any more
  auto meet = [&](int t) {
    if (t + N - 2 < steps) wait_stage<kLoads * (N - 2)>();
    else wait_stage<0>();
    if (t + N - 1 < steps) fetch(t + N - 1);
  };
  if (steps == 0) return;
  for (int t = 0; t < N - 1 && t < steps; ++t) fetch(t);
  meet(0);
  read(0, 0, 0);
  for (int t = 0; t < steps; ++t) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read(t, s + 1, (s + 1) & 1);
      } else if (t + 1 < steps) {
        meet(t + 1);
        read(t + 1, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      multiply(s & 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The same on the 256 x 256 tile; c_hi: the up rows of a split operand.
template <bool CSTR, bool RSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product256(Acc &acc, const Source &c, const Source &c_hi, const Source &r, int steps,
                                           int64_t k_all, lds_u8 *lds, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v16f{};
  if (steps == 0) return;
  Pipe256<CSTR, RSTR, 2, SPLIT> p;
  p.init(c, c_hi, r, k_all, lds, wave, lane);
  p.template begin<0>(steps, [](int) {});
  bf16x8 fc[2][4], fr[2][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    fr[0][s] = p.read_r(0, 0, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) fc[i][s] = p.read_c(0, i, s);
  }
  auto step = [&](int t, auto last) {
    constexpr bool kLast = decltype(last)::value;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 1) p.template meet1<0, kLast>(t, steps);
      if (q == 3) p.template meet3<0, kLast>(t, steps);
      const bool more = q < 3 || !kLast || t + 1 < steps;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[i][s], fr[q & 1][s], acc[i][q], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (more) {
          fr[(q + 1) & 1][s] = p.read_r(q < 3 ? t : t + 1, (q + 1) & 3, s);
          if (q == 3) {
            // this step's column fragments have been used for the last time
#pragma unroll
            for (int i = 0; i < 2; ++i) fc[i][s] = p.read_c(t + 1, i, s);
          }
        }
        if (s < 2) p.template fetch<kLast>(t, q, s, steps);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int t = 0;
  for (; t + 2 < steps; ++t) step(t, Flag<false>());
  for (; t < steps; ++t) step(t, Flag<true>());
}

// Four values of the checkpoint.
[[maybe_unused]] __device__ __forceinline__ void load4_bf16(const char *p, float (&v)[4]) {
  const u32x2 q = *(const u32x2 *)p;
  v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
}
[[maybe_unused]] __device__ __forceinline__ void load4_fp8(const char *p, float scale, float (&v)[4]) {
  const uint32_t q = *(const uint32_t *)p;
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q, true);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
}

template <class S, int MODE>
__global__ __launch_bounds__(S::kThreads) void rows_kernel(RowArgs p) {
#ifdef __HIP_DEVICE_COMPILE__     // the core uses device-only types
  constexpr bool kSplit = MODE == kUp, kCStr = MODE == kGradX || MODE == kGradAct;
  constexpr int kCols = kSplit ? S::BN / 2 : S::BN;         // output columns of a tile
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int half = lane >> 5, wn = wave % S::WN, wm = wave / S::WN;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int64_t units = (int64_t)g.first[p.E] * nc;
  for (int64_t round = 0;; ++round) {
    const int64_t unit = unit_of_round(round);
    if (unit >= units) return;                               // uniform; later rounds only have larger units
    const RowTile u = row_tile(g, p.E, p.offsets, unit, nc, S::BM);
    const int64_t row0 = u.row0;
    const int e = u.e, rows = u.rows, n0 = u.tc * kCols;
    const Source r{p.r + row0 * p.k * 2, (int64_t)p.k * 2, rows};
    Source c;
    if constexpr (kSplit) {
      const int from = (!S::kDeep && wave >= S::kWaves / 2 ? p.n : 0) + n0;
      c = Source{p.c + ((int64_t)e * 2 * p.n + from) * p.k * 2, (int64_t)p.k * 2, min(kCols, p.n - n0)};
    } else if constexpr (kCStr) {
      c = Source{p.c + ((int64_t)e * p.k * p.n + n0) * 2, (int64_t)p.n * 2, p.n - n0};
    } else {
      c = Source{p.c + ((int64_t)e * p.n + n0) * p.k * 2, (int64_t)p.k * 2, min(kCols, p.n - n0)};
    }
    v16f acc[S::CF][S::RF];
    if constexpr (S::kDeep) {
      const Source c_hi{c.base + (int64_t)p.n * p.k * 2, c.pitch, c.valid};
      product256<kCStr, false, kSplit>(acc, c, c_hi, r, p.k / 64, p.k, lds, wave, lane);
    } else {
      product<S, kCStr, false, kSplit>(acc, c, r, p.k / 64, p.k, lds, wave, lane);
    }
    __syncthreads();                                         // the stages are free
    if constexpr (MODE == kUp) {
      static_assert(MODE != kUp || S::CF == 2, "one gate and one up fragment a wave");
      const int n = n0 + wn * 32, cols = p.n - n;
      uint32_t *top = (uint32_t *)smem;                      // [2][WN][BM] bits of the largest magnitudes
      if (p.ck_form == kCkFp8) {
#pragma unroll
        for (int j = 0; j < S::RF; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t m = row_amax(acc[i][j]);
            if (half == 0) top[(i * S::WN + wn) * S::BM + (wm * S::RF + j) * 32 + lane] = m;
          }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < S::RF; ++j) {
        const int at = (wm * S::RF + j) * 32 + (lane & 31);
        const bool ok = at < rows && cols > 0;
        const int64_t row = row0 + at;
        const v16f &gt = acc[0][j], &up = acc[1][j];
        float a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = act(p.act, gt[i]) * up[i];
        store_bf16(p.out + (row * p.n + n) * 2, half, ok ? cols : 0, [&](int i) { return a[i]; });
        if (p.ck_form == kCkBf16) {
          char *q = p.ck + (row * 2 * p.n + n) * 2;
          store_bf16(q, half, ok ? cols : 0, [&](int i) { return gt[i]; });
          store_bf16(q + (int64_t)p.n * 2, half, ok ? cols : 0, [&](int i) { return up[i]; });
        }
        if (p.ck_form == kCkFp8) {
          // the whole 128-column block of the checkpoint lies in the tile
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < S::WN; ++w) m = max(m, top[(i * S::WN + w) * S::BM + at]);
            const Block128 b = block128(EP_QUANT_FP8_B128, m);
            store_codes(p.ck + row * 2 * p.n + i * p.n + n, half, ok, acc[i][j], b);
            if (ok && wn == 0 && half == 0) p.ck_scales[row * (2 * p.n / 128) + (i * p.n + n0) / 128] = b.scale;
          }
        }
      }
    } else if constexpr (MODE == kGradAct) {
#pragma unroll
      for (int i = 0; i < S::CF; ++i) {
        const int n = n0 + (wn * S::CF + i) * 32, cols = p.n - n;
#pragma unroll
        for (int j = 0; j < S::RF; ++j) {
          const int at = (wm * S::RF + j) * 32 + (lane & 31);
          const bool ok = at < rows && cols > 0;
          const int64_t row = row0 + at;
          float dg[16], du[16], a[16];
          float sg = 0.0f, su = 0.0f;
          if (p.ck_form == kCkFp8) {
            if (ok) {
              sg = p.ck_scales[row * (2 * p.n / 128) + n / 128];
              su = p.ck_scales[row * (2 * p.n / 128) + (p.n + n) / 128];
            }
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float gt[4] = {}, up[4] = {};
            const int m = n + 8 * b + 4 * half;
            if (ok) {
              if (p.ck_form == kCkFp8) {
                load4_fp8(p.ck + row * 2 * p.n + m, sg, gt);
                load4_fp8(p.ck + row * 2 * p.n + p.n + m, su, up);
              } else {
                load4_bf16(p.ck + (row * 2 * p.n + m) * 2, gt);
                load4_bf16(p.ck + (row * 2 * p.n + p.n + m) * 2, up);
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float da = acc[i][j][4 * b + q];
              float f, df;
              act_grad(p.act, gt[q], f, df);
              dg[4 * b + q] = da * up[q] * df;
              du[4 * b + q] = da * f;
              a[4 * b + q] = f * up[q];
            }
          }
          char *d = p.d + (row * 2 * p.n + n) * 2;
          store_bf16(d, half, ok ? cols : 0, [&](int q) { return dg[q]; });
          store_bf16(d + (int64_t)p.n * 2, half, ok ? cols : 0, [&](int q) { return du[q]; });
          store_bf16(p.out + (row * p.n + n) * 2, half, ok ? cols : 0, [&](int q) { return a[q]; });
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::CF; ++i) {
        const int n = n0 + (wn * S::CF + i) * 32, cols = p.n - n;
#pragma unroll
        for (int j = 0; j < S::RF; ++j) {
          const int at = (wm * S::RF + j) * 32 + (lane & 31);
          store_bf16(p.out + ((row0 + at) * p.n + n) * 2, half, at < rows ? cols : 0,
                     [&](int q) { return acc[i][j][q]; });
        }
      }
    }
    __syncthreads();                                         // before the next unit's stages
  }
#endif
}

struct WeightArgs {
  const int *offsets;
  const int64_t *recv_count;
  int E;
  const char *r, *c;       // [rows, nr] and [rows, nc] bf16
  int nr, nc;
  char *out;               // [E, nr, nc] bf16
};

// out[e] = R_e^T C_e over the rows of expert e (zeros without rows).
template <class S>
__global__ __launch_bounds__(S::kThreads) void weights_kernel(WeightArgs p) {
#ifdef __HIP_DEVICE_COMPILE__     // the core uses device-only types
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int half = lane >> 5, wn = wave % S::WN, wm = wave / S::WN;
  order_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count);
  const int tr_all = (p.nr + S::BM - 1) / S::BM, tc_all = (p.nc + S::BN - 1) / S::BN;
  const int64_t per = (int64_t)tr_all * tc_all, units = per * p.E;
  for (int64_t round = 0;; ++round) {
    const int64_t unit = unit_of_round(round);
    if (unit >= units) return;
    const int place = (int)(unit / per);
    const int e = __builtin_amdgcn_readfirstlane(g.order[place]);
    const int rows = __builtin_amdgcn_readfirstlane(g.rows[e]);
    int tr, tc;
    tile_of_unit(unit - place * per, tr_all, tc_all, tr, tc);
    tr = __builtin_amdgcn_readfirstlane(tr);
    tc = __builtin_amdgcn_readfirstlane(tc);
    const int r0 = tr * S::BM, c0 = tc * S::BN;
    const int64_t row0 = p.offsets[e];
    const Source r{p.r + (row0 * p.nr + r0) * 2, (int64_t)p.nr * 2, p.nr - r0};
    const Source c{p.c + (row0 * p.nc + c0) * 2, (int64_t)p.nc * 2, p.nc - c0};
    v16f acc[S::CF][S::RF];
    product256<true, true, false>(acc, c, c, r, (rows + 63) / 64, rows, lds, wave, lane);
#pragma unroll
    for (int i = 0; i < S::CF; ++i) {
      const int n = c0 + (wn * S::CF + i) * 32, cols = p.nc - n;
#pragma unroll
      for (int j = 0; j < S::RF; ++j) {
        const int at = r0 + (wm * S::RF + j) * 32 + (lane & 31);
        store_bf16(p.out + (((int64_t)e * p.nr + at) * p.nc + n) * 2, half, at < p.nr ? cols : 0,
                   [&](int q) { return acc[i][j][q]; });
      }
    }
    __syncthreads();
  }
#endif
}

typedef Shape<2, 4, 4, 2, 2> Large;      // 256 rows x 256 columns
typedef Shape<2, 2, 4, 2, 3> Medium;     // 128 rows
typedef Shape<2, 1, 4, 2, 3> Small;      // 64 rows
typedef Shape<2, 1, 4, 1, 4> Tiny;       // 32 rows

template <class S, int MODE>
hipError_t rows_launch(const RowArgs &p, int64_t pairs, hipStream_t s) {
  const int cols = MODE == kUp ? S::BN / 2 : S::BN;
  const int64_t tiles = (pairs + S::BM - 1) / S::BM + (p.E < pairs ? p.E : pairs);
  const int64_t units = tiles * ((p.n + cols - 1) / cols);
  hipLaunchKernelGGL((rows_kernel<S, MODE>), dim3((unsigned)persistent_grid(units)), dim3(S::kThreads), 0, s, p);
  return hipGetLastError();
}

template <int MODE>
hipError_t rows_shape(const RowArgs &p, int64_t pairs, hipStream_t s) {
  const int64_t mean = pairs / p.E;
  if (mean <= 32) return rows_launch<Tiny, MODE>(p, pairs, s);
  if (mean <= 64) return rows_launch<Small, MODE>(p, pairs, s);
  if (mean <= 192) return rows_launch<Medium, MODE>(p, pairs, s);
  return rows_launch<Large, MODE>(p, pairs, s);
}

RowArgs row_args(const FfnArgs &f, const void *r, const void *c, int k, int n, void *out) {
  RowArgs p{f.h.offsets, f.recv_count, f.h.num_experts, (const char *)r, (const char *)c, k, n, (char *)out, f.act,
            !f.ck ? kCkNone : f.ck_quant == EP_QUANT_NONE ? kCkBf16 : kCkFp8, (char *)f.ck, nullptr, nullptr};
  if (p.ck_form == kCkFp8)
    p.ck_scales = (float *)((char *)f.ck + recv_geom(f.h.max_rows, 2 * f.inter, f.ck_quant).scale_off);
  return p;
}

// rows that hold a pair, at most
int64_t pairs_of(const ep_handle_t &h) {
  const int64_t n = h.num_tokens * h.num_topk;
  return n < h.max_rows ? n : h.max_rows;
}

hipError_t weights_launch(const FfnArgs &f, const void *r, int nr, const void *c, int nc, void *out, hipStream_t s) {
  const WeightArgs p{f.h.offsets, f.recv_count, f.h.num_experts, (const char *)r, (const char *)c, nr, nc, (char *)out};
  typedef Large S;
  const int64_t units = (int64_t)((nr + S::BM - 1) / S::BM) * ((nc + S::BN - 1) / S::BN) * p.E;
  hipLaunchKernelGGL((weights_kernel<S>), dim3((unsigned)persistent_grid(units)), dim3(S::kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn(const FfnArgs &f, hipStream_t s) {
  const int64_t pairs = pairs_of(f.h);
  if (pairs == 0) return hipSuccess;
  char *a = f.ws + ffn_ws(f.h.max_rows, f.inter, 0).a;
  const hipError_t e = rows_shape<kUp>(row_args(f, f.x, f.w1, f.hidden, f.inter, a), pairs, s);
  if (e != hipSuccess) return e;
  return rows_shape<kDown>(row_args(f, a, f.w2, f.inter, f.hidden, f.out), pairs, s);
}

hipError_t launch_ffn_backward(const FfnGradArgs &g, hipStream_t s) {
  const FfnArgs &f = g.f;
  const int64_t pairs = pairs_of(f.h);
  const FfnWs w = ffn_ws(f.h.max_rows, f.inter, 1);
  char *a = f.ws + w.a, *d = f.ws + w.d;
  hipError_t e;
  if (pairs > 0) {
    RowArgs p = row_args(f, g.grad_out, f.w2, f.hidden, f.inter, a);
    p.d = d;
    if ((e = rows_shape<kGradAct>(p, pairs, s)) != hipSuccess) return e;
    if ((e = rows_shape<kGradX>(row_args(f, d, f.w1, 2 * f.inter, f.hidden, g.grad_x), pairs, s)) !=
        hipSuccess)
      return e;
  }
  if ((e = weights_launch(f, d, 2 * f.inter, f.x, f.hidden, g.grad_w1, s)) != hipSuccess) return e;
  return weights_launch(f, g.grad_out, f.hidden, a, f.inter, g.grad_w2, s);
}

}  // namespace ep
