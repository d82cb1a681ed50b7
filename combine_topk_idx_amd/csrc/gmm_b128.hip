// Grouped product of e4m3 rows with a scale per 128 channels and e4m3 weights
// with a scale per 128 x 128 block:
//   out[r][n] = sum over blocks b of s_x[r][b] s_w[n / 128][b] (sum_{k in b} x[r][k] w[n][k])
// A stage of the core holds exactly one block of 128 k, so the inner sum is
// two matrix instructions from a zero accumulator, and the running sum takes
// it times the product of the two scales with one fused multiply-add a value.
#include "ffn.hpp"
#include "gemm_core.hpp"

namespace ep {

namespace {

using namespace gemm;

struct GmmArgs {
  const int *offsets;
  const int64_t *recv_count;
  int E;
  const char *r;           // [rows, k] e4m3
  const char *r_scales;    // [rows, k / 128] float32 or e8m0
  const char *c;           // weights [E, n, k], or [E, k, n]
  const float *c_scales;   // by 128 x 128 block, in the weights' order
  int k, n;                // n: output columns (gated: of gate and up each)
  int bytes;               // row scales are e8m0 bytes
  int act, out_quant;      // of a gated product
  char *out;               // bf16 rows or e4m3 codes
  char *out_scales;
};

// Row scales: a group of four blocks for every row of the tile, transposed
// in LDS ([block][row]), two groups in turn.
template <int BM>
struct RowScales {
  float v[4];
  // thread t < BM holds row t
  __device__ __forceinline__ void load(const GmmArgs &p, int64_t row0, int rows, int group) {
    const int kb = p.k / 128, t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = group * 4 + i;
      v[i] = 0.0f;
      if (t < rows && b < kb) {
        const int64_t at = (row0 + t) * kb + b;
        v[i] = p.bytes ? e8m0_decode(((const uint8_t *)p.r_scales)[at]) : ((const float *)p.r_scales)[at];
      }
    }
  }
  __device__ __forceinline__ void put(float *lds, int group) const {
    if ((int)threadIdx.x < BM) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lds[((group & 1) * 4 + i) * BM + threadIdx.x] = v[i];
    }
  }
};

template <class S, bool CSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product(Acc &acc, const GmmArgs &p, const Source &c, const Source &r,
                                        int64_t row0, int e, int n0, float *sa, lds_u8 *lds, int wave, int lane) {
  typedef Loader<S::BN, CSTR, 1, S::kWaves, SPLIT> LC;
  typedef Loader<S::BM, false, 1, S::kWaves, false> LR;
  constexpr int kLoads = LC::kLoads + LR::kLoads, N = S::kStages;
  constexpr int kCStride = SPLIT ? S::BN / 2 : 32;
  LC lc;
  LR lr;
  lc.init(wave, lane, c);
  lr.init(wave, lane, r);
  Reader<S::BN, CSTR, 1, S::CF> rc;
  Reader<S::BM, false, 1, S::RF> rr;
  const int wn = wave % S::WN, wm = wave / S::WN;
  rc.init(lane, SPLIT ? wn * 32 : wn * S::CF * 32, kCStride);
  rr.init(lane, wm * S::RF * 32, 32);
#pragma unroll
  for (int i = 0; i < S::CF; ++i)
#pragma unroll
    for (int j = 0; j < S::RF; ++j) acc[i][j] = v16f{};
  const int steps = p.k / 128, kb = p.k / 128;
  // weight scales of the wave's columns (64 or fewer, gated: of one gate and
  // one up block)
  const int nb_all = SPLIT ? 2 * p.n / 128 : p.n / 128;
  const int nb = min(n0 / 128 + (SPLIT ? 0 : wn * S::CF * 32 / 128), nb_all - 1);
  const float *sw = p.c_scales + (int64_t)e * nb_all * kb + (CSTR ? nb : (int64_t)nb * kb);
  const int64_t sw_step = CSTR ? nb_all : 1, sw_up = SPLIT ? (int64_t)(p.n / 128) * kb : 0;
  auto fetch = [&](int t) {
    lds_u8 *at = lds + (t % N) * S::kStage;
    lc.load(at, c, t, p.k - (int64_t)t * 128);
    lr.load(at + S::BN * kKBytes, r, t, p.k - (int64_t)t * 128);
  };
  RowScales<S::BM> scales;
  scales.load(p, row0, r.valid, 0);
  for (int t = 0; t < N - 1 && t < steps; ++t) fetch(t);
  scales.put(sa, 0);
  float w0 = sw[0], w1 = SPLIT ? sw[sw_up] : 0.0f;
  for (int t = 0; t < steps; ++t) {
    if (t + N - 2 < steps) wait_stage<kLoads * (N - 2)>();
    else wait_stage<0>();
    if (t + N - 1 < steps) fetch(t + N - 1);
    if ((t & 3) == 0) scales.load(p, row0, r.valid, t / 4 + 1);
    const int next = min(t + 1, steps - 1);
    const float w0n = sw[next * sw_step], w1n = SPLIT ? sw[next * sw_step + sw_up] : 0.0f;
    const lds_u8 *tc = lds + (t % N) * S::kStage, *tr = tc + S::BN * kKBytes;
    const float *srow = sa + (((t >> 2) & 1) * 4 + (t & 3)) * S::BM + wm * S::RF * 32 + (lane & 31);
    v8i fc[S::CF][2];
#pragma unroll
    for (int i = 0; i < S::CF; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) fc[i][s] = rc.template fp8<kCStride>(tc, i, s);
#pragma unroll
    for (int j = 0; j < S::RF; ++j) {
      const v8i f0 = rr.template fp8<32>(tr, j, 0), f1 = rr.template fp8<32>(tr, j, 1);
      const float sr = srow[j * 32];
#pragma unroll
      for (int i = 0; i < S::CF; ++i) {
        v16f q = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fc[i][0], f0, v16f{}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                                 0x7f7f7f7f);
        q = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fc[i][1], f1, q, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
        const float by = sr * (SPLIT && i ? w1 : w0);
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[i][j][x] = __builtin_fmaf(q[x], by, acc[i][j][x]);
      }
    }
    if ((t & 3) == 3) scales.put(sa, t / 4 + 1);
    w0 = w0n;
    w1 = w1n;
  }
}

// GATED: gate and up rows in, n columns act(gate) * up out
template <class S, bool CSTR, bool GATED>
__global__ __launch_bounds__(S::kThreads) void gmm_kernel(GmmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__     // the core uses device-only types
  constexpr bool kSplit = GATED;
  constexpr int kCols = kSplit ? S::BN / 2 : S::BN;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  __shared__ float sa[8 * S::BM];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int half = lane >> 5, wn = wave % S::WN, wm = wave / S::WN;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int64_t units = (int64_t)g.first[p.E] * nc;
  for (int64_t round = 0;; ++round) {
    const int64_t unit = unit_of_round(round);
    if (unit >= units) return;
    RowTile u = row_tile(g, p.E, p.offsets, unit, nc, S::BM);
    const int n0 = u.tc * kCols;
    const Source r{p.r + u.row0 * p.k, p.k, u.rows};
    Source c;
    if constexpr (kSplit) {
      const int from = (wave >= S::kWaves / 2 ? p.n : 0) + n0;
      c = Source{p.c + ((int64_t)u.e * 2 * p.n + from) * p.k, p.k, min(kCols, p.n - n0)};
    } else if constexpr (CSTR) {
      c = Source{p.c + (int64_t)u.e * p.k * p.n + n0, p.n, p.n - n0};
    } else {
      c = Source{p.c + ((int64_t)u.e * p.n + n0) * p.k, p.k, min(kCols, p.n - n0)};
    }
    v16f acc[S::CF][S::RF];
    product<S, CSTR, kSplit>(acc, p, c, r, u.row0, u.e, n0, sa, lds, wave, lane);
    __syncthreads();
    if constexpr (!kSplit) {
#pragma unroll
      for (int i = 0; i < S::CF; ++i) {
        const int n = n0 + (wn * S::CF + i) * 32, cols = p.n - n;
#pragma unroll
        for (int j = 0; j < S::RF; ++j) {
          const int at = (wm * S::RF + j) * 32 + (lane & 31);
          store_bf16(p.out + ((u.row0 + at) * p.n + n) * 2, half, at < u.rows ? cols : 0,
                     [&](int q) { return acc[i][j][q]; });
        }
      }
    } else {
      const int n = n0 + wn * 32;                            // n is a multiple of 128: the tile lies inside
      uint32_t *top = (uint32_t *)smem;                      // [WN][BM] bits of the largest magnitudes
#pragma unroll
      for (int j = 0; j < S::RF; ++j) {
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[0][j][q] = act(p.act, acc[0][j][q]) * acc[S::CF - 1][j][q];
        if (p.out_quant != EP_QUANT_NONE) {
          const uint32_t m = row_amax(acc[0][j]);
          if (half == 0) top[wn * S::BM + (wm * S::RF + j) * 32 + lane] = m;
        }
      }
      if (p.out_quant != EP_QUANT_NONE) __syncthreads();
#pragma unroll
      for (int j = 0; j < S::RF; ++j) {
        const int at = (wm * S::RF + j) * 32 + (lane & 31);
        const int64_t row = u.row0 + at;
        const bool ok = at < u.rows;
        if (p.out_quant == EP_QUANT_NONE) {
          store_bf16(p.out + (row * p.n + n) * 2, half, ok ? 32 : 0, [&](int q) { return acc[0][j][q]; });
        } else {
          uint32_t m = 0;
#pragma unroll
          for (int w = 0; w < S::WN; ++w) m = max(m, top[w * S::BM + at]);
          const Block128 b = block128(p.out_quant, m);
          store_codes(p.out + row * p.n + n, half, ok, acc[0][j], b);
          if (ok && wn == 0 && half == 0) {
            const int64_t to = row * (p.n / 128) + n0 / 128;
            if (p.out_quant == EP_QUANT_FP8_B128_UE8M0) ((uint8_t *)p.out_scales)[to] = (uint8_t)b.byte;
            else ((float *)p.out_scales)[to] = b.scale;
          }
        }
      }
    }
    __syncthreads();
  }
#endif
}

typedef Shape<2, 4, 4, 2, 2> Large;
typedef Shape<2, 2, 4, 2, 3> Medium;
typedef Shape<2, 1, 4, 2, 3> Small;
typedef Shape<2, 1, 4, 1, 4> Tiny;

template <class S, bool CSTR, bool GATED>
hipError_t launch(const GmmArgs &p, int64_t pairs, hipStream_t s) {
  const int cols = GATED ? S::BN / 2 : S::BN;
  const int64_t tiles = (pairs + S::BM - 1) / S::BM + (p.E < pairs ? p.E : pairs);
  const int64_t units = tiles * ((p.n + cols - 1) / cols);
  hipLaunchKernelGGL((gmm_kernel<S, CSTR, GATED>), dim3((unsigned)persistent_grid(units)), dim3(S::kThreads), 0, s, p);
  return hipGetLastError();
}

template <bool CSTR, bool GATED>
hipError_t by_shape(const GmmArgs &p, int64_t pairs, hipStream_t s) {
  const int64_t mean = pairs / p.E;
  if (mean <= 32) return launch<Tiny, CSTR, GATED>(p, pairs, s);
  if (mean <= 64) return launch<Small, CSTR, GATED>(p, pairs, s);
  if (mean <= 192) return launch<Medium, CSTR, GATED>(p, pairs, s);
  return launch<Large, CSTR, GATED>(p, pairs, s);
}

}  // namespace

hipError_t launch_gmm_b128(const GmmB128Args &a, hipStream_t s) {
  const int64_t pairs = a.h.num_tokens * a.h.num_topk < a.h.max_rows ? a.h.num_tokens * a.h.num_topk : a.h.max_rows;
  if (pairs == 0) return hipSuccess;
  const int n = a.act != EP_ACT_NONE ? a.n / 2 : a.n;
  GmmArgs p{a.h.offsets, a.recv_count, a.h.num_experts, a.a, a.a + recv_geom(a.h.max_rows, a.k, a.a_quant).scale_off,
            (const char *)a.w, a.w_scales, a.k, n, a.a_quant == EP_QUANT_FP8_B128_UE8M0, a.act, a.out_quant, a.out, nullptr};
  if (a.out_quant != EP_QUANT_NONE) p.out_scales = a.out + recv_geom(a.h.max_rows, n, a.out_quant).scale_off;
  if (a.transposed) return by_shape<true, false>(p, pairs, s);
  return a.act == EP_ACT_NONE ? by_shape<false, false>(p, pairs, s) : by_shape<false, true>(p, pairs, s);
}

}  // namespace ep
