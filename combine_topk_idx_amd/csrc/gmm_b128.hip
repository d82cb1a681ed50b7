// Grouped product of e4m3 rows with a scale per 128 channels and e4m3 weights
// with a scale per 128 x 128 block:
//   out[r][n] = sum over blocks b of s_x[r][b] s_w[n / 128][b] (sum_{k in b} x[r][k] w[n][k])
// A stage of the core holds exactly one block of 128 k, so the inner sum is
// one matrix instruction from a zero accumulator, and the running sum takes
// it times the product of the two scales with one fused multiply-add a value.
// (The matrix cores' own scales are powers of two: they do not hold a float32.)
//
// What bounds it: with few rows an expert the weights' bytes (figures at
// TileFew); with many the matrix cores and the vector instructions beside them
// at the clock that the power limit leaves: a pair of matrix instructions
// takes 64 cycles, its eight fused multiply-adds and two products of scales 40,
// so a pair is scaled while the next one runs -- within a wave; counted over a
// SIMD the two still add up to 93 % of its cycles (56 + 37; transposed 79: 48 + 31).
// 32768 rows in 32 experts: gate and up 7168 -> 2 x 2048 960-977 us a pass (1.97-2.0
// PFLOP/s), transposed 4096 -> 7168 1062-1077 us (1.8; four transposing reads a
// fragment for two plain ones); another card of this kind took 3 % longer.
// 64 experts of 84 rows, 1408 -> 4096: 102 us a pass, 128-row tiles.
// The 256-row forms but the plain one with float32 scales keep 8 to 18 registers in
// memory, read back between two units, each behind the loads in flight.
// Roundings: the output alone (bf16, or e4m3 with a scale per 128).
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
  int act, out_quant;      // of a gated product
  char *out;               // bf16 rows or e4m3 codes
  char *out_scales;
};

// The row scales of a stage lie behind the stages: one dword a row (a float32,
// or a byte extended), fetched by the first waves together with the stage.
template <class S>
struct ScaleArea {
  static constexpr int kRows = S::BM < kWave ? kWave : S::BM;
  static constexpr int kWaves = kRows / kWave;               // waves that fetch 64 rows each
  static constexpr int kBytes = kRows * 4;
};

// What the compiler may read through the scalar cache: uniform, and written
// by no kernel that runs beside this one.
typedef const __attribute__((address_space(4))) float *const_floats;

// The product over k of a tile, after p.begin().
//   sw, step_w, up   the weight scales of the wave's columns by block of k, and
//                    of the up columns
template <class S, bool CSTR, bool SPLIT, bool BYTES, class Acc, class Fetch>
__device__ __forceinline__ void product(Acc &acc, const PipeN<S, CSTR, 1, SPLIT> &p, const lds_u8 *area, int wave, int lane,
                                        const_floats sw, int64_t step_w, int64_t up, Fetch fetch_scales) {
  typedef ScaleArea<S> A;
  constexpr int CF = 2 * S::CF, RF = 2 * S::RF, N = S::kStages;   // of 16 x 16
  const int wm = wave / S::WN;
#pragma unroll
  for (int i = 0; i < CF; ++i)
#pragma unroll
    for (int j = 0; j < RF; ++j) acc[i][j] = v4f{};
  float w0 = sw[0], w1 = SPLIT ? sw[up] : 0.0f;
  for (int t = 0; t < p.steps; ++t) {
    p.template meet<1>(t, wave < A::kWaves, fetch_scales);
    const int next = min(t + 1, p.steps - 1);
    const float w0n = sw[next * step_w], w1n = SPLIT ? sw[next * step_w + up] : 0.0f;
    const lds_u8 *tc = p.stage_c(t), *tr = p.stage_r(t);
    const lds_u8 *srow = area + (t % N) * A::kBytes + (wm * RF * 16 + (lane & 15)) * 4;
    auto row_scale = [&](int j) {
      const uint32_t v = *(const __attribute__((address_space(3))) uint32_t *)(srow + j * 64);
      return BYTES ? e8m0_decode(v) : __uint_as_float(v);
    };
    v8i fc[CF];
#pragma unroll
    for (int i = 0; i < CF; ++i) fc[i] = p.rc.fp8(tc, i, p.c_index(i));
    // one row fragment ahead; a fragment's products are scaled and added
    // while the matrix cores work on the next one's
    v8i fr = p.rr.fp8(tr, 0, 0);
    float sr = row_scale(0), sp = 0.0f;
    v4f q[CF];
#pragma unroll
    for (int j = 0; j <= RF; ++j) {
      v8i fn;
      float sn = 0.0f;
      if (j + 1 < RF) {
        fn = p.rr.fp8(tr, j + 1, (j + 1) * 16);
        sn = row_scale(j + 1);
      }
#pragma unroll
      for (int i = 0; i < CF; ++i) {
        const v4f was = q[i];
        if (j < RF) q[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fc[i], fr, v4f{}, 0, 0, 0, 0, 0, 0);
        if (j > 0) {
          const float by = sp * (SPLIT && i >= S::CF ? w1 : w0);
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[i][j - 1][x] = __builtin_fmaf(was[x], by, acc[i][j - 1][x]);
          acc[i][j - 1] = pin(acc[i][j - 1]);                // here, not after the loop's branches
        }
      }
      fr = fn;
      sp = sr;
      sr = sn;
      __builtin_amdgcn_sched_barrier(0);
    }
    w0 = w0n;
    w1 = w1n;
  }
}

// The same on the 256 x 256 tile, after p.begin(): its first NQ quarters.
// A pair of matrix instructions is scaled and added while the next pair runs.
template <int NQ, bool CSTR, bool SPLIT, bool BYTES, class Acc, class Fetch>
__device__ __forceinline__ void product256(Acc &acc, const Pipe256<CSTR, false, 1, SPLIT> &p, const lds_u8 *area, int wm,
                                           int lane, const_floats sw, int64_t step_w, int64_t up, Fetch fetch_scales) {
  auto row_scale = [&](int t, int q, int f) {
    const uint32_t v = *(const __attribute__((address_space(3))) uint32_t *)(
        area + (t & 3) * 1024 + (q * 64 + wm * 32 + f * 16 + (lane & 15)) * 4);
    return BYTES ? e8m0_decode(v) : __uint_as_float(v);
  };
  p.template meet0<1, 0>(false);
  v8i fc[4], fr[2][2];
  float sr[2][2], coef[2][2];
  v4f part[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    fr[0][f] = p.read_r8(0, 0, f);
    sr[0][f] = row_scale(0, 0, f);
    part[1][f] = v4f{};
    coef[1][f] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) fc[i] = p.read_c(0, i);
  float w[2] = {sw[0], SPLIT ? sw[up] : 0.0f};
  auto add = [&](int q, int i, int from) {                   // the pair (q, i)
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      v4f &a = acc[i][2 * q + f];
#pragma unroll
      for (int x = 0; x < 4; ++x) a[x] = __builtin_fmaf(part[from][f][x], coef[from][f], a[x]);
      a = pin(a);                                            // here, not after the loop's branches
    }
  };
  auto step = [&](int t, auto edge) {
    constexpr bool kEdge = decltype(edge)::value;
    const int next_t = kEdge ? min(t + 1, p.steps - 1) : t + 1;
    const float wn[2] = {sw[next_t * step_w], SPLIT ? sw[next_t * step_w + up] : 0.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 1) p.template meet1<1, kEdge, 0>(t, false);
      if (q == 3) p.template meet3<1, kEdge, 0>(t, false);
      const bool next = !kEdge || t + 1 < p.steps;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (q < NQ) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            part[i & 1][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fc[i], fr[q & 1][f], v4f{}, 0, 0, 0, 0, 0, 0);
            coef[i & 1][f] = sr[q & 1][f] * w[SPLIT ? i >> 1 : 0];
          }
          __builtin_amdgcn_sched_barrier(0);
          if (i > 0) add(q, i - 1, (i & 1) ^ 1);
          else if (q > 0) add(q - 1, 3, 1);
          else add(NQ - 1, 3, 1);                            // of the stage before (zeros before the first)
        }
        if (i < 2) {
          if (q + 1 < NQ) {
            fr[(q + 1) & 1][i] = p.read_r8(t, q + 1, i);
            sr[(q + 1) & 1][i] = row_scale(t, q + 1, i);
          } else if (q == 3 && next) {
            fr[0][i] = p.read_r8(t + 1, 0, i);
            sr[0][i] = row_scale(t + 1, 0, i);
          }
          p.template fetch<kEdge>(t, q, i);
        } else if (i == 2 && q == 1 && (!kEdge || t + 2 < p.steps)) {
          fetch_scales(t + 2);
        }
        // this stage's column fragment has been used for the last time
        if (q == 3 && next) fc[i] = p.read_c(t + 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    w[0] = wn[0];
    w[1] = wn[1];
  };
  int t = 0;
  for (; t + 2 < p.steps; ++t) step(t, Flag<false>());
  for (; t < p.steps; ++t) step(t, Flag<true>());
  add(NQ - 1, 3, 1);
}

// Fragments (i, j) of a wave: columns col + 16 i .. (gated: gate, then up), the
// tile's rows row_of(j) + 0..15.
template <bool GATED, int RF, int BM, class Acc, class Row>
__device__ __forceinline__ void epilogue(const GmmArgs &p, const RowTile &u, int n0, int wn, int lane, Acc &acc, Row row_of,
                                         uint32_t *top) {
  if constexpr (!GATED) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int n = n0 + (wn * 4 + i) * 16, cols = p.n - n;
#pragma unroll
      for (int j = 0; j < RF; ++j) {
        const int at = row_of(j) + (lane & 15);
        store_bf16_pair(p.out + ((u.row0 + at) * p.n + n) * 2, lane, at < u.rows ? cols : 0, acc[i][j], acc[i + 1][j]);
      }
    }
  } else {
    const int n = n0 + wn * 32;                              // n is a multiple of 128: the tile lies inside
    with_act(p.act, [&](auto kind) {
#pragma unroll
      for (int j = 0; j < RF; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = act<decltype(kind)::value>(acc[i][j][q]) * acc[2 + i][j][q];
    });
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      if (p.out_quant != EP_QUANT_NONE) {
        const uint32_t m = row_amax(acc[0][j], acc[1][j]);
        if (lane < 16) top[wn * BM + row_of(j) + lane] = m;
      }
    }
    if (p.out_quant != EP_QUANT_NONE) lds_barrier();
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      const int at = row_of(j) + (lane & 15);
      const int64_t row = u.row0 + at;
      const bool ok = at < u.rows;
      if (p.out_quant == EP_QUANT_NONE) {
        store_bf16_pair(p.out + (row * p.n + n) * 2, lane, ok ? 32 : 0, acc[0][j], acc[1][j]);
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max(m, top[w * BM + at]);
        const Block128 b = block128(p.out_quant, m);
        store_codes_pair(p.out + row * p.n + n, lane, ok, acc[0][j], acc[1][j], b);
        if (ok && wn == 0 && lane < 16) {
          const int64_t to = row * (p.n / 128) + n0 / 128;
          if (p.out_quant == EP_QUANT_FP8_B128_UE8M0) ((uint8_t *)p.out_scales)[to] = (uint8_t)b.byte;
          else ((float *)p.out_scales)[to] = b.scale;
        }
      }
    }
  }
}

// The tile's part of the weights; `up`: of the up rows.
template <bool CSTR, bool GATED>
__device__ __forceinline__ Source weights_of(const GmmArgs &p, int e, int n0, bool up, int cols) {
  if constexpr (GATED)
    return Source{p.c + ((int64_t)e * 2 * p.n + (up ? p.n : 0) + n0) * p.k, p.k, min(cols, p.n - n0)};
  else if constexpr (CSTR)
    return Source{p.c + (int64_t)e * p.k * p.n + n0, p.n, p.n - n0};
  else
    return Source{p.c + ((int64_t)e * p.n + n0) * p.k, p.k, min(cols, p.n - n0)};
}

// The wave's weight scales: by block of k from `at`, `step` apart; the up
// columns' `up` further.
struct ColumnScales {
  const_floats at;
  int64_t step, up;
};
template <bool CSTR, bool GATED>
__device__ __forceinline__ ColumnScales column_scales(const GmmArgs &p, int e, int n0, int wn) {
  const int kb = p.k / 128, nb_all = GATED ? 2 * p.n / 128 : p.n / 128;
  // a wave has 64 columns or fewer, gated: of one gate and one up block
  const int nb = min(n0 / 128 + (GATED ? 0 : wn * 64 / 128), nb_all - 1);
  return {(const_floats)(p.c_scales + (int64_t)e * nb_all * kb + (CSTR ? nb : (int64_t)nb * kb)), CSTR ? nb_all : 1,
          GATED ? (int64_t)(p.n / 128) * kb : 0};
}

// GATED: gate and up rows in, n columns act(gate) * up out.  The next unit's
// first stages are fetched before the epilogue of a unit.
template <class S, bool CSTR, bool GATED, bool BYTES>
__global__ __launch_bounds__(S::kThreads) void gmm_kernel(GmmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__     // the core uses device-only types
  constexpr int kCols = GATED ? S::BN / 2 : S::BN, kScale = BYTES ? 1 : 4;   // bytes of a row scale in memory
  static_assert(S::CF == 2 && S::WN == 4, "the epilogue's columns");
  typedef ScaleArea<S> A;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds + S::kStages * A::kBytes];
  __shared__ uint32_t top[GATED ? 4 * S::BM : 1];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
  const int wn = wave % S::WN, wm = wave / S::WN, kb = p.k / 128;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int units = uniform(g.first[p.E]) * nc;
  PipeN<S, CSTR, 1, GATED> pipe;
  RowTile u;
  int n0;
  u32x4 scales;
  const int scale_row = (wave * kWave + lane) * kb * kScale;  // rows past the tile's are past the range
  const uint32_t scale_to = (uint32_t)(uintptr_t)lds + S::kLds + wave * kWave * 4;
  auto fetch_scales = [&](int t) {
    if (wave < A::kWaves) load_lds4<BYTES>(scale_to + (t % S::kStages) * A::kBytes, scale_row, scales, t * kScale);
  };
  auto start = [&](int unit) {
    u = row_tile(g, p.E, p.offsets, unit, nc, S::BM);
    n0 = u.tc * kCols;
    scales = descriptor(p.r_scales + u.row0 * kb * kScale, (uint32_t)(u.rows * kb * kScale));
    pipe.init(weights_of<CSTR, GATED>(p, u.e, n0, GATED && wave >= S::kWaves / 2, kCols),
              Source{p.r + u.row0 * p.k, p.k, u.rows}, p.k, lds, wave, lane);
    pipe.begin(fetch_scales);
  };
  int unit = unit_of_round(0);
  if (unit >= units) return;
  start(unit);
  for (int round = 1;; ++round) {
    constexpr int RF = 2 * S::RF;
    v4f acc[4][RF];
    const ColumnScales w = column_scales<CSTR, GATED>(p, u.e, n0, wn);
    product<S, CSTR, GATED, BYTES>(acc, pipe, lds + S::kLds, wave, lane, w.at, w.step, w.up, fetch_scales);
    lds_barrier();                                           // the stages are free
    const RowTile done = u;
    const int done_n0 = n0;
    unit = unit_of_round(round);
    if (unit < units) start(unit);
    epilogue<GATED, RF, S::BM>(p, done, done_n0, wn, lane, acc, [&](int j) { return (wm * RF + j) * 16; }, top);
    if (unit >= units) return;
  }
#endif
}

template <bool CSTR, bool GATED, bool BYTES>
__global__ __launch_bounds__(Tile256::kThreads) void gmm256_kernel(GmmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef Tile256 S;
  constexpr int kCols = GATED ? S::BN / 2 : S::BN, kScale = BYTES ? 1 : 4;
  // two stages, then four stages' row scales
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds + 4 * 1024];
  __shared__ uint32_t top[GATED ? 4 * S::BM : 1];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
  const int wn = S::wn(wave), kb = p.k / 128;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const Plan256 plan = plan_units(uniform(g.first[p.E]), nc);
  const int units = plan.units;
  Pipe256<CSTR, false, 1, GATED> pipe;
  RowTile u;
  int n0;
  u32x4 scales;
  // waves w and w + 4 fetch the same rows' scales: as many loads in every wave
  const int scale_row = ((wave & 3) * kWave + lane) * kb * kScale;
  const uint32_t scale_to = (uint32_t)(uintptr_t)lds + S::kLds + (wave & 3) * kWave * 4;
  auto fetch_scales = [&](int t) { load_lds4<BYTES>(scale_to + (t & 3) * 1024, scale_row, scales, t * kScale); };
  auto start = [&](int unit) {
    u = row_tile256(g, plan, p.E, p.offsets, unit, nc);
    n0 = u.tc * kCols;
    scales = descriptor(p.r_scales + u.row0 * kb * kScale, (uint32_t)(u.rows * kb * kScale));
    pipe.init(weights_of<CSTR, GATED>(p, u.e, n0, false, kCols), weights_of<CSTR, GATED>(p, u.e, n0, true, kCols),
              Source{p.r + u.row0 * p.k, p.k, u.rows}, p.k, lds, wave, lane);
    pipe.begin(fetch_scales);
  };
  int unit = unit_of_round(0);
  if (unit >= units) return;
  start(unit);
  for (int round = 1;; ++round) {
    v4f acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = v4f{};
    const ColumnScales w = column_scales<CSTR, GATED>(p, u.e, n0, wn);
    const lds_u8 *area = lds + S::kLds;
    const int wm = S::wm(wave);
    if (u.rows > 192) product256<4, CSTR, GATED, BYTES>(acc, pipe, area, wm, lane, w.at, w.step, w.up, fetch_scales);
    else if (u.rows > 128) product256<3, CSTR, GATED, BYTES>(acc, pipe, area, wm, lane, w.at, w.step, w.up, fetch_scales);
    else if (u.rows > 64) product256<2, CSTR, GATED, BYTES>(acc, pipe, area, wm, lane, w.at, w.step, w.up, fetch_scales);
    else product256<1, CSTR, GATED, BYTES>(acc, pipe, area, wm, lane, w.at, w.step, w.up, fetch_scales);
    lds_barrier();                                           // the stages are free
    const RowTile done = u;
    const int done_n0 = n0;
    unit = unit_of_round(round);
    if (unit < units) start(unit);
    epilogue<GATED, 8, S::BM>(p, done, done_n0, wn, lane, acc,
                              [&](int j) { return S::row(wave, j >> 1, (j & 1) * 16); }, top);
    if (unit >= units) return;
  }
#endif
}

// Few rows an expert, bf16 out: the wave's sums are joined and wave w has
// fragment i = w of both row fragments (gated: columns 16 (w % 2) .. of row
// fragment w / 2).  Bounded by the weights' bytes (at TileFew).
template <bool GATED, bool BYTES>
__global__ __launch_bounds__(TileFew::kThreads) void few_kernel(GmmArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef TileFew S;
  constexpr int kCols = GATED ? 32 : 64, kScale = BYTES ? 1 : 4;
  constexpr int kArea = kWave * 4;                           // row scales of a stage: a dword a lane
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds + S::kWaves * S::kBuffers * kArea];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave), kb = p.k / 128;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int units = uniform(g.first[p.E]) * nc;
  PipeFew<1> pipe;
  pipe.init(p.k, p.k, p.k, lds, wave, lane);
  struct Unit {
    RowTile u;
    int n0;
    const_floats sw;                                         // the unit's weight scales by block of k
  };
  u32x4 scales;                                              // row scales of the unit being fetched
  const lds_u8 *area = lds + S::kLds + wave * S::kBuffers * kArea;
  const uint32_t area_to = (uint32_t)(uintptr_t)area;
  const int scale_row = lane * kb * kScale;                  // rows past the tile's are past the range
  // 64 columns lie in one block of 128 (gated: 32 gate and 32 up columns)
  const int nb_all = GATED ? 2 * p.n / 128 : p.n / 128;
  const int64_t up = GATED ? (int64_t)(p.n / 128) * kb : 0;
  v4f acc[4][2];
  few_units<1, 1>(
      pipe, units,
      [&](int unit) {
        Unit x{row_tile(g, p.E, p.offsets, unit, nc, S::BM), 0, nullptr};
        x.n0 = x.u.tc * kCols;
        x.sw = (const_floats)(p.c_scales + ((int64_t)x.u.e * nb_all + x.n0 / 128) * kb);
        scales = descriptor(p.r_scales + x.u.row0 * kb * kScale, (uint32_t)(x.u.rows * kb * kScale));
        pipe.c[0] = weights_of<false, GATED>(p, x.u.e, x.n0, false, 32);
        pipe.c[1] = GATED ? weights_of<false, GATED>(p, x.u.e, x.n0, true, 32)
                          : Source{pipe.c[0].base + 32 * pipe.c[0].pitch, pipe.c[0].pitch, 32};
        pipe.r = Source{p.r + x.u.row0 * p.k, p.k, x.u.rows};
        return x;
      },
      [&](int t, int b) { load_lds4<BYTES>(area_to + b * kArea, scale_row, scales, t * kScale); },
      [&](const Unit &) {
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c][0] = acc[c][1] = v4f{};
      },
      [&](const Unit &now, int i, int b) {
        const int t = pipe.first + i * S::kWaves;
        const float w[2] = {now.sw[t], GATED ? now.sw[t + up] : 0.0f};
        const lds_u8 *at = pipe.stage(b);
        v8i fr[2];
        float sr[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          fr[j] = pipe.rd.fp8(at + 64 * kKBytes, 0, j * 16);
          const uint32_t v =
              *(const __attribute__((address_space(3))) uint32_t *)(area + b * kArea + (j * 16 + (lane & 15)) * 4);
          sr[j] = BYTES ? e8m0_decode(v) : __uint_as_float(v);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v8i fc = pipe.rd.fp8(at, 0, c * 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const v4f q = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fc, fr[j], v4f{}, 0, 0, 0, 0, 0, 0);
            const float by = sr[j] * w[GATED ? c >> 1 : 0];
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[c][j][x] = __builtin_fmaf(q[x], by, acc[c][j][x]);
          }
        }
      },
      [&](const Unit &done, auto join) {
        typedef __attribute__((address_space(3))) v4f lds_v4f;
        const int own = join(wave);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) *(lds_v4f *)(lds + own + ((c * 2 + j) * kWave + lane) * 16) = acc[c][j];
        lds_barrier();
        // gated: gate and up of one fragment; else one column fragment, both row fragments
        const int first = GATED ? (wave & 1) * 2 + (wave >> 1) : wave * 2, second = GATED ? first + 4 : first + 1;
        v4f a = {}, b = {};
#pragma unroll
        for (int w = 0; w < S::kWaves; ++w) {
          const int at = join(w);
          a += *(const lds_v4f *)(lds + at + (first * kWave + lane) * 16);
          b += *(const lds_v4f *)(lds + at + (second * kWave + lane) * 16);
        }
        lds_barrier();                                       // before a stage goes there
        auto store4 = [](char *dst, const v4f &v) {
          *(u32x2 *)dst = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        };
        const int row = (lane & 15) + (GATED ? wave >> 1 : 0) * 16;
        const int n = done.n0 + (GATED ? wave & 1 : wave) * 16 + 4 * (lane >> 4);
        char *dst = p.out + ((done.u.row0 + row) * p.n + n) * 2;
        if constexpr (GATED) {
          with_act(p.act, [&](auto kind) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = act<decltype(kind)::value>(a[i]) * b[i];
          });
          if (row < done.u.rows) store4(dst, a);
        } else {
          if (row < done.u.rows) store4(dst, a);
          if (row + 16 < done.u.rows) store4(dst + (int64_t)16 * p.n * 2, b);
        }
      });
#endif
}

template <int BM>
struct ShapeOf;
template <>
struct ShapeOf<32> : Shape<2, 1, 4, 1, 4> {};
template <>
struct ShapeOf<64> : Shape<2, 1, 4, 2, 3> {};
template <>
struct ShapeOf<128> : Shape<2, 2, 4, 2, 3> {};
template <>
struct ShapeOf<256> : Tile256 {};

template <bool CSTR, bool GATED, bool BYTES>
hipError_t launch(const GmmArgs &p, int64_t pairs, hipStream_t s) {
  const int cols = GATED ? 128 : 256;
  const int64_t nc = (p.n + cols - 1) / cols, used = p.E < pairs ? p.E : pairs;
  // (a block's scale takes 128 columns of a tile)
  const bool few = !CSTR && p.out_quant == EP_QUANT_NONE;
  return with_height(pairs, p.E, nc, few, [&](auto bm) {
    constexpr int BM = decltype(bm)::value;
    if constexpr (BM == 0) {
      if constexpr (!CSTR) {
        const int64_t units = (pairs / 32 + used) * (p.n / (GATED ? 32 : 64));
        hipLaunchKernelGGL((few_kernel<GATED, BYTES>), dim3((unsigned)persistent_grid(units)), dim3(TileFew::kThreads), 0,
                           s, p);
      }
    } else {
      typedef ShapeOf<BM> S;
      const int64_t tiles = (pairs + BM - 1) / BM + used;
      // 256-row tiles may be cut in 4
      const dim3 grid((unsigned)persistent_grid(tiles * nc * (BM == 256 ? 4 : 1))), block(S::kThreads);
      if constexpr (BM == 256) hipLaunchKernelGGL((gmm256_kernel<CSTR, GATED, BYTES>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((gmm_kernel<S, CSTR, GATED, BYTES>), grid, block, 0, s, p);
    }
    return hipGetLastError();
  });
}

template <bool BYTES>
hipError_t by_form(const GmmArgs &p, const GmmB128Args &a, int64_t pairs, hipStream_t s) {
  if (a.transposed) return launch<true, false, BYTES>(p, pairs, s);
  return a.act == EP_ACT_NONE ? launch<false, false, BYTES>(p, pairs, s) : launch<false, true, BYTES>(p, pairs, s);
}

}  // namespace

hipError_t launch_gmm_b128(const GmmB128Args &a, hipStream_t s) {
  const int64_t pairs = a.h.num_tokens * a.h.num_topk < a.h.max_rows ? a.h.num_tokens * a.h.num_topk : a.h.max_rows;
  if (pairs == 0) return hipSuccess;
  const int n = a.act != EP_ACT_NONE ? a.n / 2 : a.n;
  GmmArgs p{a.h.offsets, a.recv_count, a.h.num_experts, a.a, a.a + recv_geom(a.h.max_rows, a.k, a.a_quant).scale_off,
            (const char *)a.w, a.w_scales, a.k, n, a.act, a.out_quant, a.out, nullptr};
  if (a.out_quant != EP_QUANT_NONE) p.out_scales = a.out + recv_geom(a.h.max_rows, n, a.out_quant).scale_off;
  return a.a_quant == EP_QUANT_FP8_B128_UE8M0 ? by_form<true>(p, a, pairs, s) : by_form<false>(p, a, pairs, s);
}

}  // namespace ep
