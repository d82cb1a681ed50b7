// Gated feed-forward block over expert rows, forward and backward (bf16):
//   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a W2^T
//   da = dy W2,  dg = da u act'(g),  du = da act(g)
//   dx = [dg du] W1,  dW1 = [dg du]^T x,  dW2 = dy^T a
// Every product runs on the core of gemm_core.hpp: both projections, the
// activation, the product of the two and the checkpoint in one launch; the
// activation's gradient in the epilogue of dy W2.
//
// Roundings to bf16: a, dg and du, because they are the next product's operands
// on the matrix cores; the checkpoint (or e4m3 with a scale per 128); the
// outputs.  Sums, the activation and its gradient are float32.
//
// Launches: forward 2, backward 3 (dy W2 with a, dg, du; dx; both weight
// gradients).  What bounds them, and what they take:
//   few rows an expert    the weights' bytes (figures at TileFew)
//   32 to 192 rows        a few tiles a CU: the last round and the stages' latency.
//                         64 experts of 129 rows, 2048 -> 2 x 768, 8-bit checkpoint:
//                         gate and up 161 us, down 63, dy W2 72, dx 108, weights 209
//   many                  the matrix cores at the clock that the power limit leaves.
//                         32768 rows in 32 experts, 7168 -> 2 x 2048: gate and up
//                         1.61 ms (1.20 PFLOP/s), down 0.90 (1.07), dy W2 1.12 (0.86:
//                         its epilogue reads and writes 540 MB, and does so in part
//                         behind the next unit's stages), dx 1.79 (1.08), weights 2.87
//                         (1.01: sums of 1024 rows, 2.8 GB written)
// (medians of a profiled run whose inputs change from pass to pass; another
// card of this kind took 4 to 6 % longer)
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

// The product over k of a tile, after p.begin(): acc[c][r] = C fragment c . R
// fragment r.  Fragments are read one k step of 16 ahead, across the stages'
// borders: the waves meet before the last step's matrix instructions, which
// then cover the first reads of the next stage.
template <class S, bool CSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product(Acc &acc, const PipeN<S, CSTR, 2, SPLIT> &p) {
  auto none = [](int) {};
#pragma unroll
  for (int i = 0; i < S::CF; ++i)
#pragma unroll
    for (int j = 0; j < S::RF; ++j) acc[i][j] = v16f{};
  bf16x8 fc[2][S::CF], fr[2][S::RF];
  auto read = [&](int t, int s, int to) {
    const lds_u8 *tc = p.stage_c(t), *tr = p.stage_r(t);
#pragma unroll
    for (int i = 0; i < S::CF; ++i) fc[to][i] = p.rc.bf16(tc, i, p.c_index(i), s);
#pragma unroll
    for (int j = 0; j < S::RF; ++j) fr[to][j] = p.rr.bf16(tr, j, j * 32, s);
  };
  p.template meet<0>(0, false, none);
  read(0, 0, 0);
  for (int t = 0; t < p.steps; ++t) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read(t, s + 1, (s + 1) & 1);
      } else if (t + 1 < p.steps) {
        p.template meet<0>(t + 1, false, none);
        read(t + 1, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < S::RF; ++j)
#pragma unroll
        for (int i = 0; i < S::CF; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[s & 1][i], fr[s & 1][j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The same on the 256 x 256 tile, after p.begin(): its first NQ quarters.
template <int NQ, int STORES, bool CSTR, bool RSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product256(Acc &acc, const Pipe256<CSTR, RSTR, 2, SPLIT> &p, bool after) {
  p.template meet0<0, STORES>(after);
  bf16x8 fc[2][4], fr[2][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    fr[0][s] = p.read_r(0, 0, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) fc[i][s] = p.read_c(0, i, s);
  }
  // EDGE: t may be the first stage or one of the last two
  auto step = [&](int t, auto edge) {
    constexpr bool kEdge = decltype(edge)::value;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 1) p.template meet1<0, kEdge, STORES>(t, after);
      if (q == 3) p.template meet3<0, kEdge, STORES>(t, after);
      const bool next = !kEdge || t + 1 < p.steps;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (q < NQ) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fc[i][s], fr[q & 1][s], acc[i][q], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (q + 1 < NQ) fr[(q + 1) & 1][s] = p.read_r(t, q + 1, s);
        if (q == 3 && next) {
          // this step's column fragments have been used for the last time
          fr[0][s] = p.read_r(t + 1, 0, s);
#pragma unroll
          for (int i = 0; i < 2; ++i) fc[i][s] = p.read_c(t + 1, i, s);
        }
        if (s < 2) p.template fetch<kEdge>(t, q, s);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int t = 0;
  if (STORES) step(t++, Flag<true>());
  for (; t + 2 < p.steps; ++t) step(t, Flag<false>());
  for (; t < p.steps; ++t) step(t, Flag<true>());
}

// `rows`: valid rows of the tile (each height has a loop of its own: branches
// between the quarters cost more than the quarters they left out).
// STORES, after: of the pipe's meetings.
template <int STORES, bool CSTR, bool RSTR, bool SPLIT, class Acc>
__device__ __forceinline__ void product256(Acc &acc, const Pipe256<CSTR, RSTR, 2, SPLIT> &p, int rows, bool after) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v16f{};
  if (p.steps == 0) return;
  if (rows > 192) product256<4, STORES>(acc, p, after);
  else if (rows > 128) product256<3, STORES>(acc, p, after);
  else if (rows > 64) product256<2, STORES>(acc, p, after);
  else product256<1, STORES>(acc, p, after);
}

// Eight values of the checkpoint.
[[maybe_unused]] __device__ __forceinline__ void decode8(u32x4 q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(q[i]);
    v[2 * i + 1] = bf16_hi(q[i]);
  }
}

// What becomes of a tile's accumulators.  A wave's fragment (i, j) holds 32
// output columns (of the gate and of the up rows: the same) and the tile's rows
// row_of(j) + 0..31.
//   top         LDS [2][4][BM]: largest magnitudes (8-bit checkpoint)
template <int RF, int BM, int ACT, class Acc, class Row>
__device__ __forceinline__ void epilogue_up(const RowArgs &p, const RowTile &u, int n0, int wn, int lane, Acc &acc,
                                            Row row_of, uint32_t *top) {
  const int half = lane >> 5, n = n0 + wn * 32, cols = p.n - n;
  if (p.ck_form == kCkFp8) {
#pragma unroll
    for (int j = 0; j < RF; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t m = row_amax(acc[i][j]);
        if (half == 0) top[(i * 4 + wn) * BM + row_of(j) + lane] = m;
      }
    lds_barrier();
  }
#pragma unroll
  for (int j = 0; j < RF; ++j) {
    const int at = row_of(j) + (lane & 31);
    const bool ok = at < u.rows && cols > 0;
    const int64_t row = u.row0 + at;
    const v16f &gt = acc[0][j], &up = acc[1][j];
    float a[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = act<ACT>(gt[i]) * up[i];
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
        for (int w = 0; w < 4; ++w) m = max(m, top[(i * 4 + w) * BM + at]);
        const Block128 b = block128(EP_QUANT_FP8_B128, m);
        store_codes(p.ck + row * 2 * p.n + i * p.n + n, half, ok, acc[i][j], b);
        if (ok && wn == 0 && half == 0) p.ck_scales[row * (2 * p.n / 128) + (i * p.n + n0) / 128] = b.scale;
      }
    }
  }
}

// da in acc: dg, du and a to memory.  The next fragment's checkpoint is asked
// for before a fragment is worked on; rows and columns past the tile's read its
// first ones.  On 256-row tiles the kernel needs 11 registers more than there
// are: those are read back here, each time behind everything in flight (the next
// unit's first stages, the stores, the checkpoint), so that the loads overlap
// with the work in part only, and this is the slowest of the row products.
template <int RF, int ACT, bool FP8, class Acc, class Row>
__device__ __forceinline__ void epilogue_act(const RowArgs &p, const RowTile &u, int n0, int wn, int lane, Acc &acc,
                                             Row row_of) {
  const int half = lane >> 5;
  struct Piece {
    u32x4 g[2], u[2];                      // 8 values each: bf16, or e4m3 in the first two words
    float sg, su;
  };
  auto load = [&](int f) {
    const int i = f / RF, j = f % RF, at = row_of(j) + (lane & 31), n = n0 + (wn * 2 + i) * 32;
    const int64_t row = u.row0 + (at < u.rows ? at : 0);
    const int col = (n < p.n ? n : n0) + 8 * half;
    Piece q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t to = row * 2 * p.n + col + 16 * h;
      if constexpr (FP8) {
        const u32x2 a = *(const u32x2 *)(p.ck + to), b = *(const u32x2 *)(p.ck + to + p.n);
        q.g[h] = u32x4{a.x, a.y, 0, 0};
        q.u[h] = u32x4{b.x, b.y, 0, 0};
      } else {
        q.g[h] = *(const u32x4 *)(p.ck + to * 2);
        q.u[h] = *(const u32x4 *)(p.ck + (to + p.n) * 2);
      }
    }
    if constexpr (FP8) {
      const float *s = p.ck_scales + row * (2 * p.n / 128);
      q.sg = s[col / 128];
      q.su = s[(p.n + col) / 128];
    }
    return q;
  };
  Piece next = load(0);
#pragma unroll
  for (int f = 0; f < 2 * RF; ++f) {
    const Piece q = next;
    if (f + 1 < 2 * RF) next = load(f + 1);
    const int i = f / RF, j = f % RF, at = row_of(j) + (lane & 31), n = n0 + (wn * 2 + i) * 32;
    const int64_t row = u.row0 + at;
    float da[16];
    columns_of(acc[i][j], da);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float gt[8], up[8], dg[8], du[8], a[8];
      if constexpr (FP8) {
        e4m3x8_decode(u32x2{q.g[h].x, q.g[h].y}, gt);
        e4m3x8_decode(u32x2{q.u[h].x, q.u[h].y}, up);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          gt[x] *= q.sg;
          up[x] *= q.su;
        }
      } else {
        decode8(q.g[h], gt);
        decode8(q.u[h], up);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float v, dv;
        act_grad<ACT>(gt[x], v, dv);
        dg[x] = da[8 * h + x] * up[x] * dv;
        du[x] = da[8 * h + x] * v;
        a[x] = v * up[x];
      }
      const int col = n + 16 * h + 8 * half;
      if (at < u.rows && col < p.n) {
        char *d = p.d + (row * 2 * p.n + col) * 2;
        store8_bf16(d, dg);
        store8_bf16(d + (int64_t)p.n * 2, du);
        store8_bf16(p.out + (row * p.n + col) * 2, a);
      }
    }
  }
}

template <int MODE, int RF, int BM, class Acc, class Row>
__device__ __forceinline__ void epilogue(const RowArgs &p, const RowTile &u, int n0, int wn, int lane, Acc &acc, Row row_of,
                                         uint32_t *top) {
  if constexpr (MODE == kUp) {
    with_act(p.act, [&](auto a) { epilogue_up<RF, BM, decltype(a)::value>(p, u, n0, wn, lane, acc, row_of, top); });
  } else if constexpr (MODE == kGradAct) {
    if (u.rows <= 0) return;
    with_act(p.act, [&](auto a) {
      if (p.ck_form == kCkFp8) epilogue_act<RF, decltype(a)::value, true>(p, u, n0, wn, lane, acc, row_of);
      else epilogue_act<RF, decltype(a)::value, false>(p, u, n0, wn, lane, acc, row_of);
    });
  } else {
    const int half = lane >> 5;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = n0 + (wn * 2 + i) * 32, cols = p.n - n;
#pragma unroll
      for (int j = 0; j < RF; ++j) {
        const int at = row_of(j) + (lane & 31);
        store_bf16(p.out + ((u.row0 + at) * p.n + n) * 2, half, at < u.rows ? cols : 0, [&](int q) { return acc[i][j][q]; });
      }
    }
  }
}

// The tile's part of the weights; `up`: of the up rows.
template <int MODE>
__device__ __forceinline__ Source weights_of(const RowArgs &p, int e, int n0, bool up, int cols) {
  if constexpr (MODE == kUp)
    return Source{p.c + ((int64_t)e * 2 * p.n + (up ? p.n : 0) + n0) * p.k * 2, (int64_t)p.k * 2, min(cols, p.n - n0)};
  else if constexpr (MODE == kDown)
    return Source{p.c + ((int64_t)e * p.n + n0) * p.k * 2, (int64_t)p.k * 2, min(cols, p.n - n0)};
  else
    return Source{p.c + ((int64_t)e * p.k * p.n + n0) * 2, (int64_t)p.n * 2, p.n - n0};
}

// The next unit's first stages are fetched before the epilogue of a unit.
template <class S, int MODE>
__global__ __launch_bounds__(S::kThreads) void rows_kernel(RowArgs p) {
#ifdef __HIP_DEVICE_COMPILE__     // the core uses device-only types
  constexpr bool kSplit = MODE == kUp, kCStr = MODE == kGradX || MODE == kGradAct;
  constexpr int kCols = kSplit ? S::BN / 2 : S::BN;         // output columns of a tile
  static_assert(S::CF == 2 && S::WN == 4, "the epilogue's columns");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  __shared__ uint32_t top[MODE == kUp ? 2 * 4 * S::BM : 1];
  __shared__ Groups g;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
  const int wn = wave % S::WN, wm = wave / S::WN;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int units = uniform(g.first[p.E]) * nc;
  PipeN<S, kCStr, 2, kSplit> pipe;
  RowTile u;
  int n0;
  auto start = [&](int unit) {
    u = row_tile(g, p.E, p.offsets, unit, nc, S::BM);
    n0 = u.tc * kCols;
    pipe.init(weights_of<MODE>(p, u.e, n0, kSplit && wave >= S::kWaves / 2, kCols),
              Source{p.r + u.row0 * p.k * 2, (int64_t)p.k * 2, u.rows}, p.k, (lds_u8 *)smem, wave, lane);
    pipe.begin([](int) {});
  };
  int unit = unit_of_round(0);
  if (unit >= units) return;                                 // uniform; later rounds only have larger units
  start(unit);
  for (int round = 1;; ++round) {
    v16f acc[S::CF][S::RF];
    product(acc, pipe);
    lds_barrier();                                           // the stages are free
    const RowTile done = u;
    const int done_n0 = n0;
    unit = unit_of_round(round);
    if (unit < units) start(unit);
    epilogue<MODE, S::RF, S::BM>(p, done, done_n0, wn, lane, acc, [&](int j) { return (wm * S::RF + j) * 32; }, top);
    if (unit >= units) return;
  }
#endif
}

// The same on 256 x 256 tiles: the next unit's first stages are fetched before
// the epilogue of a unit.
template <int MODE>
__global__ __launch_bounds__(Tile256::kThreads) void rows256_kernel(RowArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef Tile256 S;
  constexpr bool kSplit = MODE == kUp, kCStr = MODE == kGradX || MODE == kGradAct;
  constexpr int kCols = kSplit ? S::BN / 2 : S::BN;
  // whole lines out through LDS where the epilogue is a plain store
  constexpr bool kLines = MODE == kDown || MODE == kGradX;
  constexpr int kStores = kLines ? kTileStores : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds + (kLines ? kStoreLds : 0)];
  __shared__ uint32_t top[MODE == kUp ? 2 * 4 * S::BM : 1];
  __shared__ Groups g;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
  const int nc = (p.n + kCols - 1) / kCols;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const Plan256 plan = plan_units(uniform(g.first[p.E]), nc);
  const int units = plan.units;
  Pipe256<kCStr, false, 2, kSplit> pipe;
  RowTile u;
  int n0;
  auto start = [&](int unit) {
    u = row_tile256(g, plan, p.E, p.offsets, unit, nc);
    n0 = u.tc * kCols;
    pipe.init(weights_of<MODE>(p, u.e, n0, false, kCols), weights_of<MODE>(p, u.e, n0, true, kCols),
              Source{p.r + u.row0 * p.k * 2, (int64_t)p.k * 2, u.rows}, p.k, (lds_u8 *)smem, wave, lane);
    pipe.begin([](int) {});
  };
  int unit = unit_of_round(0);
  if (unit >= units) return;
  start(unit);
  for (int round = 1;; ++round) {
    v16f acc[2][4];
    product256<kStores>(acc, pipe, u.rows, round > 1);
    lds_barrier();                                           // the stages are free
    const RowTile done = u;
    const int done_n0 = n0;
    unit = unit_of_round(round);
    if (unit < units) start(unit);
    if constexpr (kLines)
      store_tile256(acc, (lds_u8 *)smem + S::kLds, p.out + (done.row0 * p.n + done_n0) * 2, (int64_t)p.n * 2, done.rows,
                    p.n - done_n0, wave, lane);
    else
      epilogue<MODE, 4, S::BM>(p, done, done_n0, S::wn(wave), lane, acc, [&](int j) { return S::row(wave, j, 0); }, top);
    if (unit >= units) return;
  }
#endif
}

// Few rows an expert (kUp without an 8-bit checkpoint, kDown): sums joined over
// the waves, wave w then has columns 8 w + 4 (l / 32) + 0..3 of row l % 32.
// Bounded by the weights' bytes, in small models by the launch (at TileFew).
template <int MODE>
__global__ __launch_bounds__(TileFew::kThreads) void few_kernel(RowArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef TileFew S;
  constexpr bool kSplit = MODE == kUp;
  constexpr int kCols = kSplit ? 32 : 64;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  __shared__ Groups g;
  lds_u8 *lds = (lds_u8 *)smem;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave), half = lane >> 5;
  scan_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count, S::BM);
  const int nc = (p.n + kCols - 1) / kCols;
  const int units = uniform(g.first[p.E]) * nc;
  PipeFew<2> pipe;
  pipe.init((int64_t)p.k * 2, (int64_t)p.k * 2, p.k, lds, wave, lane);
  struct Unit {
    RowTile u;
    int n0;
  };
  v16f acc[2];
  few_units<2, 0>(
      pipe, units,
      [&](int unit) {
        Unit x{row_tile(g, p.E, p.offsets, unit, nc, S::BM), 0};
        x.n0 = x.u.tc * kCols;
        pipe.c[0] = weights_of<MODE>(p, x.u.e, x.n0, false, 32);
        pipe.c[1] = kSplit ? weights_of<MODE>(p, x.u.e, x.n0, true, 32)
                           : Source{pipe.c[0].base + 32 * pipe.c[0].pitch, pipe.c[0].pitch, 32};
        pipe.r = Source{p.r + x.u.row0 * p.k * 2, (int64_t)p.k * 2, x.u.rows};
        return x;
      },
      [](int, int) {}, [&](const Unit &) { acc[0] = acc[1] = v16f{}; },
      [&](const Unit &, int, int b) {
        const lds_u8 *at = pipe.stage(b);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const bf16x8 r = pipe.rd.bf16(at + 64 * kKBytes, 0, 0, s);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pipe.rd.bf16(at, 0, c * 32, s), r, acc[c], 0, 0, 0);
        }
      },
      [&](const Unit &done, auto join) {
        typedef __attribute__((address_space(3))) v4f lds_v4f;
        const int own = join(wave);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *(lds_v4f *)(lds + own + ((c * 4 + b) * kWave + lane) * 16) =
                v4f{acc[c][4 * b], acc[c][4 * b + 1], acc[c][4 * b + 2], acc[c][4 * b + 3]};
        lds_barrier();
        v4f sum[2] = {};
#pragma unroll
        for (int w = 0; w < S::kWaves; ++w) {
          const int at = join(w);
#pragma unroll
          for (int c = 0; c < 2; ++c) sum[c] += *(const lds_v4f *)(lds + at + ((c * 4 + wave) * kWave + lane) * 16);
        }
        lds_barrier();                                       // before a stage goes there
        const int64_t row = done.u.row0 + (lane & 31);
        if ((lane & 31) >= done.u.rows) return;
        auto store4 = [](char *dst, const v4f &v) {
          *(u32x2 *)dst = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        };
        const int n = done.n0 + 8 * wave + 4 * half;
        if constexpr (kSplit) {
          v4f a;
          with_act(p.act, [&](auto kind) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = act<decltype(kind)::value>(sum[0][i]) * sum[1][i];
          });
          store4(p.out + (row * p.n + n) * 2, a);
          if (p.ck_form == kCkBf16) {
            char *q = p.ck + (row * 2 * p.n + n) * 2;
            store4(q, sum[0]);
            store4(q + (int64_t)p.n * 2, sum[1]);
          }
        } else {
          store4(p.out + (row * p.n + n) * 2, sum[0]);
          store4(p.out + (row * p.n + n + 32) * 2, sum[1]);
        }
      });
#endif
}

struct WeightArgs {
  const int *offsets;
  const int64_t *recv_count;
  int E;
  struct {
    const char *r, *c;     // [rows, nr] and [rows, nc] bf16
    int nr, nc;
    char *out;             // [E, nr, nc] bf16
  } of[2];
};

// out[e] = R_e^T C_e over the rows of expert e (zeros without rows), for both
// weights in one launch: fewer units left over, and the last units, where
// they would fill at most half of a round, are cut into 2 or 4 pieces.  Both
// operands are k strided and are read through the transposing LDS reads.  A sum
// is as long as an expert's rows, so short ones are bounded by the gradients'
// bytes: 64 experts of 129 rows, 2048 x 2 x 768 and 768 x 2048: 604 MB written
// in 209 us (240 before the stores left in whole lines, unwaited).  One expert
// of 8192 rows, 4096 x 2 x 1408 and 1408 x 4096: 326 us, 870 TFLOP/s (272 tiles
// on 256 CUs).
__global__ __launch_bounds__(Tile256::kThreads) void weights256_kernel(WeightArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef Tile256 S;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds + kStoreLds];
  __shared__ Groups g;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
  order_rows<S::kThreads>(g, p.E, p.offsets, p.recv_count);
  auto tiles = [](int n) { return (n + 255) / 256; };
  const int per0 = tiles(p.of[0].nr) * tiles(p.of[0].nc), per = per0 + tiles(p.of[1].nr) * tiles(p.of[1].nc);
  const int grid = (int)gridDim.x, all = per * p.E, over = all % grid;
  const int parts = over * 4 <= grid ? 4 : over * 2 <= grid ? 2 : 1;
  const int whole = all - over, units = whole + over * parts;
  Pipe256<true, true, 2, false> pipe;
  int e, r0, c0, rows_out, which, nr, nc;
  auto start = [&](int unit) {
    int piece = 0, height = 256;
    if (unit >= whole) {
      piece = (unit - whole) % parts;
      unit = whole + (unit - whole) / parts;
      height = 256 / parts;
    }
    const int place = unit / per;
    e = uniform(g.order[place]);
    const int rows = uniform(g.rows[e]);
    int local = unit - place * per;
    which = uniform((int)(local >= per0));
    if (which) local -= per0;
    nr = uniform(which ? p.of[1].nr : p.of[0].nr);
    nc = uniform(which ? p.of[1].nc : p.of[0].nc);
    int tr, tc;
    tile_of_unit(local, tiles(nr), tiles(nc), tr, tc);
    r0 = uniform(tr * 256 + piece * height);
    c0 = uniform(tc * 256);
    rows_out = uniform(max(min(height, nr - r0), 0));
    const int64_t row0 = p.offsets[e];
    const char *rb = which ? p.of[1].r : p.of[0].r, *cb = which ? p.of[1].c : p.of[0].c;
    const Source c{cb + uniform((row0 * nc + c0) * 2), (int64_t)nc * 2, nc - c0};
    pipe.init(c, c, Source{rb + uniform((row0 * nr + r0) * 2), (int64_t)nr * 2, rows_out}, rows, (lds_u8 *)smem, wave, lane);
    pipe.begin([](int) {});
  };
  int unit = unit_of_round(0);
  if (unit >= units) return;
  start(unit);
  for (int round = 1;; ++round) {
    v16f acc[2][4];
    product256<kTileStores>(acc, pipe, rows_out, round > 1);
    lds_barrier();
    const int done_nc = nc, done_c0 = c0, done_rows = rows_out;
    char *out = (which ? p.of[1].out : p.of[0].out) + (((int64_t)e * nr + r0) * nc + c0) * 2;
    unit = unit_of_round(round);
    if (unit < units) start(unit);
    store_tile256(acc, (lds_u8 *)smem + S::kLds, out, (int64_t)done_nc * 2, done_rows, done_nc - done_c0, wave, lane);
    if (unit >= units) return;
  }
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

template <int MODE>
hipError_t rows_launch(const RowArgs &p, int64_t pairs, hipStream_t s) {
  const int cols = MODE == kUp ? 128 : 256;
  const int64_t nc = (p.n + cols - 1) / cols, used = p.E < pairs ? p.E : pairs;
  // (a checkpoint's scale takes 128 columns of a tile)
  const bool few = MODE == kDown || (MODE == kUp && p.ck_form != kCkFp8);
  return with_height(pairs, p.E, nc, few, [&](auto bm) {
    constexpr int BM = decltype(bm)::value;
    if constexpr (BM == 0) {
      if constexpr (MODE == kDown || MODE == kUp) {
        const int64_t units = (pairs / 32 + used) * (p.n / (MODE == kUp ? 32 : 64));
        hipLaunchKernelGGL(few_kernel<MODE>, dim3((unsigned)persistent_grid(units)), dim3(TileFew::kThreads), 0, s, p);
      }
    } else {
      typedef ShapeOf<BM> S;
      const int64_t tiles = (pairs + BM - 1) / BM + used;
      // 256-row tiles may be cut in 4
      const dim3 grid((unsigned)persistent_grid(tiles * nc * (BM == 256 ? 4 : 1))), block(S::kThreads);
      if constexpr (BM == 256) hipLaunchKernelGGL(rows256_kernel<MODE>, grid, block, 0, s, p);
      else hipLaunchKernelGGL((rows_kernel<S, MODE>), grid, block, 0, s, p);
    }
    return hipGetLastError();
  });
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

hipError_t weights_launch(const WeightArgs &p, hipStream_t s) {
  typedef Tile256 S;
  int64_t tiles = 0;
  for (const auto &o : p.of) tiles += (int64_t)((o.nr + 255) / 256) * ((o.nc + 255) / 256);
  hipLaunchKernelGGL(weights256_kernel, dim3((unsigned)persistent_grid(tiles * 4 * p.E)), dim3(S::kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn(const FfnArgs &f, hipStream_t s) {
  const int64_t pairs = pairs_of(f.h);
  if (pairs == 0) return hipSuccess;
  char *a = f.ws + ffn_ws(f.h.max_rows, f.inter, 0).a;
  const hipError_t e = rows_launch<kUp>(row_args(f, f.x, f.w1, f.hidden, f.inter, a), pairs, s);
  if (e != hipSuccess) return e;
  return rows_launch<kDown>(row_args(f, a, f.w2, f.inter, f.hidden, f.out), pairs, s);
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
    if ((e = rows_launch<kGradAct>(p, pairs, s)) != hipSuccess) return e;
    if ((e = rows_launch<kGradX>(row_args(f, d, f.w1, 2 * f.inter, f.hidden, g.grad_x), pairs, s)) !=
        hipSuccess)
      return e;
  }
  return weights_launch({f.h.offsets, f.recv_count, f.h.num_experts,
                         {{d, (const char *)f.x, 2 * f.inter, f.hidden, (char *)g.grad_w1},
                          {(const char *)g.grad_out, a, f.hidden, f.inter, (char *)g.grad_w2}}},
                        s);
}

}  // namespace ep
