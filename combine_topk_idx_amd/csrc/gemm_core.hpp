// Grouped matrix-product core of the feed-forward block (ffn.hip) and the
// block-scaled product (gmm_b128.hip) on gfx950.
//
// A workgroup computes one BN x BM tile of out[row][col] = sum_k R[row][k]
// C[col][k]: "R" are the rows of an expert's block, "C" the operand whose
// index runs along an output row.  C is the matrix instructions' first
// operand, so a lane's accumulators are consecutive output columns of one
// row (vector stores, one row scale a lane).
//
// Operand tiles cover 128 bytes of k (64 bf16 or 128 e4m3) and come in two
// forms: k contiguous in memory ([index][k], LDS rows of 128 bytes), or k
// strided ([k][index], LDS rows of one k), which gfx950's transposing LDS
// reads turn into fragments.  Tiles go from memory to LDS without passing
// through registers, 16 bytes a lane; a lane's LDS place is fixed by the
// instruction, so the 16-byte chunks of a row are permuted by choosing which
// chunk each lane fetches, such that the fragment reads of a wave spread over
// all LDS banks.  Rows and columns past the end of an operand are out of the
// range of the buffer descriptor and arrive as zeros.
#pragma once

#include "common.hpp"
#include "formats.hpp"
#include "ring.hpp"

namespace ep {

// Workgroups of a launch of at most that many units (moe.hip): no more than
// CUs -- the stages fill a CU's LDS -- and a multiple of the XCD count.
int64_t persistent_grid(int64_t units_upper);

namespace gemm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <int N>
struct Int {
  static constexpr int value = N;
};
template <bool B>
struct Flag {
  static constexpr bool value = B;
};

constexpr int kXcds = 8;
constexpr int kKBytes = 128;              // bytes of k in a stage

// A value that is the same in every lane, kept in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)v) | (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32);
}

// ---------------------------------------------------------------------------
// which tile a workgroup computes
// ---------------------------------------------------------------------------

struct Groups {                           // the experts' rows, in LDS
  int first[kMaxExperts + 1];             // first row tile of each expert; [E] = all
  int rows[kMaxExperts];
  int order[kMaxExperts];                 // experts by descending row count (weight gradients)
};

// Rows of expert e: recv_count when given, never more than its block.
__device__ __forceinline__ int expert_rows(const int *__restrict__ offsets, const int64_t *__restrict__ recv_count,
                                           int e) {
  const int block = offsets[e + 1] - offsets[e];
  return recv_count ? (int)min((int64_t)block, max(recv_count[e], (int64_t)0)) : max(block, 0);
}

// Fills g.rows and the exclusive scan of the experts' tiles of `bm` rows.
template <int THREADS>
__device__ __forceinline__ void scan_rows(Groups &g, int E, const int *__restrict__ offsets,
                                          const int64_t *__restrict__ recv_count, int bm) {
  constexpr int kPer = (kMaxExperts + THREADS - 1) / THREADS, kWaves = THREADS / kWave;
  __shared__ int wsum[kWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
  int tiles[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = tid * kPer + q;
    const int n = e < E ? expert_rows(offsets, recv_count, e) : 0;
    tiles[q] = (n + bm - 1) / bm;
    sum += tiles[q];
    if (e < E) g.rows[e] = n;
  }
  int x = sum;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == kWave - 1) wsum[wv] = x;
  __syncthreads();
  int before = x - sum, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    before += i < wv ? wsum[i] : 0;
    all += wsum[i];
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = tid * kPer + q;
    if (e < E) g.first[e] = before;
    before += tiles[q];
  }
  if (tid == 0) g.first[E] = all;
  __syncthreads();
}

// Fills g.rows and g.order (a product over an expert's rows takes time in
// their number: the longest first).
template <int THREADS>
__device__ __forceinline__ void order_rows(Groups &g, int E, const int *__restrict__ offsets,
                                           const int64_t *__restrict__ recv_count) {
  for (int e = threadIdx.x; e < E; e += THREADS) g.rows[e] = expert_rows(offsets, recv_count, e);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {
    const int n = g.rows[e];
    int at = 0;
    for (int i = 0; i < E; ++i) at += g.rows[i] > n || (g.rows[i] == n && i < e);
    g.order[at] = e;
  }
  __syncthreads();
}

// Workgroup b runs on XCD b % 8 (the hardware deals them out in turn); in
// each round an XCD takes consecutive units, which share operands in its L2.
__device__ __forceinline__ int unit_of_round(int round) {
  const int slots = (int)gridDim.x / kXcds;
  return (round * kXcds + (int)blockIdx.x % kXcds) * slots + (int)blockIdx.x / kXcds;
}

// Units of nr x nc tiles in groups kGroupRows row tiles deep: the units in
// flight on an XCD form a compact rectangle.
constexpr int kGroupRows = 8;
__device__ __forceinline__ void tile_of_unit(int local, int nr, int nc, int &tr, int &tc) {
  const int per = kGroupRows * nc, g = local / per, rem = local - g * per;
  const int depth = min(kGroupRows, nr - g * kGroupRows);
  tc = rem / depth;
  tr = g * kGroupRows + rem - tc * depth;
}

// The rows and column tile of a unit (expert-major, uniform).
struct RowTile {
  int e, rows, tc;
  int64_t row0;
};
__device__ __forceinline__ RowTile row_tile(const Groups &g, int E, const int *__restrict__ offsets, int unit,
                                            int nc, int bm) {
  const int item = unit / nc;
  int lo = 0, hi = E;                                        // the last expert whose first tile is <= item
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (g.first[mid] <= item) lo = mid; else hi = mid;
  }
  RowTile u;
  u.e = __builtin_amdgcn_readfirstlane(lo);
  const int rows = __builtin_amdgcn_readfirstlane(g.rows[u.e]);
  int tr;
  tile_of_unit(unit - g.first[u.e] * nc, (rows + bm - 1) / bm, nc, tr, u.tc);
  tr = __builtin_amdgcn_readfirstlane(tr);
  u.tc = __builtin_amdgcn_readfirstlane(u.tc);
  u.row0 = (int64_t)offsets[u.e] + (int64_t)tr * bm;
  u.rows = min(bm, rows - tr * bm);
  return u;
}

// Height of a launch's row tiles from its mean rows an expert (256 columns a
// tile; gated: 128).  Measured on 64 experts of 129 rows (2048 -> 2 x 768, 8-bit
// checkpoint; 32, 64, 128, 256 rows): gate and up 202, 157, 177, 177 us, dy W2
// 102, 69, 97, 87 us -- under 2.5 rounds of 128-row tiles the last, nearly empty
// round costs more than the weights read once more for each 64 rows; a W2 103,
// 78, 62, 66 us, its gradient 172, 130, 104, 106 us, at 2.8 rounds.  16 experts
// of 127 rows, 2 column tiles: 17, 21, 30, 27 us, by the CUs that have a unit.
// Many rows an expert: 256-row tiles (half the bytes a product), whose
// leftover ones are cut.
// Up to 32 rows an expert, `few`: TileFew (launch(Int<0>())).
// (640 and 128 units: 2.5 rounds and half a round of 256 CUs.)
template <class F>
__host__ inline hipError_t with_height(int64_t pairs, int64_t E, int64_t nc, bool few, F launch) {
  const int64_t used = E < pairs ? E : pairs, mean = pairs / used;
  if (mean <= 32 && few) return launch(Int<0>());
  auto units = [&](int bm) { return (pairs / bm + (used + 1) / 2) * nc; };
  if (mean > 192) return launch(Int<256>());
  if (mean > 32 && units(128) >= 640) return launch(Int<128>());
  if (mean > 32 && units(64) >= 128) return launch(Int<64>());
  return launch(Int<32>());
}

// ---------------------------------------------------------------------------
// staging
// ---------------------------------------------------------------------------

struct Source {                           // uniform over a wave
  const char *base;                       // the tile's first element at k = 0
  int64_t pitch;                          // bytes between rows of the matrix in memory
  int valid;                              // indexes (rows of the tile) inside the operand
};

// A buffer descriptor: base, range in bytes (reads past it give zeros).
__device__ __forceinline__ u32x4 descriptor(const char *base, uint32_t bytes) {
  const uint64_t a = (uint64_t)base;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}

// 16 bytes a lane from memory to LDS: lane l's go to lds + 16 l.  Written as
// assembly because the compiler, which cannot tell the stages apart, would
// wait for every such load before the next LDS read: wait_stage() does the
// waiting.  (The loads have no destination registers; nothing else in these
// kernels uses m0.)
// `first`: of a group with one descriptor, which a vector instruction may have
// written just before (five wait states).
__device__ __forceinline__ void load_lds16(uint32_t lds, int voff, u32x4 desc, int soff, bool first) {
  if (first)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(desc), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(desc), "s"(soff)
                 : "memory");
}

// One dword, or one byte extended to a dword, a lane: lane l's goes to lds + 4 l.
template <bool BYTE>
__device__ __forceinline__ void load_lds4(uint32_t lds, int voff, u32x4 desc, int soff) {
  if (BYTE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(desc), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(desc), "s"(soff)
                 : "memory");
}

// Loads the wave's share of a tile of ROWS indexes: pieces of 1 KB.
//   SPLIT   the first half of the indexes comes from one source, the second
//           half from another (gate and up rows): the caller gives each wave
//           its own
template <int ROWS, bool STRIDED, int EB, int WAVES, bool SPLIT>
struct Loader {
  static constexpr int kTile = ROWS * kKBytes;
  static constexpr int kPieces = kTile / 1024;
  // a tile of fewer pieces than waves: some waves fetch the same piece, so
  // that every wave has the same number of loads in flight
  static constexpr int kLoads = kPieces >= WAVES ? kPieces / WAVES : 1;
  static constexpr int kPitch = ROWS * EB;                // LDS bytes of one k (strided)
  static constexpr int kSteps = kKBytes / EB;             // k of a stage
  int voff[kLoads];
  int lds0;

  // chunk permutation of one k's row (strided form): a fragment read of bf16
  // covers 64 bytes of 4 k in 32 lanes, one of e4m3 16 bytes of 16 k
  static_assert(!STRIDED || kPitch >= 256, "rows of one k span all banks");
  static __device__ __forceinline__ int strided_key(int k) {
    return EB == 2 ? (k & 3) << 2 : (k & 7) << 1 | ((k >> 4) & 1);
  }

  __device__ __forceinline__ void init(int wave, int lane, const Source &s) {
    const int p0 = kPieces >= WAVES ? wave * kLoads : wave % kPieces;
    lds0 = p0 * 1024;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int at = (p0 + j) * 1024 + lane * 16;         // the lane's place in the tile
      if constexpr (STRIDED) {
        const int k = at / kPitch, chunk = (at % kPitch) / 16;
        const int col = (chunk ^ strided_key(k)) * (16 / EB);
        // past the operand's columns: past the descriptor's range
        voff[j] = col < s.valid ? (int)(k * s.pitch) + col * EB : 0x7fffff00;
      } else {
        const int row = at / kKBytes, chunk = (at % kKBytes) / 16;
        const int local = SPLIT ? row % (ROWS / 2) : row;
        voff[j] = local * (int)s.pitch + (chunk ^ ((row >> 1) & 7)) * 16;
      }
    }
  }

  // stage t of k; `steps_left`: k from this stage on (strided form)
  __device__ __forceinline__ void load(lds_u8 *tile, const Source &s, int t, int64_t k_left) const {
    u32x4 r;
    int soff = 0;
    if constexpr (STRIDED) {
      const int64_t rows = k_left < kSteps ? k_left : kSteps;
      r = descriptor(s.base + (int64_t)t * kSteps * s.pitch, (uint32_t)(rows * s.pitch));
    } else {
      r = descriptor(s.base, (uint32_t)(s.valid * s.pitch));
      soff = t * kKBytes;
    }
    const uint32_t to = (uint32_t)(uintptr_t)tile + lds0;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load_lds16(to + j * 1024, voff[j], r, soff, j == 0);
  }
};

// Fragment reads.
//   bf16 (32x32x16): lane l holds index l % 32, k = 8 (l / 32) + 0..7 of step s
//   e4m3 (16x16x128): lane l holds index l % 16, k = 16 (l / 16) + 0..15 and
//   the same + 64
// (both operands alike: the order of k inside an instruction is free).
template <int ROWS, bool STRIDED, int EB, int FRAGS>
struct Reader {
  static constexpr int kPitch = ROWS * EB;
  static constexpr int kIndexes = EB == 2 ? 32 : 16;      // of a fragment
  static constexpr int kAddrs = STRIDED ? FRAGS : (EB == 2 ? 4 : 2);
  typedef Loader<ROWS, STRIDED, EB, 4, false> L;
  int addr[kAddrs];

  // fragment f begins at tile index row0 + index_of(f)
  template <class F>
  __device__ __forceinline__ void init(int lane, int row0, F index_of) {
    if constexpr (STRIDED) {
      const int j = lane & 15, g = lane >> 4;
#pragma unroll
      for (int f = 0; f < FRAGS; ++f) {
        const int at = row0 + index_of(f);
        if constexpr (EB == 2) {
          const int k = 8 * (g >> 1) + (j >> 2);
          const int chunk = at / 8 + 2 * (g & 1) + ((j & 3) >> 1);
          addr[f] = k * kPitch + (chunk ^ L::strided_key(k)) * 16 + (j & 1) * 8;
        } else {
          const int k = 16 * g + (j >> 1);
          addr[f] = k * kPitch + (at / 16 ^ L::strided_key(k)) * 16 + (j & 1) * 8;
        }
      }
    } else {
      const int r = row0 + (lane & (kIndexes - 1)), key = (r >> 1) & 7;
#pragma unroll
      for (int s = 0; s < kAddrs; ++s)
        addr[s] = r * kKBytes + ((EB == 2 ? 2 * s + (lane >> 5) : 4 * s + (lane >> 4)) ^ key) * 16;
    }
  }

  // bf16 fragment f of k step s (0..3); index: index_of(f)
  __device__ __forceinline__ bf16x8 bf16(const lds_u8 *tile, int f, int index, int s) const {
    if constexpr (STRIDED) {
      const lds_u8 *p = tile + addr[f] + s * 16 * kPitch;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
      const s16x4 b =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p + 4 * kPitch));
      const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(bf16x8, v);
    } else {
      return *(const __attribute__((address_space(3))) bf16x8 *)(tile + addr[s] + index * kKBytes);
    }
  }

  // e4m3 fragment f
  __device__ __forceinline__ v8i fp8(const lds_u8 *tile, int f, int index) const {
    if constexpr (STRIDED) {
      const lds_u8 *p = tile + addr[f];
      v2i q[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        q[t] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) v2i *)(p + (64 * (t >> 1) + 8 * (t & 1)) * kPitch));
      return v8i{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
    } else {
      const u32x4 a = *(const __attribute__((address_space(3))) u32x4 *)(tile + addr[0] + index * kKBytes);
      const u32x4 b = *(const __attribute__((address_space(3))) u32x4 *)(tile + addr[1] + index * kKBytes);
      return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    }
  }
};

// Waits until at most N of the wave's loads are in flight; its LDS reads are
// done; then (wait_stage) for the other waves.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_waves() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A barrier that orders LDS accesses alone: loads in flight stay there.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  wait_waves();
}
template <int N>
__device__ __forceinline__ void wait_stage() {
  wait_loads<N>();
  wait_waves();
}

// Tile shape: WN x WM waves of CF x RF fragments of 32 x 32, STAGES tiles of k
// in LDS.
template <int CF_, int RF_, int WN_, int WM_, int STAGES_>
struct Shape {
  static constexpr int CF = CF_, RF = RF_, WN = WN_, WM = WM_, kStages = STAGES_;
  static constexpr int kWaves = WN * WM, kThreads = kWaves * kWave;
  static constexpr int BN = 32 * CF * WN, BM = 32 * RF * WM;
  static constexpr int kStage = (BN + BM) * kKBytes;
  static constexpr int kLds = kStage * kStages;
};

// The operands of a tile of Shape S on their way through N = S::kStages stages:
// stage t + N - 1 is fetched when every wave has read stage t - 1.  Three or
// four small stages instead of two large ones: with a few tiles a CU the time is
// the stages' latency (on 64-row tiles a stage takes a wave 256 matrix-core
// cycles, far less than a load from memory), so what counts is how many are on
// their way.
//   EXTRA   more loads a stage that `extra(t)` issues, in the first
//           `extra_waves` waves
template <class S, bool CSTR, int EB, bool SPLIT>
struct PipeN {
  typedef Loader<S::BN, CSTR, EB, S::kWaves, SPLIT> LC;
  typedef Loader<S::BM, false, EB, S::kWaves, false> LR;
  static constexpr int kLoads = LC::kLoads + LR::kLoads, N = S::kStages, kSteps = kKBytes / EB;
  static constexpr int kCFrags = EB == 2 ? S::CF : 2 * S::CF, kRFrags = EB == 2 ? S::RF : 2 * S::RF;
  static constexpr int kWide = EB == 2 ? 32 : 16;
  LC lc;
  LR lr;
  Reader<S::BN, CSTR, EB, kCFrags> rc;
  Reader<S::BM, false, EB, kRFrags> rr;
  Source c, r;
  int64_t k_all;
  int steps;
  lds_u8 *lds;

  // split: the wave's first half of fragments are gate rows, the others the same up rows
  static __device__ __forceinline__ int c_index(int f) {
    return SPLIT ? f / (kCFrags / 2) * (S::BN / 2) + f % (kCFrags / 2) * kWide : f * kWide;
  }
  __device__ __forceinline__ void init(const Source &cs, const Source &rs, int64_t k, lds_u8 *l, int wave, int lane) {
    c = cs;
    r = rs;
    k_all = k;
    steps = (int)((k + kSteps - 1) / kSteps);
    lds = l;
    lc.init(wave, lane, c);
    lr.init(wave, lane, r);
    const int wn = wave % S::WN, wm = wave / S::WN;
    rc.init(lane, wn * (SPLIT ? S::CF * 16 : S::CF * 32), [](int f) { return c_index(f); });
    rr.init(lane, wm * S::RF * 32, [](int f) { return f * kWide; });
  }
  __device__ __forceinline__ const lds_u8 *stage_c(int t) const { return lds + (t % N) * S::kStage; }
  __device__ __forceinline__ const lds_u8 *stage_r(int t) const { return stage_c(t) + S::BN * kKBytes; }
  template <class F>
  __device__ __forceinline__ void fetch(int t, F extra) const {
    lds_u8 *at = lds + (t % N) * S::kStage;
    lc.load(at, c, t, k_all - (int64_t)t * kSteps);
    lr.load(at + S::BN * kKBytes, r, t, k_all - (int64_t)t * kSteps);
    extra(t);
  }
  // Before the loop, as soon as the stages are free.
  template <class F>
  __device__ __forceinline__ void begin(F extra) const {
    for (int t = 0; t < N - 1 && t < steps; ++t) fetch(t, extra);
  }
  // Stage t is there and no wave reads stage t - 1 any more.
  template <int EXTRA, class F>
  __device__ __forceinline__ void meet(int t, bool with_extra, F extra) const {
    if (t + N - 2 >= steps) wait_loads<0>();
    else if (EXTRA && with_extra) wait_loads<(kLoads + EXTRA) * (N - 2)>();
    else wait_loads<kLoads * (N - 2)>();
    wait_waves();
    if (t + N - 1 < steps) fetch(t + N - 1, extra);
  }
};

// ---------------------------------------------------------------------------
// few rows: 64 columns x 32 rows, k split over the waves
// ---------------------------------------------------------------------------
//
// With a few rows an expert a launch is the weights' way through the chip.
// Each of four waves takes every fourth stage of k through three buffers of
// its own, so nothing but its own loads holds it up; the sums are joined in
// wave order through LDS.  64 columns (gated: 32 gate rows and the same 32 up
// rows) make units enough for the whole card in small models.  k contiguous
// operands.  Measured: 5 tokens, two of 8 experts 1024 -> 2 x 512, bf16 gate and
// up 7.7 us, down 5.9 (together 19 with common stages): launch, first load and
// join; 128 tokens, 6 of 64 experts 2048 -> 2 x 768: 403 MB of gate and up
// weights in 82 us, 4.9 TB/s, 201 MB of down weights in 46 (85 and 49 when a
// unit's first stages were fetched after the last of the one before had
// arrived); 128 tokens, 8 of 256 e4m3 experts 7168 -> 2 x 2048: 7.4 GB in 1165
// us, 6.35 TB/s, the card's rate of reads.
struct TileFew {
  static constexpr int BN = 64, BM = 32, kWaves = 4, kThreads = kWaves * kWave;
  static constexpr int kStage = (BN + BM) * kKBytes, kBuffers = 3;
  static constexpr int kMine = kBuffers * kStage, kLds = kWaves * kMine;
};

// A wave's stages run through its buffers in turn, from one unit into the next:
// two are in flight at any time, also while a unit's sums are joined and
// written.  The sums are joined in the buffer that each wave read last, which is
// the one that no stage in flight goes to.
template <int EB>
struct PipeFew {
  static constexpr int kSteps = kKBytes / EB, kLoads = TileFew::kStage / 1024;
  typedef Loader<32, false, EB, 1, false> L;                 // 32 rows, 4 loads
  Source c[2], r;                                            // columns 0..31, 32..63, of the unit being fetched
  L lc, lr;
  Reader<32, false, EB, 1> rd;
  int all, steps, first;                                     // stages of a unit; the wave's: first, first + 4, ..
  int fetched, flying, to, from;                             // of that unit; in flight; buffers fetched to, read from
  lds_u8 *mine;

  // the waves' stages of a unit
  __device__ __forceinline__ int steps_of(int wave) const { return (all - wave + TileFew::kWaves - 1) / TileFew::kWaves; }
  __device__ __forceinline__ void init(int64_t c_pitch, int64_t r_pitch, int k, lds_u8 *lds, int wave, int lane) {
    lc.init(0, lane, Source{nullptr, c_pitch, 32});
    lr.init(0, lane, Source{nullptr, r_pitch, 32});
    rd.init(lane, 0, [](int) { return 0; });
    first = wave;
    all = k / kSteps;
    steps = steps_of(wave);
    fetched = flying = to = from = 0;
    mine = lds + wave * TileFew::kMine;
  }
  static __device__ __forceinline__ int after(int buffer) { return buffer + 1 == TileFew::kBuffers ? 0 : buffer + 1; }
  __device__ __forceinline__ lds_u8 *stage(int buffer) const { return mine + buffer * TileFew::kStage; }
  // the next stage of the unit being fetched; extra(t, buffer)
  template <class F>
  __device__ __forceinline__ void fetch(F extra) {
    const int t = first + fetched * TileFew::kWaves;
    lds_u8 *at = stage(to);
    lc.load(at, c[0], t, kSteps);
    lc.load(at + 32 * kKBytes, c[1], t, kSteps);
    lr.load(at + 64 * kKBytes, r, t, kSteps);
    extra(t, to);
    to = after(to);
    ++fetched;
    ++flying;
  }
  // The oldest stage in flight is there: in the buffer returned.
  template <int EXTRA>
  __device__ __forceinline__ int arrived() {
    if (flying > 1) wait_loads<kLoads + EXTRA>();
    else wait_loads<0>();
    --flying;
    const int b = from;
    from = after(from);
    return b;
  }
  // Where wave w has its sums, `units`: how many have been read (mod 3).
  __device__ __forceinline__ int join_of(int w, int units) const {
    return w * TileFew::kMine + (units * steps_of(w) + TileFew::kBuffers - 1) % TileFew::kBuffers * TileFew::kStage;
  }
};

// The units of a workgroup on that pipe, one after the other.
//   open(unit)        sets the pipe's sources to a unit's, returns what finish() needs
//   extra(t, buffer)  issues EXTRA more loads with a stage
//   work(now, i, b)   the wave's i-th stage of the unit `now`, in buffer b
//   finish(now, join) the unit's sums are complete in registers; join(w): wave w's place
template <int EB, int EXTRA, class Open, class Extra, class Begin, class Work, class Finish>
__device__ __forceinline__ void few_units(PipeFew<EB> &p, int units, Open open, Extra extra, Begin begin, Work work,
                                          Finish finish) {
  int next = unit_of_round(0);
  if (next >= units) return;                                 // uniform; later rounds only have larger units
  auto now = open(next);
  next = unit_of_round(1);
  auto coming = now;
  bool opened = false;                                       // the next unit, which stages are fetched of
  auto fetch = [&] {
    if (p.fetched == p.steps) {
      if (opened || next >= units || p.steps == 0) return;
      coming = open(next);
      p.fetched = 0;
      opened = true;
    }
    p.fetch(extra);
  };
  for (int round = 2, done = 1;; ++round, done = done == 2 ? 0 : done + 1) {
    begin(now);
    while (p.flying < 2 && p.fetched < p.steps) fetch();     // before the first unit
    for (int i = 0; i < p.steps; ++i) {
      const int b = p.template arrived<EXTRA>();
      if (p.flying < 2) fetch();
      work(now, i, b);
    }
    wait_lds();
    finish(now, [&](int w) { return p.join_of(w, done); });
    if (next >= units) return;
    if (!opened) {                                           // a wave without stages
      coming = open(next);
      p.fetched = 0;
    }
    now = coming;
    opened = false;
    next = unit_of_round(round);
  }
}

// ---------------------------------------------------------------------------
// the 256 x 256 tile
// ---------------------------------------------------------------------------
//
// Eight waves: 4 along the columns, 2 along the rows, two stages of 64 KB.  A
// stage is worked through in quarters of 64 rows (32 a wave; 8 matrix
// instructions of bf16, 8 of e4m3); a wave's column fragments of the whole
// stage stay in registers.  A part of a stage is fetched again (for two
// stages on) as soon as every wave has read it, a quarter of the bytes in
// every quarter:
//   quarter    fetched                         the waves meet first, so that
//   0          row quarters 2, 3 of stage t+1
//   1          row quarters 0, 1 of stage t+2  (row quarters 2, 3 of t are there)
//   2          first half of C of stage t+2
//   3          second half of C of stage t+2   (C, row quarters 0, 1 of t+1 are there)
// which leaves every load at least four quarters (2048 matrix-core cycles)
// and never queues more than two a wave: issued in one burst, the 64 loads of
// a stage held every wave's next instruction back for about 1000 cycles.
// Fragments are read a quarter ahead, between the matrix instructions.
// Why this tile: a 256 x 256 tile reads 128 products a byte fetched, and 128 KB
// of stages with 8 waves of 128 accumulators fill LDS and registers of a CU.
// No LDS bank conflicts are counted; matrix cores are busy 71-73 % of the CUs'
// cycles in bf16 (32768 rows in 32 experts of 7168 -> 2 x 2048: 1.6 ms, 1.2
// PFLOP/s at the 1.8 GHz that the power limit leaves) and 56 % in e4m3, whose
// scaled sums take 37 % in vector instructions, hardly any of them under the
// matrix instructions of the other wave (transposed: 48 and 31 %).  LDS reads are
// active 28, 25 and 22 %.
struct Tile256 {
  static constexpr int BN = 256, BM = 256, kThreads = 512, WN = 4, WM = 2;
  static constexpr int kStage = 512 * kKBytes, kLds = 2 * kStage;
  static constexpr int kR = 256 * kKBytes;               // the row part of a stage
  static __device__ __forceinline__ int wn(int wave) { return wave >> 1; }
  static __device__ __forceinline__ int wm(int wave) { return wave & 1; }
  // row of the tile of row `i` (0..31) of a wave's quarter q
  static __device__ __forceinline__ int row(int wave, int q, int i) { return q * 64 + wm(wave) * 32 + i; }
};

// The units of a launch on 256-row tiles.  Every workgroup takes every
// gridDim-th unit, so a round of units takes as long as its slowest.  Where
// the units past whole rounds would fill at most half of the last one, the
// row tiles they belong to, the launch's last, are cut into 2 or 4 equal
// pieces (352 units of 4096-long sums on 256 CUs: 232 -> 205 us).
// Working off the experts' short last tiles together at the end, by height,
// evens out the rounds too, but reads every expert's weights a second time
// (measured: no faster).
struct Plan256 {
  int whole, parts, units;                // row tiles not cut; pieces of each other one
};
__device__ __forceinline__ Plan256 plan_units(int tiles, int nc) {
  const int grid = (int)gridDim.x, over = tiles * nc % grid;
  Plan256 p{tiles, 1, tiles * nc};
  if (over * 2 <= grid) {
    const int cut = (over + nc - 1) / nc;
    p.parts = over * 4 <= grid ? 4 : 2;
    p.whole = tiles - cut;
    p.units = (p.whole + cut * p.parts) * nc;
  }
  return p;
}

// The rows and column tile of a unit (uniform; rows may be 0).
__device__ __forceinline__ RowTile row_tile256(const Groups &g, const Plan256 &p, int E,
                                               const int *__restrict__ offsets, int unit, int nc) {
  int item = unit / nc, piece = -1;
  const int col = unit - item * nc;
  if (item >= p.whole) {
    const int past = item - p.whole;
    item = p.whole + past / p.parts;
    piece = past % p.parts;
  }
  int lo = 0, hi = E;                                        // the last expert whose first tile is <= item
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (g.first[mid] <= item) lo = mid; else hi = mid;
  }
  RowTile u;
  u.e = uniform(lo);
  const int first = uniform(g.first[u.e]), rows = uniform(g.rows[u.e]);
  int tr = item - first, height = 256, at = 0;
  u.tc = col;
  if (piece >= 0) {
    height = 256 / p.parts;
    at = piece * height;
  } else {
    tile_of_unit(unit - first * nc, min((rows + 255) / 256, p.whole - first), nc, tr, u.tc);
  }
  tr = uniform(tr);
  u.tc = uniform(u.tc);
  at = uniform(at);
  u.row0 = (int64_t)offsets[u.e] + (int64_t)tr * 256 + at;
  u.rows = uniform(max(min(height, rows - tr * 256 - at), 0));
  return u;
}

template <bool CSTR, bool RSTR, int EB, bool SPLIT>
struct Pipe256 {
  static constexpr int kSteps = kKBytes / EB;             // k of a stage
  static_assert(EB == 2 || !RSTR, "e4m3 rows are k contiguous");
  // e4m3 fragments are 16 wide, two to a quarter
  static constexpr int kCFrags = EB == 2 ? 2 : 4, kWide = EB == 2 ? 32 : 16;
  typedef Reader<256, CSTR, EB, kCFrags> RC;
  typedef Reader<RSTR ? 128 : 256, RSTR, EB, 2> RR;
  Source c[2], r[2];                                      // halves of C; row quarters 0, 1 and 2, 3
  int64_t k_all;
  int steps;
  lds_u8 *lds;
  uint32_t to;                                            // the wave's place in a half
  int vc[2], vr[RSTR ? 2 : 1][2];
  RC rc;
  RR rr;

  static __device__ __forceinline__ int c_index(int f) {
    if constexpr (EB == 2) return f * (SPLIT ? 128 : 32);
    else return SPLIT ? f / 2 * 128 + f % 2 * 16 : f * 16;
  }

  // c_hi: the second half's source of a split operand (else unused); k: the
  // reduction's length
  __device__ __forceinline__ void init(const Source &cs, const Source &c_hi, const Source &rs, int64_t k, lds_u8 *l,
                                       int wave, int lane) {
    k_all = k;
    steps = (int)((k + kSteps - 1) / kSteps);
    lds = l;
    to = (uint32_t)(uintptr_t)l + wave * 2048;
    c[0] = cs;
    if constexpr (SPLIT) c[1] = c_hi;
    else if constexpr (CSTR) c[1] = Source{cs.base + kSteps / 2 * cs.pitch, cs.pitch, cs.valid};
    else c[1] = Source{cs.base + 128 * cs.pitch, cs.pitch, max(cs.valid - 128, 0)};
    r[0] = rs;
    r[1] = Source{rs.base + (RSTR ? 128 * EB : 128 * rs.pitch), rs.pitch, max(rs.valid - 128, 0)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = (wave * 2 + j) * 1024 + lane * 16;     // in a half
      if constexpr (CSTR) {
        const int row = at / (256 * EB), chunk = at % (256 * EB) / 16;
        const int col = (chunk ^ RC::L::strided_key(row)) * (16 / EB);
        vc[j] = col < cs.valid ? (int)(row * cs.pitch) + col * EB : 0x7fffff00;
      } else {
        const int row = at / kKBytes, chunk = at % kKBytes / 16;
        vc[j] = row * (int)cs.pitch + (chunk ^ ((row >> 1) & 7)) * 16;
      }
      if constexpr (RSTR) {
        const int row = at / 256, chunk = at % 256 / 16;
        const int col = (chunk ^ RR::L::strided_key(row)) * (16 / EB);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          vr[h][j] = col < rs.valid - h * 128 ? (int)(row * rs.pitch) + col * EB : 0x7fffff00;
      } else {
        const int row = at / kKBytes, chunk = at % kKBytes / 16;
        vr[0][j] = row * (int)rs.pitch + (chunk ^ ((row >> 1) & 7)) * 16;
      }
    }
    const int wn = Tile256::wn(wave), wm = Tile256::wm(wave);
    rc.init(lane, SPLIT ? wn * 32 : wn * 64, [](int f) { return c_index(f); });
    rr.init(lane, wm * 32, [](int f) { return RSTR ? f * 64 : f * kWide; });
  }

  template <bool STR>
  __device__ __forceinline__ void load(const Source &s, int t, int k0, const int (&v)[2], uint32_t at, int j) const {
    u32x4 d;
    int soff = 0;
    if constexpr (STR) {
      const int64_t left = k_all - (int64_t)t * kSteps - k0;
      const int64_t rows = left < 0 ? 0 : left < kSteps ? left : kSteps;
      d = descriptor(s.base + (int64_t)t * kSteps * s.pitch, (uint32_t)(rows * s.pitch));
    } else {
      d = descriptor(s.base, (uint32_t)(s.valid * s.pitch));
      soff = t * kKBytes;
    }
    load_lds16(at + j * 1024, v[j], d, soff, true);
  }
  // load j (0, 1) of half h of C, of the row quarters 2h, 2h + 1
  __device__ __forceinline__ void load_c(int t, int h, int j) const {
    load<CSTR>(c[h], t, CSTR ? h * (kSteps / 2) : 0, vc, to + (t & 1) * Tile256::kStage + h * 16384, j);
  }
  __device__ __forceinline__ void load_r(int t, int h, int j) const {
    load<RSTR>(r[h], t, 0, vr[RSTR ? h : 0], to + (t & 1) * Tile256::kStage + Tile256::kR + h * 16384, j);
  }
  __device__ __forceinline__ const lds_u8 *stage_c(int t) const { return lds + (t & 1) * Tile256::kStage; }
  __device__ __forceinline__ const lds_u8 *stage_r(int t, int q) const {
    return stage_c(t) + Tile256::kR + (q >> 1) * 16384;
  }
  __device__ __forceinline__ bf16x8 read_c(int t, int f, int s) const { return rc.bf16(stage_c(t), f, c_index(f), s); }
  __device__ __forceinline__ v8i read_c(int t, int f) const { return rc.fp8(stage_c(t), f, c_index(f)); }
  __device__ __forceinline__ bf16x8 read_r(int t, int q, int s) const {
    return rr.bf16(stage_r(t, q), q & 1, (q & 1) * 64, s);
  }
  __device__ __forceinline__ v8i read_r8(int t, int q, int f) const {
    return rr.fp8(stage_r(t, q), 0, (q & 1) * 64 + f * 16);
  }

  // The fetches of quarter q of stage t, j = 0, 1.
  // EDGE: t may be one of the last two stages.
  template <bool EDGE>
  __device__ __forceinline__ void fetch(int t, int q, int j) const {
    if (q == 0) {
      if (!EDGE || t + 1 < steps) load_r(t + 1, 1, j);
    } else if (!EDGE || t + 2 < steps) {
      if (q == 1) load_r(t + 2, 0, j);
      else load_c(t + 2, q - 2, j);
    }
  }
  // Before the loop: stage 0 and, but for its row quarters 2, 3, stage 1;
  // `extra`: issues EXTRA more loads that go with row quarters 0, 1.
  template <class F>
  __device__ __forceinline__ void begin(F extra) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t < steps) {
#pragma unroll
        for (int j = 0; j < 2; ++j) load_r(t, 0, j);
        extra(t);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_c(t, j >> 1, j & 1);
        if (t == 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j) load_r(0, 1, j);
        }
      }
    }
  }
  // STORES: memory instructions that the wave issued between begin() and
  // meet0() and that need not be waited for yet (`after`: whether it did).
  template <int EXTRA, int STORES>
  __device__ __forceinline__ void meet0(bool after) const {
    if (STORES && after) {
      if (steps > 1) wait_stage<8 + EXTRA + STORES>();
      else wait_stage<2 + STORES>();
    } else if (steps > 1) {
      wait_stage<8 + EXTRA>();
    } else {
      wait_stage<2>();
    }
  }
  // The meetings before quarters 1 and 3: loads that may still be in flight are
  // those issued after the ones waited for.
  // EDGE: t may be the first stage or one of the last two.
  template <int EXTRA, bool EDGE, int STORES>
  __device__ __forceinline__ void meet1(int t, bool after) const {
    if (EDGE && STORES && after && t == 0) {
      if (t + 1 < steps) wait_stage<8 + EXTRA + STORES>();
      else wait_stage<STORES>();
    } else if (!EDGE || t + 1 < steps) {
      wait_stage<8 + EXTRA>();
    } else {
      wait_stage<0>();
    }
  }
  template <int EXTRA, bool EDGE, int STORES>
  __device__ __forceinline__ void meet3(int t, bool after) const {
    if (EDGE && STORES && after && t == 0) {
      if (t + 2 < steps) wait_stage<6 + EXTRA + STORES>();
      else if (t + 1 < steps) wait_stage<2 + STORES>();
    } else if (!EDGE || t + 2 < steps) {
      wait_stage<6 + EXTRA>();
    } else if (t + 1 < steps) {
      wait_stage<2>();
    }
  }
};

// ---------------------------------------------------------------------------
// epilogue helpers
// ---------------------------------------------------------------------------

// Accumulator 4b + i of lane l: column 8b + 4 (l / 32) + i of the fragment,
// row l % 32.  Exchanging halves of lanes l and l + 32 gives each lane eight
// consecutive columns: 16p + 8 (l / 32) + 0..7 for p = 0, 1.
__device__ __forceinline__ void swap_halves(uint32_t &x, uint32_t &y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

// Stores a fragment of 16 values a lane as bf16: dst = the row's first
// column of the fragment; columns at or past `cols` are left out (cols is a
// multiple of 8).
template <class F>
__device__ __forceinline__ void store_bf16(char *dst, int half, int cols, F value) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t x0 = pack_bf16x2(value(8 * p), value(8 * p + 1)), x1 = pack_bf16x2(value(8 * p + 2), value(8 * p + 3));
    uint32_t y0 = pack_bf16x2(value(8 * p + 4), value(8 * p + 5)), y1 = pack_bf16x2(value(8 * p + 6), value(8 * p + 7));
    swap_halves(x0, y0);
    swap_halves(x1, y1);
    const int n = 16 * p + 8 * half;
    if (n < cols) *(u32x4 *)(dst + n * 2) = u32x4{x0, x1, y0, y1};
  }
}

// A fragment's values in that order: v[8 p + i] is column 16 p + 8 (l / 32) + i.
__device__ __forceinline__ void columns_of(const v16f &a, float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x = __float_as_uint(a[8 * p + i]), y = __float_as_uint(a[8 * p + 4 + i]);
      swap_halves(x, y);
      v[8 * p + i] = __uint_as_float(x);
      v[8 * p + 4 + i] = __uint_as_float(y);
    }
}
__device__ __forceinline__ void store8_bf16(char *dst, const float *v) {
  *(u32x4 *)dst = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// The same for a pair of 16-column fragments of 16 x 16 (accumulator i of
// lane l: column 4 (l / 16) + i, row l % 16): rows of 16 lanes exchanged, lane
// l has columns pair_column(l) + 0..7 of the pair's 32.
__device__ __forceinline__ int pair_column(int lane) { return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8; }
__device__ __forceinline__ void swap_rows(uint32_t &x, uint32_t &y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}
__device__ __forceinline__ void store_bf16_pair(char *dst, int lane, int cols, const v4f &a, const v4f &b) {
  uint32_t x0 = pack_bf16x2(a[0], a[1]), x1 = pack_bf16x2(a[2], a[3]);
  uint32_t y0 = pack_bf16x2(b[0], b[1]), y1 = pack_bf16x2(b[2], b[3]);
  swap_rows(x0, y0);
  swap_rows(x1, y1);
  const int n = pair_column(lane);
  if (n < cols) *(u32x4 *)(dst + n * 2) = u32x4{x0, x1, y0, y1};
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Stores a 256 x 256 tile of bf16 in whole lines: a wave's 64 columns of 16
// rows pass through 2 KB of its own LDS, so that eight lanes write 128
// consecutive bytes (in fragment order every store instruction would touch 32
// lines with 32 bytes each: the weight gradients of 64 experts of 129 rows spent
// 100 of 241 us on them).  Rows and columns past the tile's are out of the
// descriptor's range: always kTileStores instructions.
constexpr int kTileStores = 16;
constexpr int kStoreLds = 8 * 2048;
template <class Acc>
__device__ __forceinline__ void store_tile256(const Acc &acc, lds_u8 *lds, char *out, int64_t pitch, int rows, int cols,
                                              int wave, int lane) {
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  lds_u8 *mine = lds + wave * 2048;
  const int wn = Tile256::wn(wave), half = lane >> 5, r = lane & 15;
  const __amdgpu_buffer_rsrc_t d =
      __builtin_amdgcn_make_buffer_rsrc(out, 0, (uint32_t)((int64_t)rows * pitch), 0x00020000);
  const int to = wn * 64 < cols ? Tile256::row(wave, 0, lane >> 3) * (int)pitch + (wn * 64 + (lane & 7) * 8) * 2 : 0x7ffffff0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u32x4 q[4];                                              // chunks 4 i + 2 p + half
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const v16f &a = acc[i][j];
        uint32_t x0 = pack_bf16x2(a[8 * p], a[8 * p + 1]), x1 = pack_bf16x2(a[8 * p + 2], a[8 * p + 3]);
        uint32_t y0 = pack_bf16x2(a[8 * p + 4], a[8 * p + 5]), y1 = pack_bf16x2(a[8 * p + 6], a[8 * p + 7]);
        swap_halves(x0, y0);
        swap_halves(x1, y1);
        q[2 * i + p] = u32x4{x0, x1, y0, y1};
      }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      wave_lds_fence();
      if (((lane >> 4) & 1) == pass) {
#pragma unroll
        for (int c = 0; c < 4; ++c) *(lds_u32x4 *)(mine + r * 128 + ((2 * c + half) ^ (r & 7)) * 16) = q[c];
      }
      wave_lds_fence();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (lane >> 3) + 8 * k;
        const u32x4 v = *(const lds_u32x4 *)(mine + row * 128 + ((lane & 7) ^ (row & 7)) * 16);
        __builtin_amdgcn_raw_buffer_store_b128(v, d, to + (j * 64 + pass * 16 + k * 8) * (int)pitch, 0, 0);
      }
    }
  }
}

// Bits of the largest magnitude of a lane's 16 values and of its row's other
// 16 (as integers: a value that is not a number counts as the largest).
__device__ __forceinline__ uint32_t row_amax(const v16f &v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, magnitude(v[i]));
  return max(m, (uint32_t)__shfl_xor((int)m, 32));
}

// The same of a pair of 16 x 16 fragments.
__device__ __forceinline__ uint32_t row_amax(const v4f &a, const v4f &b) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(magnitude(a[i]), magnitude(b[i])));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  return max(m, (uint32_t)__shfl_xor((int)m, 32));
}

// Multiplier and scale of a block of 128 from the bits of its largest
// magnitude: the rules of the per-128 receive formats.  A block that holds an
// infinity or a NaN gets a scale that is not finite.
struct Block128 {
  float m, scale;
  uint32_t byte;                          // the scale's e8m0 form
  bool zero;
};
__device__ __forceinline__ Block128 block128(int quant, uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  const float s0 = amax / 448.0f;
  Block128 b;
  if (quant == EP_QUANT_FP8_B128) {
    b.m = 448.0f / amax;
    b.zero = amax_bits == 0 || __builtin_isinf(b.m);
    b.scale = b.zero ? 0.0f : s0;
    b.byte = 0;
  } else {
    const uint32_t bits = __float_as_uint(s0);
    const bool finite = bits < 0x7f800000u;
    const int e = bits && finite ? ceil_log2_bits(bits) : 0;
    b.zero = bits == 0 || e < -127;
    const int ec = b.zero ? 0 : e;
    b.m = finite ? __uint_as_float((uint32_t)(127 - ec) << 23) : __uint_as_float(0x7fc00000u);
    b.byte = b.zero ? 0u : finite ? (uint32_t)(ec + 127) : 0xffu;
    b.scale = b.zero ? 0.0f : e8m0_decode(b.byte);
  }
  return b;
}

// Four e4m3 codes.
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const Block128 &b) {
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = v[i] * b.m;
    z[i] = x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x;              // NaN stays
  }
  uint32_t q = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], q, true);
  return b.zero ? 0 : q;
}

// e4m3 codes of a fragment (of a pair of 16 x 16 fragments): dst = the row's
// first column.
__device__ __forceinline__ void store_codes(char *dst, int half, bool ok, const v16f &v, const Block128 &b) {
  uint32_t q[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) q[c] = codes4({v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]}, b);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    swap_halves(q[2 * p], q[2 * p + 1]);
    if (ok) *(u32x2 *)(dst + 16 * p + 8 * half) = u32x2{q[2 * p], q[2 * p + 1]};
  }
}
__device__ __forceinline__ void store_codes_pair(char *dst, int lane, bool ok, const v4f &x, const v4f &y,
                                                 const Block128 &b) {
  uint32_t p = codes4({x[0], x[1], x[2], x[3]}, b), q = codes4({y[0], y[1], y[2], y[3]}, b);
  swap_rows(p, q);
  if (ok) *(u32x2 *)(dst + pair_column(lane)) = u32x2{p, q};
}

// The gate's activation.
// e^z as 2^(z log2 e): the product's rounding costs |z| 2^-24 of the value
__device__ __forceinline__ float fast_exp(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504f); }
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-z)); }
// The normal distribution: Phi(-|z|) = tail t P(t) with t = 1 / (1 + 0.3625 |z|)
// and P the polynomial of degree 6 with the smallest largest relative error
// (8e-7) over |z| <= 13.6, below which Phi is no float32; tail: e^(-z^2 / 2),
// which the density needs too.  Relative to the value also far below zero,
// where the up value may be large: within 2^-18 + z^2 2^-23.  (7.1.26 of
// Abramowitz and Stegun, two multiply-adds shorter, bounds the absolute error
// alone: 0.36 % off at z = -6, a bf16 step, and 3.4 % at -12.5.)
__device__ __forceinline__ float normal_cdf(float z, float tail) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.3625f, 1.0f));
  float q = __builtin_fmaf(t, 0.04806285f, -0.17974226f);
  q = __builtin_fmaf(t, q, 0.17510378f);
  q = __builtin_fmaf(t, q, 0.02968257f);
  q = __builtin_fmaf(t, q, 0.13925666f);
  q = __builtin_fmaf(t, q, 0.14293639f);
  q = __builtin_fmaf(t, q, 0.14470038f);
  q = t * q * tail;
  return z > 0.0f ? 1.0f - q : q;
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  return z * (ACT == EP_ACT_SILU ? sigmoid(z) : normal_cdf(z, fast_exp(-0.5f * z * z)));
}

// the activation and its derivative
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float &f, float &df) {
  if constexpr (ACT == EP_ACT_SILU) {
    const float p = sigmoid(z);
    f = z * p;
    df = p + f * (1.0f - p);
  } else {
    const float tail = fast_exp(-0.5f * z * z), p = normal_cdf(z, tail);
    f = z * p;
    df = p + z * 0.39894228f * tail;
  }
}

// Calls f with the activation as a constant: one branch, not one a value.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == EP_ACT_SILU) f(Int<EP_ACT_SILU>());
  else f(Int<EP_ACT_GELU>());
}

}  // namespace gemm
}  // namespace ep
