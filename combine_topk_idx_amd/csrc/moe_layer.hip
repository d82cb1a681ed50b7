// The whole expert layer of a MoE block for a few tokens, in two launches
// (three above 8 tokens): no receive rows, no layout, no combine pass.
//
// What is computed, for token t with ids e_j = topk_idx[t, j]:
//   a_j    = silu(G[e_j] x_t) * (U[e_j] x_t)
//   out[t] = sum over j (ascending) of w[t, j] * (D[e_j] a_j)
// with W1 = [G; U] and W2 = D in bf16, MXFP8 or MXFP4, x and out in bf16.
//
// With few tokens every used expert's weights are read for a handful of
// rows, so the weights' bytes bound the time.  A workgroup owns (a used
// expert, a block of 32-row weight groups); its waves split the reduction
// axis, each streaming its own weight fragments from memory straight into
// registers, and the waves' partial tiles are summed through LDS in a fixed
// order.  Weight codes become bf16 in registers (exactly: a power-of-two scale times
// at most 4 significant bits) and are the A operand of the bf16 matrix
// cores, up to 32 of the expert's tokens the B operand; sums are float32.
//
// Launch 1 ends in SwiGLU and keeps a_j as bf16 rows: one rounding (2^-8 of a value
// at most), where the separate calls quantise it to MXFP8; the output is then off
// by 2.3e-3 of its norm, 1.7e-3 of it from its own rounding to bf16.  Two bf16
// parts would leave the 1.7e-3 and double launch 2's products and row bytes.  Launch 2 leaves its
// float32 rows D a_j in the workspace, and the last workgroup to finish a
// block of output columns (a counter per block, cleared by launch 1) sums
// them over j in ascending order: the result does not depend on which
// workgroup that is.  For more than 8 tokens a third launch sums them, in the
// same order.
#include <math.h>

#include "common.hpp"
#include "formats.hpp"
#include "moe_layer.hpp"
#include "ring.hpp"

namespace ep {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Measured (us, both launches): one token of 256 MXFP8 experts (H 7168, I
// 2048, top 8) 39 + 27 with 4 waves, 2 groups and 2 steps in flight, 39 + 29
// with 3 steps; 128 tokens 1150 + 750, against 1130 + 720; 33 tokens of MXFP4
// experts 93 + 69, against 102 + 79; 13 tokens of bf16 experts 52 + 34, against
// 57 + 42.  With 8 waves launch 2 took a third longer, with 1 group everything
// at least half as long again.
constexpr int kWaves = 4;
constexpr int kGroups = 2;                        // 32-row weight groups of a workgroup
static_assert(kGroups == 2, "hidden and inter are multiples of 64: two groups always divide theirs");
constexpr int kRing = 2;                          // K steps in flight per wave
constexpr int kThreads = kWaves * kWave;
constexpr int kTile = 32;                         // tokens per pass over an expert's weights

// ---------------------------------------------------------------- packing
//
// The fragment order of the MXFP8 packing (see ep_moe_pack_weights) for
// every weight type: lane l = 32g + r of a fragment holds, of the group's
// row r, K [16g, 16g + 16) and [32 + 16g, 48 + 16g) of the 64-wide step.  A
// fragment is 1, 2 or 4 KB (4, 8 or 16 bits a weight) in planes of 1 KB:
// lane l's 16-byte piece p lies at 1024 p + 16 l.
__host__ __device__ inline int group_row(int j, int r, int gate_up, int inter) {
  return gate_up ? (r < 16 ? 16 * j + r : inter + 16 * j + (r - 16)) : 32 * j + r;
}

template <int Q>
__global__ void pack_kernel(const uint8_t *__restrict__ w, const uint8_t *__restrict__ scales, int E, int N, int K,
                            int gate_up, uint8_t *__restrict__ pw, uint8_t *__restrict__ ps) {
  constexpr int kPieces = fragment_bytes(Q) / 1024;
  const int ksteps = K / 64, spans = (ksteps + 3) / 4, groups = N / 32, kb = K / 32, inter = N / 2;
  const int64_t row_bytes = Q == EP_QUANT_NONE ? 2 * (int64_t)K : Q == EP_QUANT_MXFP8 ? (int64_t)K : K / 2;
  const int64_t pieces = (int64_t)E * groups * ksteps * kPieces * 64;
  const int64_t first = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = first; i < pieces; i += stride) {
    const int lane = (int)(i & 63), p = (int)((i >> 6) % kPieces);
    const int64_t rest = (i >> 6) / kPieces;
    const int s = (int)(rest % ksteps);
    const int64_t eg = rest / ksteps;
    const int j = (int)(eg % groups), e = (int)(eg / groups);
    const int r = lane & 31, g = lane >> 5;
    const uint8_t *row = w + ((int64_t)e * N + group_row(j, r, gate_up, inter)) * row_bytes;
    u32x4 v;
    if constexpr (Q == EP_QUANT_NONE) {
      v = *(const u32x4 *)(row + 2 * (s * 64 + (p >> 1) * 32 + g * 16 + (p & 1) * 8));
    } else if constexpr (Q == EP_QUANT_MXFP8) {
      v = *(const u32x4 *)(row + s * 64 + p * 32 + g * 16);
    } else {
      const uint32_t *lo = (const uint32_t *)(row + s * 32 + g * 8), *hi = lo + 4;
      v = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    *(u32x4 *)(pw + ((((int64_t)s * E * groups + eg) * kPieces + p) * 64 + lane) * 16) = v;
  }
  if constexpr (Q != EP_QUANT_NONE) {
    const int64_t words = (int64_t)E * groups * spans * 64;
    for (int64_t i = first; i < words; i += stride) {
      const int lane = (int)(i & 63);
      const int64_t rest = i >> 6;
      const int t = (int)(rest % spans);
      const int64_t eg = rest / spans;
      const int j = (int)(eg % groups), e = (int)(eg / groups);
      const int r = lane & 31, g = lane >> 5;
      const uint8_t *row = scales + ((int64_t)e * N + group_row(j, r, gate_up, inter)) * kb;
      uint32_t word = 0;
      for (int u = 0; u < 4; ++u)
        if (4 * t + u < ksteps) word |= (uint32_t)row[(4 * t + u) * 2 + g] << (8 * u);
      *(uint32_t *)(ps + (((int64_t)t * E * groups + eg) * 64 + lane) * 4) = word;
    }
  }
}

// ------------------------------------------------------ rows of an expert

// Workgroup barrier for LDS hand-offs: the LDS writes before it are waited
// for, global loads in flight are not (__syncthreads would drain them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

constexpr int kIter = (int)(kLayerMaxPairs / kThreads);   // ids per thread, at most

// A call's ids in LDS, as the workgroup that looks for its expert sees them.
struct Ids {
  uint16_t id[kLayerMaxPairs];                    // kNoExpert: none
  uint32_t in_use[kMaxExperts / 32];              // bit set of the experts in use
  int cnt[kIter * kWaves];
};
constexpr uint16_t kNoExpert = 0xffff;

// Reads the ids; the rank-th expert in use (-1: there are fewer) and how many
// are.  Every thread of the workgroup takes part.
template <typename IdxT>
__device__ __forceinline__ int find_expert(const IdxT *__restrict__ idx, int P, int E, int rank, Ids &s, int &used) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  if (tid < kMaxExperts / 32) s.in_use[tid] = 0;
  lds_barrier();
  for (int p = tid; p < P; p += kThreads) {
    const int64_t v = (int64_t)idx[p];
    const bool on = v >= 0 && v < E;
    s.id[p] = on ? (uint16_t)v : kNoExpert;
    if (on) atomicOr(&s.in_use[v >> 5], 1u << (v & 31));
  }
  lds_barrier();
  // the rank-th set bit: every wave counts the 16 words in its first 16 lanes
  const uint32_t word = lane < kMaxExperts / 32 ? s.in_use[lane] : 0u;
  int upto = __popc(word);
#pragma unroll
  for (int d = 1; d < kMaxExperts / 32; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  used = __builtin_amdgcn_readlane(upto, kMaxExperts / 32 - 1);
  if (rank >= used) return -1;                    // uniform
  const int at = __ffsll(__ballot(lane < kMaxExperts / 32 && upto > rank)) - 1;
  uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
  for (int d = rank - (__builtin_amdgcn_readlane(upto, at) - __popc(bits)); d > 0; --d) bits &= bits - 1;
  return at * 32 + __ffs(bits) - 1;
}

// The pairs of `expert` in ascending order, into `list`; returns their
// number.  Every thread takes part.
__device__ __forceinline__ int list_pairs(Ids &s, int P, int expert, uint16_t *list) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
  const int iters = (P + kThreads - 1) / kThreads;
  // pairs in (iteration, wave, lane) order
  for (int i = 0; i < iters; ++i) {
    const int p = i * kThreads + tid;
    const uint64_t mine = __ballot(p < P && s.id[p] == expert);
    if (lane == 0) s.cnt[i * kWaves + wv] = __popcll(mine);
  }
  lds_barrier();
  const int cnt = lane < iters * kWaves ? s.cnt[lane] : 0;
  int sum = cnt;
#pragma unroll
  for (int d = 1; d < kIter * kWaves; d <<= 1) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  for (int i = 0; i < iters; ++i) {
    const int p = i * kThreads + tid, before = __shfl(sum - cnt, i * kWaves + wv);
    const bool on = p < P && s.id[p] == expert;
    const uint64_t mine = __ballot(on);
    if (on) list[before + __popcll(mine & ((1ull << lane) - 1ull))] = (uint16_t)p;
  }
  lds_barrier();
  return __builtin_amdgcn_readlane(sum, kIter * kWaves - 1);
}
static_assert(kIter * kWaves <= kWave, "one count per lane");

// What launch 1 leaves for launch 2 about the rank-th expert in use: its id
// (-1: there are fewer), its pairs, and the number of experts in use.  The
// pairs follow at rank * P of the list.
struct Head {
  int expert, n, used, pad;
};

// -------------------------------------------------------------- fragments

template <int Q>
struct Frag {
  u32x4 p[fragment_bytes(Q) / 1024];
  uint32_t scale;                                 // span dword of this lane's K-block parity
};

// The four bf16 A operands of a fragment: operand m covers K (m >> 1) * 32 +
// 16 g + (m & 1) * 8 .. + 8 of the step.  `u`: the step's byte of the span.
template <int Q>
__device__ __forceinline__ void operands(const Frag<Q> &f, int u, bf16x8 (&a)[4]) {
  if constexpr (Q == EP_QUANT_NONE) {
#pragma unroll
    for (int m = 0; m < 4; ++m) a[m] = __builtin_bit_cast(bf16x8, f.p[m]);
  } else {
    // lane (r, g) holds the scales of K-blocks g: swapping the halves gives
    // both blocks' scales to every lane
    const auto both = __builtin_amdgcn_permlane32_swap(f.scale, f.scale, false, false);
    const float s0 = e8m0_decode((both[0] >> (8 * u)) & 0xff), s1 = e8m0_decode((both[1] >> (8 * u)) & 0xff);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float s = m < 2 ? s0 : s1;
      bf16x2 v0, v1, v2, v3;
      if constexpr (Q == EP_QUANT_MXFP8) {
        const uint32_t lo = f.p[m >> 1][2 * (m & 1)], hi = f.p[m >> 1][2 * (m & 1) + 1];
        v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
        v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
        v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
        v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
      } else {
        const uint32_t w = f.p[0][m];
        v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
        v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
        v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
        v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
      }
      a[m] = bf16x8{v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
    }
  }
}

// Partial products of this wave's share [s0, s1) of the K steps: NG weight
// groups from `wp` (fragments of one step: groups, then lanes) times the
// lane's activation row (K bf16 values), which `row()` finds while the first
// weights are on their way (every wave calls it, so it may hold a barrier).
template <int Q, int NG, typename Row>
__device__ __forceinline__ void product(const uint8_t *wp, size_t wstep, const uint8_t *sp, size_t sspan, int s0,
                                        int s1, Row row, v16f (&acc)[NG]) {
  constexpr int kPieces = fragment_bytes(Q) / 1024;
  const uint32_t lane = threadIdx.x & (kWave - 1), g = lane >> 5;
#pragma unroll
  for (int q = 0; q < NG; ++q) acc[q] = v16f{};
  Frag<Q> w[kRing][NG];
  u32x4 bv[kRing][4];
  auto load_w = [&](int slot, int s) {
#pragma unroll
    for (int q = 0; q < NG; ++q) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        w[slot][q].p[p] = __builtin_nontemporal_load(
            (const u32x4 *)(wp + s * wstep + (size_t)q * fragment_bytes(Q) + p * 1024 + lane * 16));
      if constexpr (Q != EP_QUANT_NONE)
        w[slot][q].scale = *(const uint32_t *)(sp + (size_t)(s >> 2) * sspan + q * 256 + lane * 4);
    }
    keep_loads();
  };
  if (s0 < s1) {                                  // uniform
#pragma unroll
    for (int r = 0; r < kRing; ++r) load_w(r, min(s0 + r, s1 - 1));
  }
  const uint16_t *b = row() + g * 16;
  if (s0 >= s1) return;
  auto load_b = [&](int slot, int s) {
#pragma unroll
    for (int m = 0; m < 4; ++m) bv[slot][m] = *(const u32x4 *)(b + s * 64 + (m >> 1) * 32 + (m & 1) * 8);
    keep_loads();
  };
#pragma unroll
  for (int r = 0; r < kRing; ++r) load_b(r, min(s0 + r, s1 - 1));
  auto multiply = [&](int r, int s) {
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      bf16x8 a[4];
      operands<Q>(w[r][q], s & 3, a);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[m], __builtin_bit_cast(bf16x8, bv[r][m]), acc[q], 0, 0, 0);
    }
  };
  // whole rings without a condition in them (a load whose value only a branch
  // uses is moved into that branch), then the rest
  int s = s0;
  for (; s + kRing <= s1; s += kRing) {
#pragma unroll
    for (int r = 0; r < kRing; ++r) {
      multiply(r, s + r);
      load_w(r, min(s + r + kRing, s1 - 1));      // past the end: the last step again, never used
      load_b(r, min(s + r + kRing, s1 - 1));
    }
  }
#pragma unroll
  for (int r = 0; r < kRing - 1; ++r)
    if (s + r < s1) multiply(r, s + r);           // uniform
}

// The waves' partial tiles through LDS: [wave][group][quad of registers][lane][4].
template <int NG>
__device__ __forceinline__ void leave_partials(float *tile, const v16f (&acc)[NG]) {
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  f32x4 *to = (f32x4 *)tile + (size_t)wv * NG * 4 * kWave + lane;
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      to[(q * 4 + b) * kWave] = f32x4{acc[q][4 * b], acc[q][4 * b + 1], acc[q][4 * b + 2], acc[q][4 * b + 3]};
}
template <int NG>
__device__ __forceinline__ f32x4 summed(const float *tile, int q, int b, int lane) {
  const f32x4 *from = (const f32x4 *)tile + (q * 4 + b) * kWave + lane;
  f32x4 v = from[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += from[(size_t)w * NG * 4 * kWave];
  return v;
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }

// Two floats for a workgroup that may run on another die.
__device__ __forceinline__ void put_shared(uint64_t *to, float lo, float hi) {
  __hip_atomic_store(to, (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

// Launch 1: act[p] = silu(G x) * (U x) of every pair p; NG groups of 16
// gate and 16 up rows per workgroup.  Bound by W1's bytes: 256 MXFP8 experts of
// 7168 x 2048, top 8, read at 6.2 TB/s for one token (39 us) and 6.6 TB/s for
// 128 (1145 us).
template <int Q, int NG, typename IdxT>
__global__ __launch_bounds__(kThreads) void layer_up_kernel(LayerArgs a, uint16_t *__restrict__ act,
                                                            Head *__restrict__ heads, uint16_t *__restrict__ lists,
                                                            uint32_t *__restrict__ done, int blocks) {
  __shared__ Ids s_ids;
  __shared__ uint16_t s_list[kLayerMaxPairs];
  __shared__ __attribute__((aligned(16))) float s_tile[kWaves * NG * 16 * kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.hidden / 32; i += kThreads) done[i] = 0;
  const int blk = blockIdx.x % blocks, rank = blockIdx.x / blocks, P = (int)a.T * a.k;
  int used;
  const int expert = find_expert((const IdxT *)a.idx, P, a.E, rank, s_ids, used);
  if (expert < 0) {                               // uniform
    if (blk == 0 && tid == 0) heads[rank] = Head{-1, 0, used, 0};
    return;
  }
  const int K = a.hidden, ksteps = K / 64, groups = a.inter / 16;
  const int g0 = blk * NG;
  const size_t gidx = (size_t)expert * groups + g0;
  const int s0 = ksteps * wv / kWaves, s1 = ksteps * (wv + 1) / kWaves;
  int n = 0;
  for (int r0 = 0; r0 == 0 || r0 < n; r0 += kTile) {
    int pair = 0;
    v16f acc[NG];
    product<Q, NG>(a.w1 + gidx * fragment_bytes(Q), (size_t)a.E * groups * fragment_bytes(Q), a.w1_scales + gidx * 256,
                   (size_t)a.E * groups * 256, s0, s1,
                   [&] {
                     if (r0 == 0) n = list_pairs(s_ids, P, expert, s_list);
                     pair = s_list[min(r0 + (lane & 31), n - 1)];
                     return (const uint16_t *)a.x + (size_t)(pair / a.k) * K;
                   },
                   acc);
    if (r0 > 0) lds_barrier();
    leave_partials<NG>(s_tile, acc);
    lds_barrier();
    // lane l of quad b holds column l % 32, rows 8b + 4 (l / 32) + 0..3: quads
    // 0 and 1 are gate rows, 2 and 3 the same up rows
    for (int qb = wv; qb < NG * 2; qb += kWaves) {
      const int q = qb >> 1, h = qb & 1;
      if (r0 + (lane & 31) >= n) break;
      const f32x4 gate = summed<NG>(s_tile, q, h, lane), up = summed<NG>(s_tile, q, h + 2, lane);
      const u32x2 v = {pack_bf16x2(silu(gate.x) * up.x, silu(gate.y) * up.y),
                       pack_bf16x2(silu(gate.z) * up.z, silu(gate.w) * up.w)};
      *(u32x2 *)(act + (size_t)pair * a.inter + 16 * (g0 + q) + 8 * h + 4 * (lane >> 5)) = v;
    }
  }
  if (blk == 0) {
    if (tid == 0) heads[rank] = Head{expert, n, used, 0};
    for (int i = tid; i < n; i += kThreads) lists[(size_t)rank * P + i] = s_list[i];
  }
}

// Launch 2: y[p] = D act[p], then, if `join`, out[t] = sum_j w y[t k + j] by the
// last workgroup of each block of 32 NG columns.  W2 is read at 4.5 TB/s for one
// token (27 us), 5.6 TB/s for 128 (677 us; joined 725): a workgroup has 32 steps
// for its four waves.  Joined, without the wait for its rows' arrival and the
// count the launch takes 7 % less, without writing the rows another 12 %.  Several
// column blocks a workgroup, which wait once, were slower (890 us for four):
// the loads of many workgroups hide the wait better.
template <int Q, int NG, typename IdxT>
__global__ __launch_bounds__(kThreads) void layer_down_kernel(LayerArgs a, const uint16_t *__restrict__ act,
                                                              const Head *__restrict__ heads,
                                                              const uint16_t *__restrict__ lists, float *y,
                                                              uint32_t *done, int blocks, int join) {
  __shared__ __attribute__((aligned(16))) float s_tile[kWaves * NG * 16 * kWave];
  constexpr int kRow = 32 * NG + 4;               // floats of a pair's row in LDS
  __shared__ __attribute__((aligned(16))) float s_row[kTile * kRow];
  __shared__ int s_pair[kTile];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int blk = blockIdx.x % blocks, rank = blockIdx.x / blocks, P = (int)a.T * a.k;
  const int expert = heads[rank].expert, n = heads[rank].n, used = heads[rank].used;
  if (expert < 0 && !(join && rank == 0 && used == 0)) return;             // uniform
  const int K = a.inter, ksteps = K / 64, groups = a.hidden / 32;
  const int g0 = blk * NG;
  if (expert >= 0) {
    const size_t gidx = (size_t)expert * groups + g0;
    const int s0 = ksteps * wv / kWaves, s1 = ksteps * (wv + 1) / kWaves;
    for (int r0 = 0; r0 < n; r0 += kTile) {
      int pair = 0;
      v16f acc[NG];
      product<Q, NG>(a.w2 + gidx * fragment_bytes(Q), (size_t)a.E * groups * fragment_bytes(Q),
                     a.w2_scales + gidx * 256, (size_t)a.E * groups * 256, s0, s1,
                     [&] {
                       pair = lists[(size_t)rank * P + min(r0 + (lane & 31), n - 1)];
                       return act + (size_t)pair * K;
                     },
                     acc);
      if (r0 > 0) lds_barrier();
      leave_partials<NG>(s_tile, acc);
      lds_barrier();
      // through LDS, so that a pair's 32 NG columns leave as whole lines: past
      // the L2 every store is a write of its own (128 tokens 739 -> 725 us)
      if (wv == 0 && lane < kTile) s_pair[lane] = pair;
      for (int qb = wv; qb < NG * 4; qb += kWaves) {
        const int q = qb >> 2, h = qb & 3;
        if ((lane & 31) < n - r0)
          *(f32x4 *)(s_row + (lane & 31) * kRow + 32 * q + 8 * h + 4 * (lane >> 5)) = summed<NG>(s_tile, q, h, lane);
      }
      lds_barrier();
      const int rows = min(kTile, n - r0);
      for (int i = tid; i < rows * 16 * NG; i += kThreads) {
        const int row = i / (16 * NG), two = i - row * (16 * NG);
        const float *v = s_row + row * kRow + 2 * two;
        uint64_t *to = (uint64_t *)(y + (size_t)s_pair[row] * a.hidden + 32 * g0) + two;
        if (join) put_shared(to, v[0], v[1]);     // uniform
        else *to = (uint64_t)__float_as_uint(v[1]) << 32 | __float_as_uint(v[0]);
      }
    }
    if (!join) return;                            // uniform
    // y goes past the die's L2 (agent scope), and the wait below holds until
    // it has arrived: the count can then rise without a fence, which would
    // write back the whole L2 (at 128 tokens launch 2 took 12 times as long
    // with one)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(done + blk, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (uint32_t)used - 1;
    __syncthreads();
    if (!s_last) return;
  }
  // out[t] over the block's columns, two per thread; the rows of up to 8
  // pairs are loaded at once
  constexpr int kPairs = 16 * NG;
  const IdxT *idx = (const IdxT *)a.idx;
  for (int job = tid; job < (int)a.T * kPairs; job += kThreads) {
    const int t = job / kPairs, c = 32 * g0 + 2 * (job - t * kPairs);
    float o0 = 0.0f, o1 = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      uint64_t v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = t * a.k + min(j0 + j, a.k - 1);
        const int64_t e = (int64_t)idx[p];
        const bool on = j0 + j < a.k && e >= 0 && e < a.E;
        w[j] = a.weights[p];
        v[j] = 0;
        if (on) v[j] = __hip_atomic_load((uint64_t *)(y + (size_t)p * a.hidden + c), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
        if (!on) w[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o0 += w[j] * __uint_as_float((uint32_t)v[j]);
        o1 += w[j] * __uint_as_float((uint32_t)(v[j] >> 32));
      }
    }
    *(uint32_t *)((uint16_t *)a.out + (size_t)t * a.hidden + c) = pack_bf16x2(o0, o1);
  }
}

// Calls of more tokens sum the pairs' rows in a launch of their own: the last
// workgroups of launch 2 are one per block of columns, too few to read many
// rows.  Measured (us a call, summed in launch 2 against by a third): one token
// of 256 MXFP8 experts (7168 x 2048, top 8) 72.8, 74; 3 tokens of 32 (2048 x
// 768, top 4) 23.6, 24.5; 8 tokens 34.0, 34.3; 13 tokens of 64 bf16 experts
// (4096 x 1536, top 8) 349, 342; 128 of 64 (2048 x 768, top 8) 173, 132; 128 of
// 256 MXFP8 1810, 1800.
constexpr int64_t kJoinTokens = 8;

// out[t] = sum_j w y[t k + j] in ascending j, four columns a thread.
template <typename IdxT>
__global__ __launch_bounds__(256) void layer_sum_kernel(LayerArgs a, const float *__restrict__ y) {
  const int quads = a.hidden / 4, job = blockIdx.x * 256 + threadIdx.x, t = job / quads, c = 4 * (job - t * quads);
  if (t >= a.T) return;
  const IdxT *idx = (const IdxT *)a.idx + (int64_t)t * a.k;
  const float *weights = a.weights + (int64_t)t * a.k;
  f32x4 o = {};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    f32x4 v[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = min(j0 + j, a.k - 1);
      const int64_t e = (int64_t)idx[p];
      const bool on = j0 + j < a.k && e >= 0 && e < a.E;
      w[j] = weights[p];
      v[j] = f32x4{};
      if (on) v[j] = *(const f32x4 *)(y + ((size_t)t * a.k + p) * a.hidden + c);
      if (!on) w[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o += w[j] * v[j];
  }
  *(u32x2 *)((uint16_t *)a.out + (size_t)t * a.hidden + c) = u32x2{pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w)};
}

template <int Q, int NG, typename IdxT>
hipError_t layer_launch(const LayerArgs &a, hipStream_t s) {
  const LayerWs ws = layer_ws(a.T, a.k, a.E, a.hidden, a.inter);
  uint16_t *act = (uint16_t *)(a.ws + ws.act);
  float *y = (float *)(a.ws + ws.y);
  uint32_t *done = (uint32_t *)(a.ws + ws.done);
  Head *heads = (Head *)(a.ws + ws.heads);
  uint16_t *lists = (uint16_t *)(a.ws + ws.lists);
  const int64_t P = a.T * a.k, used = P < a.E ? P : a.E;
  const int up_blocks = a.inter / 16 / NG, down_blocks = a.hidden / 32 / NG;
  const int join = a.T <= kJoinTokens;
  hipLaunchKernelGGL((layer_up_kernel<Q, NG, IdxT>), dim3((unsigned)(used * up_blocks)), dim3(kThreads), 0, s, a, act,
                     heads, lists, done, up_blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((layer_down_kernel<Q, NG, IdxT>), dim3((unsigned)(used * down_blocks)), dim3(kThreads), 0, s, a,
                     act, heads, lists, y, done, down_blocks, join);
  e = hipGetLastError();
  if (e != hipSuccess || join) return e;
  hipLaunchKernelGGL((layer_sum_kernel<IdxT>), dim3((unsigned)((a.T * (a.hidden / 4) + 255) / 256)), dim3(256), 0, s, a, y);
  return hipGetLastError();
}
template <int Q>
hipError_t layer_q(const LayerArgs &a, hipStream_t s) {
  return a.idx64 ? layer_launch<Q, kGroups, int64_t>(a, s) : layer_launch<Q, kGroups, int32_t>(a, s);
}

}  // namespace

hipError_t launch_moe_layer(const LayerArgs &a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  switch (a.quant) {
    case EP_QUANT_NONE: return layer_q<EP_QUANT_NONE>(a, s);
    case EP_QUANT_MXFP8: return layer_q<EP_QUANT_MXFP8>(a, s);
    default: return layer_q<EP_QUANT_MXFP4>(a, s);
  }
}

hipError_t launch_pack_ex(const void *w, const void *scales, int quant, int E, int N, int K, int gate_up, void *pw,
                          void *pscales, hipStream_t s) {
  const uint8_t *from = (const uint8_t *)w, *sc = (const uint8_t *)scales;
  uint8_t *to = (uint8_t *)pw, *tos = (uint8_t *)pscales;
  const dim3 grid(2048), block(256);
  switch (quant) {
    case EP_QUANT_NONE:
      hipLaunchKernelGGL(pack_kernel<EP_QUANT_NONE>, grid, block, 0, s, from, sc, E, N, K, gate_up, to, tos);
      break;
    case EP_QUANT_MXFP8:
      hipLaunchKernelGGL(pack_kernel<EP_QUANT_MXFP8>, grid, block, 0, s, from, sc, E, N, K, gate_up, to, tos);
      break;
    default:
      hipLaunchKernelGGL(pack_kernel<EP_QUANT_MXFP4>, grid, block, 0, s, from, sc, E, N, K, gate_up, to, tos);
  }
  return hipGetLastError();
}

}  // namespace ep
