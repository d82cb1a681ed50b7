// Router of a MoE layer for gfx950: scores, (grouped) top-k selection and
// weights from the gate's logits, and the gradient of the weights with
// respect to the logits.
//
// What is computed, for one row z of E logits:
//   s_e   = softmax(z)_e or sigmoid(z_e)
//   key_e = s_e + bias_e   (without a bias the keys are the logits: both
//           scores rise with them)
//   groups: E / G consecutive experts each; a group's rank is the sum of its
//           `top` (1 or 2) largest keys; the `keep` best groups stay
//   ids   = the k largest keys of the kept groups, ties to the lower index
//   w_j   = scale * s_j, or scale * s_j / sum of the chosen s
// An expert whose logit or key is -inf or NaN is never chosen.
//
// Two keys s_e + bias_e may lie closer than float32 rounding, and then the
// order would depend on how exp was evaluated; keys with a bias and sums of
// two scores are therefore float64, to 43 significant bits.
//
// 16 lanes take a token (four tokens a wave), each a run of ceil(E / 16)
// experts.  A key and its expert are one double (the expert in the low
// mantissa bits, so that all are different and ties go to the lower id),
// which v_max_f64 / v_min_f64 compare at full rate: every lane sorts its run
// in registers, then four exchange steps inside the 16 lanes merge the
// lanes' best lists.  No LDS, no loop over the k choices.
//
// Bound by its instructions, not by the logits' bytes: 16384 tokens of 256
// experts with a bias and groups 15 us, of which the vector units are busy for
// 10 (the bytes alone: 4); 128 tokens without 4.0 us, one token with both 6.2.
#include <math.h>

#include "common.hpp"
#include "formats.hpp"
#include "ring.hpp"
#include "router.hpp"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kRow = 16;                          // lanes of a token
constexpr int kTokens = kThreads / kRow;          // tokens per workgroup
constexpr float kLargest = 3.402823466e38f;

template <int DT>
__device__ __forceinline__ float logit(const void *p, int64_t i) {
  if constexpr (DT == EP_FLOAT_F32) return ((const float *)p)[i];
  if constexpr (DT == EP_FLOAT_BF16) return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
  return (float)((const _Float16 *)p)[i];
}
template <int DT>
__device__ __forceinline__ void put(void *p, int64_t i, float v) {
  if constexpr (DT == EP_FLOAT_F32) ((float *)p)[i] = v;
  else if constexpr (DT == EP_FLOAT_BF16) ((__bf16 *)p)[i] = (__bf16)v;
  else ((_Float16 *)p)[i] = (_Float16)v;
}
// NaN and -inf: no expert (-inf); +inf: the largest finite logit
__device__ __forceinline__ float usable(float z) { return fminf(fmaxf(z, -INFINITY), kLargest); }

// This lane's run of `run` logits, [first, first + run) of a row of E (which
// starts at element `row`); -inf past them.  16-byte loads where every run
// starts on 16 bytes.
template <int DT, int I>
__device__ __forceinline__ void load_run(const void *p, int64_t row, int E, int first, int run, bool live, bool wide,
                                         float (&z)[I]) {
  constexpr int kVec = DT == EP_FLOAT_F32 ? 4 : 8;
  if constexpr (I >= kVec) {
    if (wide) {                                   // uniform; run is a multiple of kVec
#pragma unroll
      for (int v = 0; v < I / kVec; ++v) {
        u32x4 w = {};
        const bool on = live && v * kVec < run && first + v * kVec < E;
        if (on) w = *(const u32x4 *)((const char *)p + (row + first + v * kVec) * (16 / kVec));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float f;
          if constexpr (DT == EP_FLOAT_F32) f = __uint_as_float(w[i]);
          else if constexpr (DT == EP_FLOAT_BF16) f = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
          else f = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
          z[v * kVec + i] = on ? usable(f) : -INFINITY;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < I; ++i)
    z[i] = live && i < run && first + i < E ? usable(logit<DT>(p, row + first + i)) : -INFINITY;
}

// ------------------------------------------------ exchanges in 16 lanes
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;   // quad swaps, rotations by 4 and 8
constexpr int kHalf = 0x141;                      // mirror of 8 lanes: the other quad of the half
constexpr int kBcast = 0x150;                                             // + lane of the row

// max / min of doubles that are never NaN (the operator forms compile to a
// compare and two selects, fmax to extra canonicalisations)
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return max64(a, b); }

template <typename T>
__device__ __forceinline__ T row_max(T v) {
  v = max_of(v, dpp<kXor1>(v));
  v = max_of(v, dpp<kXor2>(v));
  v = max_of(v, dpp<kRor4>(v));
  return max_of(v, dpp<kRor8>(v));
}
template <typename T>
__device__ __forceinline__ T row_sum(T v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kRor4>(v);
  return v + dpp<kRor8>(v);
}

// -------------------------------------------------------- packed keys
// A key (its first 44 significant bits) with its expert in the 9 low
// mantissa bits: among equal keys the lower expert is the larger double.  An
// expert that is not there has the key kNoKey (a finite one, so that the low
// bits make no NaN of it).
constexpr double kNoKey = -1e300;
__device__ __forceinline__ double pack_key(double key, int e) {
  const uint64_t u = __builtin_bit_cast(uint64_t, key);
  const uint32_t hi = (uint32_t)(u >> 32), sign = (uint32_t)((int32_t)hi >> 31);
  const uint32_t low = ((uint32_t)(kMaxExperts - 1 - e) ^ sign) & (kMaxExperts - 1);
  const uint32_t lo = ((uint32_t)u & ~(uint32_t)(kMaxExperts - 1)) | low;
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int expert_in(double packed) {
  const uint64_t u = __builtin_bit_cast(uint64_t, packed);
  const uint32_t sign = (uint32_t)((int32_t)(u >> 32) >> 31);
  return kMaxExperts - 1 - (int)(((uint32_t)u ^ sign) & (kMaxExperts - 1));
}
__device__ __forceinline__ bool is_key(double packed) { return packed > kNoKey * 0.5; }
__device__ __forceinline__ double key_in(double packed) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, packed) & ~(uint64_t)(kMaxExperts - 1));
}
static_assert((kMaxExperts & (kMaxExperts - 1)) == 0, "the expert is a bit field");

// e^x for x <= 700 or so: 2^n times the Taylor series of e^r, |r| <= ln 2 / 2,
// whose 12th term is below 2^-46.6; 0 below e^-745.  Off by at most 2^-46 for
// |x| <= 150, and, as n times the rounding of ln 2 grows, by 2^-44.8 for |x| <=
// 700 (against 60-digit values).  A score below e^-134 is lost beside any bias
// but 0, so keys hold their 43 bits by the first bound; sums of two scores
// without a bias are told apart from a difference of 2^-43.8 on by the second.
// The coefficients are held in scalar registers (as literals each costs two
// moves a use, a quarter of the kernel's instructions).
__device__ __forceinline__ double scalar(double c) {
  asm("" : "+s"(c));
  return c;
}
__device__ __forceinline__ double exp64(double x) {
  const double n = rint(x * scalar(1.4426950408889634));
  const double r = fma(n, scalar(-0.6931471805599453), x);
  double p = 1.0 / 39916800;
  p = fma(p, r, scalar(1.0 / 3628800));
  p = fma(p, r, scalar(1.0 / 362880));
  p = fma(p, r, scalar(1.0 / 40320));
  p = fma(p, r, scalar(1.0 / 5040));
  p = fma(p, r, scalar(1.0 / 720));
  p = fma(p, r, scalar(1.0 / 120));
  p = fma(p, r, scalar(1.0 / 24));
  p = fma(p, r, scalar(1.0 / 6));
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / x of a normal x: the hardware's approximation and two Newton steps
__device__ __forceinline__ double rcp64(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(y, fma(-x, y, 1.0), y);
  return fma(y, fma(-x, y, 1.0), y);
}
// sigmoid; e^-z is kept in double's range (beyond it the score is 0 to 2^-999)
__device__ __forceinline__ double sigmoid64(float z) { return rcp64(1.0 + exp64(fmin(-(double)z, 690.0))); }

// Batcher's odd-even merge sort, descending; n a power of two.
template <int N>
__device__ __forceinline__ void sort_run(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + q];
            v[i + j] = max64(a, b);
            v[i + j + q] = min64(a, b);
          }
}
// The L largest of two descending lists, v and the one whose reverse is o: the
// element-wise maximum holds them as a bitonic sequence, which log L exchange
// steps sort.
template <int L>
__device__ __forceinline__ void merge_lists(double (&v)[L], const double (&o)[L]) {
#pragma unroll
  for (int i = 0; i < L; ++i) v[i] = max64(v[i], o[i]);
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < L; ++i)
      if ((i & d) == 0) {
        const double a = v[i], b = v[i + d];
        v[i] = max64(a, b);
        v[i + d] = min64(a, b);
      }
}
// with the list of the lane CTRL names / of lane ^ d
template <int CTRL, int L>
__device__ __forceinline__ void merge_step(double (&v)[L]) {
  double o[L];
#pragma unroll
  for (int i = 0; i < L; ++i) o[i] = dpp<CTRL>(v[L - 1 - i]);
  merge_lists(v, o);
}
template <int L>
__device__ __forceinline__ void merge_rows(double (&v)[L], int d) {
  double o[L];
#pragma unroll
  for (int i = 0; i < L; ++i) o[i] = __shfl_xor(v[L - 1 - i], d);
  merge_lists(v, o);
}

// log of the score, up to a constant of the row: z for a softmax,
// log sigmoid(z) = min(z, 0) - log(1 + e^-|z|)
__device__ __forceinline__ float log_score(int score, float z) {
  return score == EP_SCORE_SOFTMAX ? z : fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
}
__device__ __forceinline__ float sigmoidf(float z) { return 1.0f / (1.0f + expf(-z)); }

// ------------------------------------------------------------ wave path
// One token per wave with its keys in LDS: group shapes that do not fall on
// whole lanes, whose ranks are found by all lanes from the keys there.  The
// selection then is the row path's over 64 lanes (two more merges).  800
// tokens of 238 experts in 2 groups 9.6 us a call; ranking every key against
// its group and k reductions over the wave instead took 27.
struct WaveLds {
  double key[kMaxExperts], rank[kMaxGroups];
};

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) { const T o = __shfl_xor(v, d); v = o > v ? o : v; }
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The ids of token t: lane j gets the j-th (-1: none).
template <int DT>
__device__ __forceinline__ int wave_route(const RouterArgs &a, int64_t t, WaveLds &s) {
  const int lane = threadIdx.x & (kWave - 1), E = a.E;
  const double kNone = -INFINITY;
  const bool softmax = a.score == EP_SCORE_SOFTMAX;
  float top = -INFINITY;
  double sum = 1.0;
  if (softmax) {
    for (int e = lane; e < E; e += kWave) top = fmaxf(top, usable(logit<DT>(a.logits, t * E + e)));
    top = wave_max(top);
    sum = 0.0;
    for (int e = lane; e < E; e += kWave) {
      const float z = usable(logit<DT>(a.logits, t * E + e));
      sum += z > -INFINITY ? exp64(fmax((double)z - (double)top, -700.0)) : 0.0;
    }
    sum = rcp64(wave_sum(sum));
  }
  const bool by_sum = a.groups > 1 && a.top == 2;
  // the keys; without a bias the group sums need the scores first
  for (int pass = by_sum && !a.bias ? 0 : 1; pass < 2; ++pass) {
    for (int e = lane; e < E; e += kWave) {
      const float z = usable(logit<DT>(a.logits, t * E + e));
      double c = kNone;
      if (z > -INFINITY) {
        if (pass == 1 && !a.bias) {
          c = (double)z;
        } else {
          c = softmax ? exp64(fmax((double)z - (double)top, -700.0)) * sum : sigmoid64(z);
          if (a.bias) c += (double)a.bias[e];
        }
        if (!(c > kNone)) c = kNone;              // a NaN bias
      }
      s.key[e] = c;
    }
    if (a.groups > 1 && (pass == 0 || a.bias || !by_sum)) {
      const int size = E / a.groups;
      wave_lds_fence();
      // `span` lanes look through a group, their best two are joined
      int span = kWave;
      while (span * a.groups > kWave) span >>= 1;
      const int group = lane / span;
      double b0 = kNone, b1 = kNone;
      if (group < a.groups) {
#pragma unroll 4
        for (int j = lane % span; j < size; j += span) {
          const double v = s.key[group * size + j];
          if (v > b0) { b1 = b0; b0 = v; } else if (v > b1) b1 = v;
        }
      }
      for (int d = 1; d < span; d <<= 1) {
        const double o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
        const double lo = o0 < b0 ? o0 : b0, hi = o0 < b0 ? b0 : o0, second = o1 > b1 ? o1 : b1;
        b0 = hi;
        b1 = lo > second ? lo : second;
      }
      // no second key: last, even beside +inf
      if (group < a.groups && lane % span == 0)
        s.rank[group] = a.top == 1 ? b0 : b1 > kNone ? b0 + b1 : kNone;
      wave_lds_fence();
    }
  }
  if (a.groups > 1) {
    // a group stays when fewer than `keep` groups come before it
    const int size = E / a.groups;
    bool stays = false;
    if (lane < a.groups) {
      const double mine = s.rank[lane];
      int before = 0;
      for (int g = 0; g < a.groups; ++g) before += s.rank[g] > mine || (s.rank[g] == mine && g < lane);
      stays = before < a.keep;
    }
    const uint64_t kept = __ballot(stays);
    for (int e = lane; e < E; e += kWave)
      if (!((kept >> (e / size)) & 1)) s.key[e] = kNone;
  }
  // the selection as on the row path, over the whole wave
  double v[kMaxExperts / kWave], best[kMaxTopk];
#pragma unroll
  for (int i = 0; i < kMaxExperts / kWave; ++i) {
    const int e = lane + i * kWave;
    const double key = e < E ? s.key[e] : kNone;
    v[i] = pack_key(key > kNone ? fmin(key, 1e300) + 0.0 : kNoKey, e);
  }
  sort_run(v);
#pragma unroll
  for (int i = 0; i < kMaxTopk; ++i) best[i] = i < kMaxExperts / kWave ? v[i < kMaxExperts / kWave ? i : 0] : kNoKey;
  merge_step<kXor1>(best);
  merge_step<kXor2>(best);
  merge_step<kRor4>(best);
  merge_step<kRor8>(best);
  merge_rows(best, 16);
  merge_rows(best, 32);
  double mine = best[0];
#pragma unroll
  for (int i = 1; i < kMaxTopk; ++i) mine = lane == i ? best[i] : mine;
  return lane < a.k && is_key(mine) ? expert_in(mine) : -1;
}

// The weight of choice `lane` (of 16 lanes, id -1: none) and its store;
// top and sum: the row's largest logit and sum of exp(z - top).
template <int DT>
__device__ __forceinline__ void store_choice(const RouterArgs &a, int64_t t, int j, bool live, int id, float top,
                                             float sum, void *idx, int idx64, float *weights) {
  const bool softmax = a.score == EP_SCORE_SOFTMAX;
  const bool on = live && id >= 0;
  const float z = on ? fminf(logit<DT>(a.logits, t * a.E + id), kLargest) : -INFINITY;
  float w;
  if (a.renorm) {
    // s_j / sum s = softmax of the logs: no score underflows
    const float ls = on ? log_score(a.score, z) : -INFINITY;
    const float m = row_max(ls);
    const float p = on ? expf(ls - m) : 0.0f;
    const float total = row_sum(p);
    w = on ? p / total : 0.0f;
  } else {
    w = !on ? 0.0f : softmax ? expf(z - top) / sum : sigmoidf(z);
  }
  if (live && j < a.k) {
    if (idx64) ((int64_t *)idx)[t * a.k + j] = id;
    else ((int32_t *)idx)[t * a.k + j] = id;
    weights[t * a.k + j] = w * a.scale;
  }
}

// Row maximum and sum of exp(z - max), float32, over a wave's token.
template <int DT>
__device__ __forceinline__ void wave_softmax(const RouterArgs &a, int64_t t, float &top, float &sum) {
  const int lane = threadIdx.x & (kWave - 1);
  top = -INFINITY;
  for (int e = lane; e < a.E; e += kWave) top = fmaxf(top, usable(logit<DT>(a.logits, t * a.E + e)));
  top = wave_max(top);
  sum = 0.0f;
  for (int e = lane; e < a.E; e += kWave) {
    const float z = usable(logit<DT>(a.logits, t * a.E + e));
    sum += z > -INFINITY ? expf(z - top) : 0.0f;
  }
  sum = wave_sum(sum);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void wave_router_kernel(RouterArgs a, void *idx, int idx64, float *weights) {
  __shared__ WaveLds s_wave[kWaves];
  const int wv = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int64_t t = (int64_t)blockIdx.x * kWaves + wv;
  if (t >= a.T) return;                           // a whole wave; no barriers below
  const int id = wave_route<DT>(a, t, s_wave[wv]);
  float top = 0.0f, sum = 1.0f;
  if (!a.renorm && a.score == EP_SCORE_SOFTMAX) wave_softmax<DT>(a, t, top, sum);
  if (lane < kRow) store_choice<DT>(a, t, lane, true, id, top, sum, idx, idx64, weights);
}

// ------------------------------------------------------------- row path
// I: experts of a lane (its run padded to a power of two), L: length of the
// merged lists (k rounded up to 8 or 16).
template <int DT, int I, int L>
__global__ __launch_bounds__(kThreads) void row_router_kernel(RouterArgs a, void *idx, int idx64, float *weights,
                                                              int run, int wide) {
  const int j = threadIdx.x & (kRow - 1);
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kRow;
  const bool live = t < a.T;
  const bool softmax = a.score == EP_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const int first = j * run;
  float z[I];
  load_run<DT, I>(a.logits, t * a.E, a.E, first, run, live, wide & 1, z);

  float top = -INFINITY, sum = 1.0f;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < I; ++i) top = fmaxf(top, z[i]);
    top = row_max(top);
    if (!a.renorm) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < I; ++i) sum += z[i] > -INFINITY ? expf(z[i] - top) : 0.0f;
      sum = row_sum(sum);
    }
  }
  double v[I];
  if (biased) {
    float bias[I];
    if (wide & 2) {                               // uniform
#pragma unroll
      for (int i = 0; i < I; i += 4) {
        const u32x4 w = *(const u32x4 *)(a.bias + min(first + i, a.E - 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) bias[i + q] = __uint_as_float(w[q]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < I; ++i) bias[i] = a.bias[min(first + i, a.E - 1)];
    }
    double by = 1.0;
    if (softmax) {
      double sum64 = 0.0;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        v[i] = z[i] > -INFINITY ? exp64(fmax((double)z[i] - (double)top, -700.0)) : 0.0;
        sum64 += v[i];
      }
      by = rcp64(row_sum(sum64));
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const double c = (softmax ? v[i] * by : sigmoid64(z[i])) + (double)bias[i];
      // NaN fails the comparison; +inf is held below infinity, so that it stays a number
      v[i] = pack_key(z[i] > -INFINITY && c > -1e299 ? fmin(c, 1e300) : kNoKey, first + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < I; ++i) v[i] = pack_key(z[i] > -INFINITY ? (double)z[i] + 0.0 : kNoKey, first + i);
  }
  sort_run(v);

  bool stays = true;
  if (a.groups > 1) {
    // a group is kRow / groups whole lanes: its two best keys from theirs
    const int lanes = kRow / a.groups;
    double b0 = v[0], b1 = v[1];
    auto join = [&](double o0, double o1) {
      const double lo = min64(b0, o0);
      b0 = max64(b0, o0);
      b1 = max64(lo, max64(b1, o1));
    };
    if (lanes > 1) join(dpp<kXor1>(b0), dpp<kXor1>(b1));
    if (lanes > 2) join(dpp<kXor2>(b0), dpp<kXor2>(b1));
    if (lanes > 4) join(dpp<kHalf>(b0), dpp<kHalf>(b1));
    double rank = key_in(b0);
    if (a.top == 2) {
      if (biased) {
        // beside +inf (held at 1e300) the second key changes nothing: groups
        // with one and with two such keys rank alike
        rank = !is_key(b1) ? kNoKey : rank > 1e299 ? rank : rank + key_in(b1);
      } else {
        // sums of two scores (a softmax's up to the row's factor)
        const float k0 = (float)key_in(b0), k1 = (float)key_in(b1);
        const double s = softmax ? exp64(fmax((double)k0 - (double)top, -700.0)) +
                                       exp64(fmax((double)k1 - (double)top, -700.0))
                                 : sigmoid64(k0) + sigmoid64(k1);
        rank = is_key(b1) ? s : kNoKey;
      }
    }
    // a group stays when fewer than `keep` groups come before it
    const int mine = j / lanes;
    int before = 0;
#define EP_ROT(R)                                                    \
  if ((R) % lanes == 0) {                                            \
    const double o = dpp<0x120 + (R)>(rank);                         \
    before += o > rank || (o == rank && ((j - (R)) & (kRow - 1)) / lanes < mine); \
  }
    EP_ROT(1) EP_ROT(2) EP_ROT(3) EP_ROT(4) EP_ROT(5) EP_ROT(6) EP_ROT(7) EP_ROT(8)
    EP_ROT(9) EP_ROT(10) EP_ROT(11) EP_ROT(12) EP_ROT(13) EP_ROT(14) EP_ROT(15)
#undef EP_ROT
    stays = before < a.keep;
  }

  double best[L];
#pragma unroll
  for (int i = 0; i < L; ++i) best[i] = i < I && stays ? v[i < I ? i : 0] : kNoKey;
  merge_step<kXor1>(best);
  merge_step<kXor2>(best);
  merge_step<kRor4>(best);
  merge_step<kRor8>(best);
  double mine = best[0];
#pragma unroll
  for (int i = 1; i < L; ++i) mine = j == i ? best[i] : mine;
  const int id = j < a.k && is_key(mine) ? expert_in(mine) : -1;
  store_choice<DT>(a, t, j, live, id, top, sum, idx, idx64, weights);
}

// Gradient of the weights with respect to the logits.  With p_j the
// normalised weights (w_j / scale), q_j = scale * grad_j:
//   renormalised: d log-score_j = p_j (q_j - sum_i p_i q_i)
//   otherwise:    d log-score_j = s_j q_j
//   softmax: dz_e = [e chosen] d_j - s_e sum_j d_j (the sum is 0 when
//   renormalised); sigmoid: dz_j = d_j (1 - s_j)
// 16 lanes a token: lane j has choice j and the j-th run of experts.  Reads
// and writes the logits' bytes once where the softmax is not renormalised,
// else gathers the k chosen logits; 8191 tokens of 60 experts 4.0 us.
template <int DT, int I>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterArgs a, const void *idx, int idx64,
                                                                   const float *__restrict__ grad, void *dz, int run,
                                                                   int wide) {
  const int j = threadIdx.x & (kRow - 1);
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kRow;
  const bool live = t < a.T;
  const int E = a.E, k = a.k, first = j * run;
  const bool softmax = a.score == EP_SCORE_SOFTMAX, dense = softmax && !a.renorm;
  int id = -1;
  float zj = -INFINITY, q = 0.0f;
  if (live && j < k) {
    const int64_t e = idx64 ? ((const int64_t *)idx)[t * k + j] : (int64_t)((const int32_t *)idx)[t * k + j];
    if (e >= 0 && e < E) {
      zj = usable(logit<DT>(a.logits, t * E + e));
      if (zj > -INFINITY) { id = (int)e; q = grad[t * k + j] * a.scale; }
    }
  }
  float v[I];
  float top = 0.0f, inv = 0.0f;
  if (dense) {                                    // v: the scores
    load_run<DT, I>(a.logits, t * E, E, first, run, live, wide, v);
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < I; ++i) top = fmaxf(top, v[i]);
    top = row_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      v[i] = v[i] > -INFINITY ? expf(v[i] - top) : 0.0f;
      sum += v[i];
    }
    sum = row_sum(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  float d = 0.0f;
  if (a.renorm) {
    const float ls = id >= 0 ? log_score(a.score, zj) : -INFINITY;
    const float m = row_max(ls);
    float p = id >= 0 ? expf(ls - m) : 0.0f;
    const float total = row_sum(p);
    p = id >= 0 ? p / total : 0.0f;
    const float mean = row_sum(p * q);
    d = p * (q - mean);
  } else if (id >= 0) {
    d = q * (softmax ? expf(zj - top) * inv : sigmoidf(zj));
  }
  if (!softmax && id >= 0) d *= sigmoidf(-zj);
  const float pull = dense ? row_sum(d) * inv : 0.0f;
#pragma unroll
  for (int i = 0; i < I; ++i) v[i] = dense ? -v[i] * pull : 0.0f;
  // the choices in ascending j
#define EP_CHOICE(J)                                   \
  if ((J) < k) {                                       \
    const int e = dpp<kBcast + (J)>(id) - first;       \
    const float dj = dpp<kBcast + (J)>(d);             \
    _Pragma("unroll") for (int i = 0; i < I; ++i) v[i] += e == i ? dj : 0.0f; \
  }
  EP_CHOICE(0) EP_CHOICE(1) EP_CHOICE(2) EP_CHOICE(3) EP_CHOICE(4) EP_CHOICE(5) EP_CHOICE(6) EP_CHOICE(7)
  EP_CHOICE(8) EP_CHOICE(9) EP_CHOICE(10) EP_CHOICE(11) EP_CHOICE(12) EP_CHOICE(13) EP_CHOICE(14) EP_CHOICE(15)
#undef EP_CHOICE
  if (!live) return;
  constexpr int kVec = DT == EP_FLOAT_F32 ? 4 : 8;
  if constexpr (I >= kVec) {
    if (wide) {
#pragma unroll
      for (int q0 = 0; q0 < I / kVec; ++q0) {
        if (q0 * kVec >= run || first + q0 * kVec >= E) break;
        u32x4 w;
        if constexpr (DT == EP_FLOAT_F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[q0 * 4 + i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = v[q0 * kVec + (2 * i) % kVec], hi = v[q0 * kVec + (2 * i + 1) % kVec];
            if constexpr (DT == EP_FLOAT_BF16) {
              w[i] = pack_bf16x2(lo, hi);
            } else {
              w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
                     (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
            }
          }
        }
        *(u32x4 *)((char *)dz + (t * E + first + q0 * kVec) * (16 / kVec)) = w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < I; ++i)
    if (i < run && first + i < E) put<DT>(dz, t * E + first + i, v[i]);
}

// A lane's run of experts, and whether every run of every row starts on 16 bytes.
int run_of(int E) { return (E + kRow - 1) / kRow; }
bool wide_rows(const void *p, int dtype, int E, int run) {
  const int vec = dtype == EP_FLOAT_F32 ? 4 : 8;
  return (uintptr_t)p % 16 == 0 && E % vec == 0 && run % vec == 0;
}

template <int DT, int I>
hipError_t router_i(const RouterArgs &a, void *idx, int idx64, float *weights, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kThreads);
  const int run = run_of(a.E);
  const int wide = (wide_rows(a.logits, DT, a.E, run) ? 1 : 0) |
                   ((uintptr_t)a.bias % 16 == 0 && a.E % 4 == 0 && run % 4 == 0 ? 2 : 0);
  if (a.k <= 8)
    hipLaunchKernelGGL((row_router_kernel<DT, I, 8>), grid, block, 0, s, a, idx, idx64, weights, run, wide);
  else
    hipLaunchKernelGGL((row_router_kernel<DT, I, 16>), grid, block, 0, s, a, idx, idx64, weights, run, wide);
  return hipGetLastError();
}
template <int DT>
hipError_t router_dt(const RouterArgs &a, void *idx, int idx64, float *weights, hipStream_t s) {
  // groups of whole lanes: E / 16 experts a lane, 16 / groups lanes a group
  if (a.groups > 1 && (a.E % kRow != 0 || kRow % a.groups != 0)) {
    const dim3 grid((unsigned)((a.T + kWaves - 1) / kWaves)), block(kThreads);
    hipLaunchKernelGGL(wave_router_kernel<DT>, grid, block, 0, s, a, idx, idx64, weights);
    return hipGetLastError();
  }
  const int run = run_of(a.E);
  if (run <= 4) return router_i<DT, 4>(a, idx, idx64, weights, s);
  if (run <= 8) return router_i<DT, 8>(a, idx, idx64, weights, s);
  if (run <= 16) return router_i<DT, 16>(a, idx, idx64, weights, s);
  return router_i<DT, 32>(a, idx, idx64, weights, s);
}
template <int DT, int I>
hipError_t backward_i(const RouterArgs &a, const void *idx, int idx64, const float *grad, void *dz, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kThreads);
  const int run = run_of(a.E);
  const int wide = wide_rows(a.logits, DT, a.E, run) && wide_rows(dz, DT, a.E, run);
  hipLaunchKernelGGL((router_backward_kernel<DT, I>), grid, block, 0, s, a, idx, idx64, grad, dz, run, wide);
  return hipGetLastError();
}
template <int DT>
hipError_t backward_dt(const RouterArgs &a, const void *idx, int idx64, const float *grad, void *dz, hipStream_t s) {
  const int run = run_of(a.E);
  if (run <= 4) return backward_i<DT, 4>(a, idx, idx64, grad, dz, s);
  if (run <= 8) return backward_i<DT, 8>(a, idx, idx64, grad, dz, s);
  if (run <= 16) return backward_i<DT, 16>(a, idx, idx64, grad, dz, s);
  return backward_i<DT, 32>(a, idx, idx64, grad, dz, s);
}

// A launch holds fewer than 2^32 threads (the runtime cuts larger counts to 32
// bits); the wave path takes 64 a token.  More tokens go in several.
constexpr int64_t kLaunchTokens = 1 << 25;
const char *element(const void *p, int64_t i, int bytes) { return (const char *)p + i * bytes; }
int logit_bytes(int dtype) { return dtype == EP_FLOAT_F32 ? 4 : 2; }

}  // namespace

hipError_t launch_router(const RouterArgs &all, void *idx, int idx64, float *weights, hipStream_t s) {
  hipError_t e = hipSuccess;
  for (int64_t t = 0; t < all.T && e == hipSuccess; t += kLaunchTokens) {
    RouterArgs a = all;
    a.T = all.T - t < kLaunchTokens ? all.T - t : kLaunchTokens;
    a.logits = element(all.logits, t * a.E, logit_bytes(a.dtype));
    void *to = (void *)element(idx, t * a.k, idx64 ? 8 : 4);
    switch (a.dtype) {
      case EP_FLOAT_F32: e = router_dt<EP_FLOAT_F32>(a, to, idx64, weights + t * a.k, s); break;
      case EP_FLOAT_BF16: e = router_dt<EP_FLOAT_BF16>(a, to, idx64, weights + t * a.k, s); break;
      default: e = router_dt<EP_FLOAT_F16>(a, to, idx64, weights + t * a.k, s);
    }
  }
  return e;
}

hipError_t launch_router_backward(const RouterArgs &all, const void *idx, int idx64, const float *grad_weights,
                                  void *grad_logits, hipStream_t s) {
  hipError_t e = hipSuccess;
  for (int64_t t = 0; t < all.T && e == hipSuccess; t += kLaunchTokens) {
    RouterArgs a = all;
    a.T = all.T - t < kLaunchTokens ? all.T - t : kLaunchTokens;
    a.logits = element(all.logits, t * a.E, logit_bytes(a.dtype));
    const void *from = element(idx, t * a.k, idx64 ? 8 : 4);
    void *to = (void *)element(grad_logits, t * a.E, logit_bytes(a.dtype));
    const float *grad = grad_weights + t * a.k;
    switch (a.dtype) {
      case EP_FLOAT_F32: e = backward_dt<EP_FLOAT_F32>(a, from, idx64, grad, to, s); break;
      case EP_FLOAT_BF16: e = backward_dt<EP_FLOAT_BF16>(a, from, idx64, grad, to, s); break;
      default: e = backward_dt<EP_FLOAT_F16>(a, from, idx64, grad, to, s);
    }
  }
  return e;
}

}  // namespace ep
