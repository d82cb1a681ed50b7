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
// two scores are therefore held in float64.
#include <math.h>

#include "common.hpp"
#include "formats.hpp"
#include "router.hpp"

namespace ep {

namespace {

constexpr int kTokens = 4;                        // tokens (waves) per workgroup
constexpr int kItems = kMaxExperts / kWave;       // experts per lane: lane, lane + 64, ...

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

// log of the score, up to a constant of the row: z for a softmax,
// log sigmoid(z) = min(z, 0) - log(1 + e^-|z|)
__device__ __forceinline__ float log_score(int score, float z) {
  return score == EP_SCORE_SOFTMAX ? z : fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
}
__device__ __forceinline__ float sigmoidf(float z) { return 1.0f / (1.0f + expf(-z)); }

template <int DT, typename IdxT>
__global__ __launch_bounds__(kTokens *kWave) void router_kernel(RouterArgs a, IdxT *__restrict__ idx,
                                                                float *__restrict__ weights) {
  __shared__ double s_key[kTokens][kMaxExperts];
  __shared__ double s_rank[kTokens][kMaxGroups];
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wv;
  const bool live = t < a.T;
  const int E = a.E, k = a.k;
  const double kNone = -INFINITY;

  float z[kItems];
  double key[kItems];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = lane + i * kWave;
    z[i] = live && e < E ? logit<DT>(a.logits, t * E + e) : -INFINITY;
    z[i] = z[i] > -INFINITY ? fminf(z[i], 3.402823466e38f) : -INFINITY;   // NaN and -inf: not there; +inf: the largest
    top = fmaxf(top, z[i]);
  }
  top = wave_max(top);
  const bool softmax = a.score == EP_SCORE_SOFTMAX;
  double sum = 0.0;
  double s64[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool there = z[i] > -INFINITY;
    s64[i] = !there ? 0.0 : softmax ? exp((double)z[i] - (double)top) : 1.0 / (1.0 + exp(-(double)z[i]));
    sum += s64[i];
  }
  if (softmax) {
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kItems; ++i) s64[i] = sum > 0.0 ? s64[i] / sum : 0.0;
  }
  const bool by_sum = a.groups > 1 && a.top == 2;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = lane + i * kWave;
    const bool there = z[i] > -INFINITY;
    double c = kNone;
    if (there) c = s64[i] + (a.bias ? (double)a.bias[e] : 0.0);
    if (!(c > kNone)) c = kNone;                  // a NaN bias
    key[i] = a.bias ? c : (there ? (double)z[i] : kNone);
    if (a.groups > 1 && e < E) s_key[wv][e] = by_sum ? c : key[i];
  }
  if (a.groups > 1) {
    __syncthreads();
    const int size = E / a.groups;
    if (lane < a.groups) {
      double b0 = kNone, b1 = kNone;
      for (int j = 0; j < size; ++j) {
        const double v = s_key[wv][lane * size + j];
        if (v > b0) { b1 = b0; b0 = v; } else if (v > b1) b1 = v;
      }
      s_rank[wv][lane] = a.top == 2 ? b0 + b1 : b0;
    }
    __syncthreads();
    // a group stays when fewer than `keep` groups come before it
    bool stays = false;
    if (lane < a.groups) {
      const double mine = s_rank[wv][lane];
      int before = 0;
      for (int g = 0; g < a.groups; ++g) {
        const double o = s_rank[wv][g];
        before += o > mine || (o == mine && g < lane);
      }
      stays = before < a.keep;
    }
    const uint64_t kept = __ballot(stays);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int e = lane + i * kWave;
      if (e < E && !((kept >> (e / size)) & 1)) key[i] = kNone;
    }
  }

  // k rounds of the wave's largest key; lane j keeps the j-th
  int my_id = -1;
  for (int j = 0; j < k; ++j) {
    double best = kNone;
    int at = INT32_MAX;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (key[i] > best) { best = key[i]; at = lane + i * kWave; }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double ob = __shfl_xor(best, d);
      const int oa = __shfl_xor(at, d);
      if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; }
    }
    if (!(best > kNone)) break;                   // uniform: nothing left
    if (lane == j) my_id = at;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (lane + i * kWave == at) key[i] = kNone;
  }
  float zj = -INFINITY;
  if (my_id >= 0) {
    zj = fminf(logit<DT>(a.logits, t * E + my_id), 3.402823466e38f);
  }
  float w = 0.0f;
  if (a.renorm) {
    // s_j / sum s = softmax of the logs: no score underflows
    const float ls = my_id >= 0 ? log_score(a.score, zj) : -INFINITY;
    const float m = wave_max(ls);
    const float p = my_id >= 0 ? expf(ls - m) : 0.0f;
    const float total = wave_sum(p);
    w = my_id >= 0 ? p / total : 0.0f;
  } else if (my_id >= 0) {
    w = softmax ? (float)(exp((double)zj - (double)top) / sum) : sigmoidf(zj);
  }
  if (live && lane < k) {
    idx[t * k + lane] = (IdxT)my_id;
    weights[t * k + lane] = w * a.scale;
  }
}

// Gradient of the weights with respect to the logits.  With p_j the
// normalised weights (w_j / scale), q_j = scale * grad_j:
//   renormalised: d log-score_j = p_j (q_j - sum_i p_i q_i)
//   otherwise:    d log-score_j = s_j q_j
//   softmax: dz_e = [e chosen] d_j - s_e sum_j d_j (the sum is 0 when
//   renormalised); sigmoid: dz_j = d_j (1 - s_j)
template <int DT, typename IdxT>
__global__ __launch_bounds__(kTokens *kWave) void router_backward_kernel(RouterArgs a, const IdxT *__restrict__ idx,
                                                                         const float *__restrict__ grad,
                                                                         void *__restrict__ dz) {
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wv;
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  const bool softmax = a.score == EP_SCORE_SOFTMAX;
  int id = -1;
  float zj = -INFINITY, q = 0.0f;
  if (lane < k) {
    const int64_t v = (int64_t)idx[t * k + lane];
    if (v >= 0 && v < E) {
      zj = fminf(logit<DT>(a.logits, t * E + v), 3.402823466e38f);
      if (zj > -INFINITY) { id = (int)v; q = grad[t * k + lane] * a.scale; }
    }
  }
  float d = 0.0f, top = 0.0f, sum = 1.0f;
  float z[kItems];
  const bool dense = softmax && !a.renorm;
  if (dense) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int e = lane + i * kWave;
      z[i] = e < E ? logit<DT>(a.logits, t * E + e) : -INFINITY;
      z[i] = z[i] > -INFINITY ? fminf(z[i], 3.402823466e38f) : -INFINITY;
      top = fmaxf(top, z[i]);
    }
    top = wave_max(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i) sum += z[i] > -INFINITY ? expf(z[i] - top) : 0.0f;
    sum = wave_sum(sum);
  }
  if (a.renorm) {
    const float ls = id >= 0 ? log_score(a.score, zj) : -INFINITY;
    const float m = wave_max(ls);
    float p = id >= 0 ? expf(ls - m) : 0.0f;
    const float total = wave_sum(p);
    p = id >= 0 ? p / total : 0.0f;
    const float mean = wave_sum(p * q);
    d = p * (q - mean);
  } else if (id >= 0) {
    d = q * (softmax ? expf(zj - top) / sum : sigmoidf(zj));
  }
  if (!softmax && id >= 0) d *= sigmoidf(-zj);
  const float pull = dense ? wave_sum(d) : 0.0f;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = lane + i * kWave;
    if (i * kWave >= E) break;                    // uniform
    float v = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int oj = __shfl(id, j);
      const float dj = __shfl(d, j);
      if (oj == e) v += dj;
    }
    if (dense && z[i] > -INFINITY) v -= expf(z[i] - top) / sum * pull;
    if (e < E) put<DT>(dz, t * E + e, v);
  }
}

template <int DT>
hipError_t router_dt(const RouterArgs &a, void *idx, int idx64, float *weights, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kTokens * kWave);
  if (idx64)
    hipLaunchKernelGGL((router_kernel<DT, int64_t>), grid, block, 0, s, a, (int64_t *)idx, weights);
  else
    hipLaunchKernelGGL((router_kernel<DT, int32_t>), grid, block, 0, s, a, (int32_t *)idx, weights);
  return hipGetLastError();
}
template <int DT>
hipError_t backward_dt(const RouterArgs &a, const void *idx, int idx64, const float *grad, void *dz, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kTokens * kWave);
  if (idx64)
    hipLaunchKernelGGL((router_backward_kernel<DT, int64_t>), grid, block, 0, s, a, (const int64_t *)idx, grad, dz);
  else
    hipLaunchKernelGGL((router_backward_kernel<DT, int32_t>), grid, block, 0, s, a, (const int32_t *)idx, grad, dz);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router(const RouterArgs &a, void *idx, int idx64, float *weights, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  switch (a.dtype) {
    case EP_FLOAT_F32: return router_dt<EP_FLOAT_F32>(a, idx, idx64, weights, s);
    case EP_FLOAT_BF16: return router_dt<EP_FLOAT_BF16>(a, idx, idx64, weights, s);
    default: return router_dt<EP_FLOAT_F16>(a, idx, idx64, weights, s);
  }
}

hipError_t launch_router_backward(const RouterArgs &a, const void *idx, int idx64, const float *grad_weights,
                                  void *grad_logits, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  switch (a.dtype) {
    case EP_FLOAT_F32: return backward_dt<EP_FLOAT_F32>(a, idx, idx64, grad_weights, grad_logits, s);
    case EP_FLOAT_BF16: return backward_dt<EP_FLOAT_BF16>(a, idx, idx64, grad_weights, grad_logits, s);
    default: return backward_dt<EP_FLOAT_F16>(a, idx, idx64, grad_weights, grad_logits, s);
  }
}

}  // namespace ep
