// Scored routing: logits -> expert ids and weights under a moe_routing rule,
// and the gradient of the weights with respect to the logits.
//
//   s_e = sigmoid(l_e) or softmax(l)_e              the score
//   c_e = s_e + select_bias_e                       what the choice goes by
//   groups of E / n_group consecutive experts: a group's score is its largest
//       c, or the sum of its two largest; the topk_group best groups stay
//   ids = the top_k largest c of the groups that stay (ties: lower id)
//   w_j = scale * s_j / sum_i s_i  (renormalize)  or  scale * s_j
//
// Choice scores and group sums are compared in double precision: two of them
// can lie closer than fp32 rounding, and the ids must not depend on how an
// exponential rounds.  Without a bias the scores are monotone in the logits,
// and the fp32 logits themselves are compared.
#include "moe_common.h"

using namespace moe;

namespace {

constexpr int kSelMaxE = 512;
constexpr int kSelMaxPerLane = kSelMaxE / 64;

// Order-preserving 64-bit key: larger value, larger key; -0 and +0 equal;
// -inf above NaN above 0, the key of an expert that cannot be chosen.
__device__ __forceinline__ uint64_t choice_key(double v) {
  if (v != v) return 1ull;
  const uint64_t u = (uint64_t)__builtin_bit_cast(long long, v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// sum over the lanes of a wave in a fixed order, in every lane
__device__ __forceinline__ float lane0_sum(float v, int n) {
  float s = 0.f;
  for (int j = 0; j < n; ++j) s += __shfl(v, j, kWave);
  return s;
}

// A chosen expert's score up to a factor common to the row, so that
// renormalized weights stay right where every score underflows: softmax
// e^(l - m), sigmoid e^(l - min(m, 0)) / (1 + e^l) (or its mirror for l >= 0),
// with m the largest chosen logit.  Zero where every chosen logit is -inf.
__device__ __forceinline__ float shifted_score(float l, float m, bool sigmoid) {
  if (m == -INFINITY) return 0.f;
  if (!sigmoid) return expf(l - m);
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - fminf(m, 0.f)) / (1.f + expf(l));
}

__device__ __forceinline__ float sigmoid_f32(float l) {
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l) / (1.f + expf(l));
}

// One wave per token; lane l holds experts l, l + 64, ...
__global__ __launch_bounds__(256) void select_wave_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int M, int E, int top_k,
    int sigmoid, int renormalize, int n_group, int topk_group, int group_top, float scale,
    int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights) {
  __shared__ double s_c[4][kSelMaxE];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * 4 + w;
  if (t >= M) return;   // whole wave; no workgroup barrier below
  const float* row = logits + (size_t)t * E;
  float l[kSelMaxPerLane];
  double c[kSelMaxPerLane];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSelMaxPerLane; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? row[e] : -INFINITY;
    mx = fmaxf(mx, l[i]);
  }
  mx = wave_max(mx);
  // the scores in double precision, where the choice needs them
  const bool scored = bias != nullptr || (n_group > 1 && group_top == 2);
  if (scored) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i) {
      const int e = lane + 64 * i;
      if (sigmoid) {
        c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
      } else {
        c[i] = mx == -INFINITY ? 0.0 : exp((double)l[i] - (double)mx);
        if (e < E) z += c[i];
      }
    }
    if (!sigmoid) {
      z = wave_sum_f64(z);
#pragma unroll
      for (int i = 0; i < kSelMaxPerLane; ++i) c[i] = mx == -INFINITY ? 0.0 : c[i] / z;
    }
    if (bias != nullptr) {
#pragma unroll
      for (int i = 0; i < kSelMaxPerLane; ++i) {
        const int e = lane + 64 * i;
        if (e < E) c[i] += (double)bias[e];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i) c[i] = (double)l[i];
  }
  uint64_t key[kSelMaxPerLane];
#pragma unroll
  for (int i = 0; i < kSelMaxPerLane; ++i) {
    const int e = lane + 64 * i;
    // without a bias the order is the logits'
    key[i] = e < E ? choice_key(bias != nullptr ? c[i] : (double)l[i]) : 0ull;
  }
  if (n_group > 1) {
    const int gs = E / n_group;
    double* sc = s_c[w];
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i) {
      const int e = lane + 64 * i;
      if (e < E) sc[e] = c[i];
    }
    __builtin_amdgcn_wave_barrier();
    // lane g scores group g (n_group <= 64)
    uint64_t gkey = 0ull;
    if (lane < n_group) {
      uint64_t k1 = 0ull, k2 = 0ull;
      double v1 = 0.0, v2 = 0.0;
      for (int j = 0; j < gs; ++j) {
        const double v = sc[lane * gs + j];
        const uint64_t k = choice_key(v);
        if (k > k1) {
          k2 = k1; v2 = v1;
          k1 = k; v1 = v;
        } else if (k > k2) {
          k2 = k; v2 = v;
        }
      }
      gkey = choice_key(group_top == 2 ? v1 + v2 : v1);
    }
    int rank = 0;
    for (int g = 0; g < n_group; ++g) {
      const uint64_t o = __shfl(gkey, g, kWave);
      rank += (o > gkey) | ((o == gkey) & (g < lane));
    }
    const unsigned long long kept = __ballot(lane < n_group && rank < topk_group);
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / gs)) & 1ull)) key[i] = 0ull;
    }
  }
  // top_k times the largest key, the lowest expert id among equals
  int my_id = 0;
  float my_l = -INFINITY;
  for (int j = 0; j < top_k; ++j) {
    uint64_t best = 0ull;
    int at = kSelMaxE;
    float bl = 0.f;
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 64 * i;
        bl = l[i];
      }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const uint64_t ob = __shfl_xor(best, d, kWave);
      const int oa = __shfl_xor(at, d, kWave);
      const float ol = __shfl_xor(bl, d, kWave);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        bl = ol;
      }
    }
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i)
      if (at == lane + 64 * i) key[i] = 0ull;
    if (lane == j) {
      my_id = at;
      my_l = bl;
    }
  }
  float weight = 0.f;
  if (renormalize) {
    float m = -INFINITY;
    for (int j = 0; j < top_k; ++j) m = fmaxf(m, __shfl(my_l, j, kWave));
    const float sh = shifted_score(my_l, m, sigmoid != 0);
    const float total = lane0_sum(sh, top_k);
    weight = total == 0.f ? 0.f : scale * (sh / total);
  } else if (sigmoid) {
    weight = scale * sigmoid_f32(my_l);
  } else {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kSelMaxPerLane; ++i)
      if (lane + 64 * i < E) z += shifted_score(l[i], mx, false);
    z = wave_sum(z);
    weight = z == 0.f ? 0.f : scale * (shifted_score(my_l, mx, false) / z);
  }
  if (lane < top_k) {
    topk_ids[(size_t)t * top_k + lane] = my_id;
    topk_weights[(size_t)t * top_k + lane] = weight;
  }
}

// Gradient of the weights to the logits; one wave per token.  With s^ the
// renormalized scores and d_j = scale * g_j:
//   renormalize   s_j (dL/ds_j) = s^_j (d_j - sum_i d_i s^_i)
//   else          s_j (dL/ds_j) = s_j d_j
//   sigmoid       dL/dl_j = (1 - s_j) * that, 0 for the other experts
//   softmax       renormalize: dL/dl_j = that (the sum over j is zero), 0 for
//                 the others; else dL/dl_e = that - p_e sum_j p_j d_j
// An id outside [0, E) takes no part; an id that a row holds twice gets both
// slots' gradients, added in slot order.
__global__ __launch_bounds__(256) void select_backward_wave_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_ids,
    const float* __restrict__ grad_weights, int M, int E, int top_k, int sigmoid, int renormalize,
    float scale, float* __restrict__ grad_logits) {
  __shared__ float s_row[4][kSelMaxE];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * 4 + w;
  if (t >= M) return;   // whole wave; no workgroup barrier below
  const float* row = logits + (size_t)t * E;
  float* out = s_row[w];
  int id = -1;
  float l = -INFINITY, d = 0.f;
  if (lane < top_k) {
    id = topk_ids[(size_t)t * top_k + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      l = row[id];
      d = scale * grad_weights[(size_t)t * top_k + lane];
    }
  }
  const bool dense = !sigmoid && !renormalize;
  float mx = -INFINITY, z = 1.f;
  if (dense) {
    for (int e = lane; e < E; e += 64) mx = fmaxf(mx, row[e]);
    mx = wave_max(mx);
    z = 0.f;
    for (int e = lane; e < E; e += 64) z += shifted_score(row[e], mx, false);
    z = wave_sum(z);
  }
  float g;
  if (renormalize) {
    float m = -INFINITY;
    for (int j = 0; j < top_k; ++j) m = fmaxf(m, __shfl(l, j, kWave));
    const float sh = id >= 0 ? shifted_score(l, m, sigmoid != 0) : 0.f;
    const float total = lane0_sum(sh, top_k);
    const float hat = total == 0.f ? 0.f : sh / total;
    g = hat * (d - lane0_sum(hat * d, top_k));
  } else if (sigmoid) {
    g = sigmoid_f32(l) * d;
  } else {
    g = z == 0.f || id < 0 ? 0.f : shifted_score(l, mx, false) / z * d;
  }
  if (sigmoid) g *= sigmoid_f32(-l);
  const float all = dense ? lane0_sum(g, top_k) : 0.f;
  for (int e = lane; e < E; e += 64)
    out[e] = dense && z != 0.f ? -(shifted_score(row[e], mx, false) / z) * all : 0.f;
  __builtin_amdgcn_wave_barrier();
  // every slot of an id adds the same sum: which one stores it does not matter
  float sum = 0.f;
  for (int j = 0; j < top_k; ++j) {
    const int oj = __shfl(id, j, kWave);
    const float gj = __shfl(g, j, kWave);
    if (oj == id) sum += gj;
  }
  float base = 0.f;
  if (id >= 0) base = out[id];
  __builtin_amdgcn_wave_barrier();
  if (id >= 0) out[id] = base + sum;
  __builtin_amdgcn_wave_barrier();
  for (int e = lane; e < E; e += 64) grad_logits[(size_t)t * E + e] = out[e];
}

}  // namespace

namespace moe_host {

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(select_wave_kernel, dim3(ceil_div_host(a.M, 4)), dim3(256), 0, s, a.logits,
                     a.select_bias, a.M, a.E, a.top_k, a.sigmoid, a.renormalize, a.n_group,
                     a.topk_group, a.group_top, a.scale, a.topk_ids, a.topk_weights);
  return hipGetLastError();
}

hipError_t launch_select_backward(const SelectArgs& a, const float* grad_weights,
                                  float* grad_logits, hipStream_t s) {
  hipLaunchKernelGGL(select_backward_wave_kernel, dim3(ceil_div_host(a.M, 4)), dim3(256), 0, s,
                     a.logits, a.topk_ids, grad_weights, a.M, a.E, a.top_k, a.sigmoid,
                     a.renormalize, a.scale, grad_logits);
  return hipGetLastError();
}

}  // namespace moe_host
