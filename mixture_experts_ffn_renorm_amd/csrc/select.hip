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
constexpr int kSelWaves = 4;
constexpr int kCands = 64;          // candidates a token may have

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

// Maximum and sum over aligned groups of L lanes, in every lane; the order
// is fixed and the same in each lane.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  v = row16_max(v);
  if (L >= 32) {
    uint32_t a = __float_as_uint(v), b = a;
    swap16(a, b);
    v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  }
  if (L == 64) {
    uint32_t a = __float_as_uint(v), b = a;
    swap32(a, b);
    v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  }
  return v;
}
template <int kCtrl>
__device__ __forceinline__ float dpp_add_with(float v) {
  const int s = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, false);
  return v + __builtin_bit_cast(float, s);
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add_with<0xb1>(v);    // quad_perm [1, 0, 3, 2]
  v = dpp_add_with<0x4e>(v);    // quad_perm [2, 3, 0, 1]
  v = dpp_add_with<0x141>(v);   // row_half_mirror
  v = dpp_add_with<0x140>(v);   // row_mirror
  if (L >= 32) {
    uint32_t a = __float_as_uint(v), b = a;
    swap16(a, b);
    v = __uint_as_float(a) + __uint_as_float(b);
  }
  if (L == 64) {
    uint32_t a = __float_as_uint(v), b = a;
    swap32(a, b);
    v = __uint_as_float(a) + __uint_as_float(b);
  }
  return v;
}

// sum over the first n lanes of a wave in lane order, in every lane
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

constexpr float kLog2e = 1.44269504f;

struct SelectParams {
  const float* logits;
  const float* bias;
  int M, E, top_k, sigmoid, renormalize, n_group, topk_group, group_top;
  float scale;
  int32_t* ids;
  float* weights;
};

// The choice for one token by a whole wave, every comparison in double
// precision: for the rows that the fp32 pass below cannot decide.  `c` holds
// E doubles of this wave.  Kept small (no unrolled element loops): it runs
// seldom.
__device__ __forceinline__ void select_exactly(const SelectParams& a, int t, double* c) {
  const int lane = threadIdx.x & 63;
  const int E = a.E, k = a.top_k;
  const float* row = a.logits + (size_t)t * E;
  float mx = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < E; e += 64) mx = fmaxf(mx, row[e]);
  mx = wave_max(mx);
  const bool scored = a.bias != nullptr || (a.n_group > 1 && a.group_top == 2);
  if (scored) {
    // sigmoid: e^-l, softmax: e^(l - mx), summed
    const double sign = a.sigmoid ? -1.0 : 1.0, shift = a.sigmoid ? 0.0 : (double)mx;
    double z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      const double v = exp(sign * ((double)row[e] - shift));
      c[e] = v;
      z += v;
    }
    z = wave_sum_f64(z);
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      // softmax: a row of -inf alone scores 0
      double s = a.sigmoid ? 1.0 + c[e] : z;
      s = (a.sigmoid ? 1.0 : c[e]) / s;
      if (!a.sigmoid && mx == -INFINITY) s = 0.0;
      c[e] = a.bias != nullptr ? s + (double)a.bias[e] : s;
    }
  } else {
#pragma unroll 1
    for (int e = lane; e < E; e += 64) c[e] = (double)row[e];
  }
  __builtin_amdgcn_wave_barrier();
  unsigned long long kept = ~0ull;
  const int gs = E / a.n_group;
  if (a.n_group > 1) {
    // lane g scores group g (at most 64)
    uint64_t gkey = 0ull;
    if (lane < a.n_group) {
      uint64_t k1 = 0ull, k2 = 0ull;
      double v1 = 0.0, v2 = 0.0;
#pragma unroll 1
      for (int j = 0; j < gs; ++j) {
        const double v = c[lane * gs + j];
        const uint64_t q = choice_key(v);
        if (q > k1) {
          k2 = k1; v2 = v1;
          k1 = q; v1 = v;
        } else if (q > k2) {
          k2 = q; v2 = v;
        }
      }
      gkey = choice_key(a.group_top == 2 ? v1 + v2 : v1);
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.n_group; ++g) {
      const uint64_t o = __shfl(gkey, g, kWave);
      rank += (o > gkey) | ((o == gkey) & (g < lane));
    }
    kept = __ballot(lane < a.n_group && rank < a.topk_group);
  }
  __builtin_amdgcn_wave_barrier();
  // without a bias the order is the logits'
  unsigned open = 0u;   // bit i: expert lane + 64 i can still be chosen
#pragma unroll 1
  for (int i = 0, e = lane; e < E; ++i, e += 64) {
    if (a.bias == nullptr) c[e] = (double)row[e];
    if (a.n_group == 1 || ((kept >> (e / gs)) & 1ull)) open |= 1u << i;
  }
  // top_k times the largest key, the lowest expert id among equals
  int my_id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0ull;
    int at = kSelMaxE;
#pragma unroll 1
    for (int i = 0, e = lane; e < E; ++i, e += 64) {
      const uint64_t q = (open >> i) & 1u ? choice_key(c[e]) : 0ull;
      if (q > best) {
        best = q;
        at = e;
      }
    }
#pragma unroll 1
    for (int d = 32; d >= 1; d >>= 1) {
      const uint64_t ob = __shfl_xor(best, d, kWave);
      const int oa = __shfl_xor(at, d, kWave);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if ((at & 63) == lane) open &= ~(1u << (at >> 6));
    if (lane == j) my_id = at;
  }
  const float l = lane < k ? row[my_id] : -INFINITY;
  float w;
  if (a.renormalize) {
    const float m = wave_max(l);
    const float sh = shifted_score(l, m, a.sigmoid != 0);
    const float total = wave_sum(lane < k ? sh : 0.f);
    w = total == 0.f ? 0.f : a.scale * (sh / total);
  } else if (a.sigmoid) {
    w = a.scale * sigmoid_f32(l);
  } else {
    float z = 0.f;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) z += shifted_score(row[e], mx, false);
    z = wave_sum(z);
    w = z == 0.f ? 0.f : a.scale * (shifted_score(l, mx, false) / z);
  }
  if (lane < k) {
    a.ids[(size_t)t * k + lane] = my_id;
    a.weights[(size_t)t * k + lane] = w;
  }
  __builtin_amdgcn_wave_barrier();   // c may be written again
}

// L lanes per token, up to C experts per lane in pieces of V consecutive
// ones; each lane's experts lie in one group.
//
// 1. c in fp32 (without a bias: the logits, exactly).
// 2. Groups: each lane's one or two largest c, joined over the group's
//    lanes; a group stays if fewer than topk_group groups beat it.
// 3. The top_k-th largest of the L lane maxima bounds the top_k-th largest c
//    from below, so the experts at or above it (less the error) hold every
//    one that can be chosen: usually little more than top_k.  They are packed
//    into LDS, a sigmoid's choice scores evaluated again in double precision,
//    and ranked against each other.
// 4. A row that this cannot decide is done over in double precision by the
//    whole wave: two groups, or two neighbours in a biased softmax's order,
//    closer than the error of c; -inf or NaN among the chosen; more than
//    kCands candidates (rows of ties).
//
// Error of c: sigmoid 2^-22 (its slope times the exponent's rounding, two
// hardware transcendentals, two roundings), softmax 2^-19 (the common sum of
// C / 4 + 6 terms in a row, each rounding once), and 2^-24 |c| for the bias.
template <int L, int C, int V>
__global__ __launch_bounds__(64 * kSelWaves, C <= 8 ? 5 : C == 16 ? 4 : 3) void select_kernel(SelectParams a, int lpg) {
  constexpr int T = 64 / L;                    // tokens per wave
  constexpr int kList = 64;                    // rows to do over, per wave
  struct TokenLds {
    double c[kCands];                          // candidates: choice score, id, logit
    int id[kCands];
    float l[kCands];
    float lm[L];                               // lane maxima
    float top_c[34], top_l[34];                // by rank
    int top_id[34];
  };
  union WaveLds {
    TokenLds tok[T];
    double c[kSelMaxE];
  };
  __shared__ __attribute__((aligned(16))) WaveLds s_all[kSelWaves];
  __shared__ int s_list[kSelWaves][kList];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int li = lane % L, base = lane - li;   // lane within its token
  TokenLds& s = s_all[w].tok[lane / L];
  const int E = a.E, k = a.top_k, G = a.n_group;
  const int gs = E / G;
  const int grp = li / lpg, sub = li - grp * lpg;
  const bool scored = a.bias != nullptr || (G > 1 && a.group_top == 2);
  const bool by_logit = a.bias == nullptr;     // the order of experts is exact
  const float eps = a.sigmoid ? 0x1p-21f : 0x1p-18f;   // of a difference of two c
  // first expert of piece i: lane_e0 + i * V * lpg; present while below lane_end
  int lane_e0 = grp * gs + V * sub;
  const int lane_end = grp < G ? (grp + 1) * gs : 0;
  auto expert = [&](int i) { return lane_e0 + (i / V) * V * lpg + i % V; };

  const int step = (int)gridDim.x * kSelWaves * T;
  int t0 = ((int)blockIdx.x * kSelWaves + w) * T;
  while (t0 < a.M) {
    int nlist = 0;
#pragma unroll 1
    for (; t0 < a.M && nlist <= kList - T; t0 += step) {
      // keeps each expert's index from being held in a register of its own
      asm volatile("" : "+v"(lane_e0));
      const int t = t0 + lane / L;
      const bool live = t < a.M;
      const float* row = a.logits + (size_t)(live ? t : a.M - 1) * E;
      float l[C], c[C];
#pragma unroll
      for (int i = 0; i < C; i += V) {
        const int e = expert(i);
        if constexpr (V == 4) {
          f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (e < lane_end) v = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) l[i + j] = v[j];
        } else {
          l[i] = e < lane_end ? row[e] : -INFINITY;
        }
      }
      // the softmax over all experts, where it is needed
      const bool full = !a.sigmoid && (scored || !a.renormalize);
      float mx = -INFINITY, z = 0.f;
      if (full) {
#pragma unroll
        for (int i = 0; i < C; ++i) mx = fmaxf(mx, l[i]);
        mx = lanes_max<L>(mx);
        float zp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < C; ++i) {
          c[i] = __builtin_amdgcn_exp2f((l[i] - mx) * kLog2e);
          zp[i & 3] += c[i];
        }
        z = lanes_sum<L>((zp[0] + zp[1]) + (zp[2] + zp[3]));
      }
      if (scored) {
        if (a.sigmoid) {
#pragma unroll
          for (int i = 0; i < C; ++i)
            c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * l[i]));
        } else {
          const float rz = 1.f / z;
#pragma unroll
          for (int i = 0; i < C; ++i) c[i] *= rz;
        }
#pragma unroll
        for (int i = 0; i < C; i += V) {
          const int e = expert(i);
          if constexpr (V == 4) {
            f32x4 b = {0.f, 0.f, 0.f, 0.f};
            if (a.bias != nullptr) b = *reinterpret_cast<const f32x4*>(a.bias + min(e, E - 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i + j] = e < lane_end ? c[i + j] + b[j] : -INFINITY;
          } else {
            const float b = a.bias != nullptr ? a.bias[min(e, E - 1)] : 0.f;
            c[i] = e < lane_end ? c[i] + b : -INFINITY;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) c[i] = l[i];
      }
      bool unsure = false;
      bool open = grp < G;                       // this lane's group stays
      if (G > 1) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          m2 = fmaxf(m2, fminf(m1, c[i]));
          m1 = fmaxf(m1, c[i]);
        }
        const float o1 = m1, o2 = m2;
#pragma unroll 1
        for (int o = 1; o < lpg; ++o) {
          const int src = base + (open ? grp * lpg + (sub + o) % lpg : li);
          const float p1 = __shfl(o1, src, kWave), p2 = __shfl(o2, src, kWave);
          m2 = fmaxf(fmaxf(m2, p2), fminf(m1, p1));
          m1 = fmaxf(m1, p1);
        }
        const float score = a.group_top == 2 ? m1 + m2 : m1;
        int rank = 0;
#pragma unroll 2
        for (int g = 0; g < G; ++g) {
          const float o = __shfl(score, base + g * lpg, kWave);
          rank += (o > score) | ((o == score) & (g < grp));
        }
        open = open && rank < a.topk_group;
        if (scored && a.topk_group < G) {
          // the worst group that stays and the best that does not
          const float lo = -lanes_max<L>(open ? -score : -INFINITY);
          const float hi = lanes_max<L>(!open && grp < G ? score : -INFINITY);
          unsure = !(lo - hi > 2.f * eps + 0x1p-21f * fmaxf(fabsf(lo), fabsf(hi)));
        } else {
          // a group of -inf (or NaN) alone among those that stay
          unsure = lanes_max<L>(open && !(score > -INFINITY) ? 1.f : 0.f) > 0.f;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (by_logit) c[i] = l[i];
          if (!open) c[i] = -INFINITY;
        }
      }
      // the bound
      float lmax = c[0];
#pragma unroll
      for (int i = 1; i < C; ++i) lmax = fmaxf(lmax, c[i]);
      if (lmax != lmax) lmax = -INFINITY;
      s.lm[li] = lmax;
#pragma unroll
      for (int i = 0; i < kCands / L; ++i) s.c[i * L + li] = -INFINITY;
      __builtin_amdgcn_wave_barrier();
      int gt = 0;
#pragma unroll
      for (int j = 0; j < L; j += 4) {
        const f32x4 o = *reinterpret_cast<const f32x4*>(s.lm + j);
#pragma unroll
        for (int q = 0; q < 4; ++q) gt += o[q] > lmax;
      }
      const float bound = -lanes_max<L>(gt < k ? -lmax : -INFINITY);
      const float tol = by_logit ? 0.f : 2.f * eps + 0x1p-22f * fabsf(bound);
      // fewer than top_k lanes hold anything: every finite expert
      const float cut = bound > -INFINITY ? bound - tol : -3.4028235e38f;
      // candidates into LDS
      int n = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) n += c[i] >= cut;
      int pos = n;
#pragma unroll
      for (int d = 1; d < L; d <<= 1) {
        const int o = __shfl_up(pos, d, L);
        if (li >= d) pos += o;
      }
      const int total = __shfl(pos, base + L - 1, kWave);
      pos -= n;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (c[i] >= cut) {
          if (pos < kCands) {
            s.c[pos] = (double)c[i];
            s.l[pos] = l[i];
            s.id[pos] = expert(i);
          }
          ++pos;
        }
      unsure = unsure || total < k || total > kCands;
      const int most = min(kCands, (int)wave_max((float)total));
      __builtin_amdgcn_wave_barrier();
      if (!by_logit && a.sigmoid) {
#pragma unroll 1
        for (int q = li; q < most; q += L)
          if (q < total)
            s.c[q] = 1.0 / (1.0 + exp(-(double)s.l[q])) + (double)a.bias[s.id[q]];
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll 1
      for (int q = li; q < most; q += L) {
        const double my = s.c[q];
        const int id = s.id[q];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < most; ++o) {
          const double ot = s.c[o];
          rank += (ot > my) | ((ot == my) & (s.id[o] < id));
        }
        if (q < total && rank <= k) {
          s.top_c[rank] = (float)my;
          s.top_l[rank] = s.l[q];
          s.top_id[rank] = id;
        }
      }
      __builtin_amdgcn_wave_barrier();
      // lane j: slot j
      int id = 0;
      float lj = -INFINITY;
      if (li < k) {
        id = s.top_id[li];
        lj = s.top_l[li];
      }
      if (!by_logit && !a.sigmoid) {
        bool close = false;
        if (li < k && li + 1 < total) {
          const float my = s.top_c[li], nx = s.top_c[li + 1];
          close = !(my - nx > eps + 0x1p-22f * fmaxf(fabsf(my), fabsf(nx)));
        }
        unsure = unsure || lanes_max<L>(close ? 1.f : 0.f) > 0.f;
      }
      float wt;
      if (a.renormalize) {
        const float m = lanes_max<L>(lj);
        const float sh = li < k ? shifted_score(lj, m, a.sigmoid != 0) : 0.f;
        const float sum = lanes_sum<L>(sh);
        wt = sum == 0.f ? 0.f : a.scale * (sh / sum);
      } else if (a.sigmoid) {
        wt = a.scale * sigmoid_f32(lj);
      } else {
        wt = a.scale * (expf(lj - mx) / z);
      }
      if (live && !unsure && li < k) {
        a.ids[(size_t)t * k + li] = id;
        a.weights[(size_t)t * k + li] = wt;
      }
      const bool again = live && unsure && li == 0;
      const unsigned long long m = __ballot(again);
      if (again) s_list[w][nlist + __popcll(m & ((1ull << lane) - 1ull))] = t;
      nlist += __popcll(m);
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll 1
    for (int i = 0; i < nlist; ++i) select_exactly(a, s_list[w][i], s_all[w].c);
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

namespace {

template <int L, int C, int V>
void go(const SelectArgs& a, int lpg, hipStream_t s) {
  const SelectParams p{a.logits, a.select_bias, a.M, a.E, a.top_k, a.sigmoid, a.renormalize,
                       a.n_group, a.topk_group, a.group_top, a.scale, a.topk_ids,
                       a.topk_weights};
  constexpr int per = kSelWaves * 64 / L;
  // waves of a large batch take several turns: the bias stays in registers
  const int wgs = ceil_div_host(a.M, per), most = 8 * device_cu_count();
  hipLaunchKernelGGL((select_kernel<L, C, V>), dim3(wgs < most ? wgs : most), dim3(64 * kSelWaves),
                     0, s, p, lpg);
}

// Experts per lane of a layout with L lanes a token.
int per_lane(int L, int V, int G, int gs) {
  const int lpg = L / G;
  return lpg == 0 ? kSelMaxE + 1 : V * ceil_div_host(gs, V * lpg);
}

template <int V>
hipError_t launch_select_v(const SelectArgs& a, hipStream_t s) {
  const int G = a.n_group, gs = a.E / G;
  // A wave per token while the chip has waves for them; above, four or two
  // tokens per wave, as far as the lane maxima (L of them) bound top_k well.
  int L = 64;
  if (a.M > 16 * device_cu_count()) {
    if (a.top_k <= 12 && per_lane(16, V, G, gs) <= 32) L = 16;
    else if (a.top_k <= 26 && per_lane(32, V, G, gs) <= 16) L = 32;
  }
  const int n = per_lane(L, V, G, gs), lpg = L / G;
  if (L == 64) {
    if (n <= 4) go<64, 4, V>(a, lpg, s);
    else if (n <= 8) go<64, 8, V>(a, lpg, s);
    else go<64, 16, V>(a, lpg, s);
  } else if (L == 32) {
    if (n <= 4) go<32, 4, V>(a, lpg, s);
    else if (n <= 8) go<32, 8, V>(a, lpg, s);
    else go<32, 16, V>(a, lpg, s);
  } else {
    if (n <= 4) go<16, 4, V>(a, lpg, s);
    else if (n <= 8) go<16, 8, V>(a, lpg, s);
    else if (n <= 16) go<16, 16, V>(a, lpg, s);
    else go<16, 32, V>(a, lpg, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  // four consecutive experts at a time where a group holds whole fours
  return a.E / a.n_group % 4 == 0 ? launch_select_v<4>(a, s) : launch_select_v<1>(a, s);
}

hipError_t launch_select_backward(const SelectArgs& a, const float* grad_weights,
                                  float* grad_logits, hipStream_t s) {
  hipLaunchKernelGGL(select_backward_wave_kernel, dim3(ceil_div_host(a.M, 4)), dim3(256), 0, s,
                     a.logits, a.topk_ids, grad_weights, a.M, a.E, a.top_k, a.sigmoid,
                     a.renormalize, a.scale, grad_logits);
  return hipGetLastError();
}

}  // namespace moe_host
