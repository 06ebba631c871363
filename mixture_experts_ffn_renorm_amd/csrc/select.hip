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
// Candidates a token may have before its row is done over: with eight lanes
// of sixteen experts open and top_k 8, 64 are too few for one token in 8000.
constexpr int kSelCands = 128;

// Order-preserving 64-bit key: larger value, larger key; -0 and +0 equal;
// -inf above NaN above 0, the key of an expert that cannot be chosen.
__device__ __forceinline__ uint64_t choice_key(double v) {
  if (v != v) return 1ull;
  const uint64_t u = (uint64_t)__builtin_bit_cast(long long, v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double key_value(uint64_t k) {
  if (k <= 1ull) return __builtin_nan("");
  return __builtin_bit_cast(double, (long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

// A candidate's key: fp32 value in order, then the lower id first; distinct
// ids give distinct keys.  (A sigmoid's refined key: a double's upper 55 bits
// in order, then the id.)
__device__ __forceinline__ uint64_t cand_key(float v, int id) {
  uint32_t u = __float_as_uint(v + 0.f);   // -0 as +0
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)(kSelMaxE - 1 - id);
}
__device__ __forceinline__ int cand_id(uint64_t key) {
  return kSelMaxE - 1 - (int)(key & (kSelMaxE - 1));
}
__device__ __forceinline__ float cand_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// Unsigned maximum over the wave, in every lane.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_umax_with(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = dpp_umax_with<0xb1>(v);    // quad_perm [1, 0, 3, 2]
  v = dpp_umax_with<0x4e>(v);    // quad_perm [2, 3, 0, 1]
  v = dpp_umax_with<0x141>(v);   // row_half_mirror
  v = dpp_umax_with<0x140>(v);   // row_mirror
  uint32_t a = v, b = v;
  swap16(a, b);
  a = b = max(a, b);
  swap32(a, b);
  return max(a, b);
}

// e^x: x = n ln 2 + r with |r| <= ln 2 / 2 (ln 2 in two parts), the Taylor
// series of e^r to r^13 / 13! (the next term is below 2^-57), times 2^n.
// The constants are made opaque scalars where they are used: the compiler
// would hold two dozen of them in vector registers through the kernel.
__device__ __forceinline__ double exp_f64(double x) {
  const double c = fmin(fmax(x, -800.0), 800.0);
  double log2e = 0x1.71547652b82fep+0, ln2_hi = -0x1.62e42fefa39efp-1;
  double ln2_lo = -0x1.abc9e3b39803fp-56;
  asm volatile("" : "+s"(log2e), "+s"(ln2_hi), "+s"(ln2_lo));
  const double n = __builtin_rint(c * log2e);
  const double r = __builtin_fma(n, ln2_lo, __builtin_fma(n, ln2_hi, c));
  double p = 1.0 / 6227020800.0;
  asm volatile("" : "+s"(p));
  double y = p;
  constexpr double kInv[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                             1.0 / 40320.0,     1.0 / 5040.0,     1.0 / 720.0,     1.0 / 120.0,
                             1.0 / 24.0,        1.0 / 6.0};
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    double q = kInv[i];
    asm volatile("" : "+s"(q));
    y = __builtin_fma(y, r, q);
  }
  y = __builtin_fma(__builtin_fma(__builtin_fma(y, r, 0.5), r, 1.0), r, 1.0);
  y = __builtin_ldexp(y, (int)n);
  return x != x ? x : y;
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

// Inclusive prefix sums over aligned groups of L lanes (DPP shifts inside a
// row of 16, then each row's total into the next rows).
template <int kCtrl, int kRowMask, bool kBound>
__device__ __forceinline__ int dpp_shifted_addi(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xf, kBound);
}
template <int L>
__device__ __forceinline__ int lanes_scan(int v) {
  v = dpp_shifted_addi<0x111, 0xf, true>(v);    // row_shr:1
  v = dpp_shifted_addi<0x112, 0xf, true>(v);    // row_shr:2
  v = dpp_shifted_addi<0x114, 0xf, true>(v);    // row_shr:4
  v = dpp_shifted_addi<0x118, 0xf, true>(v);    // row_shr:8
  if (L >= 32) v = dpp_shifted_addi<0x142, 0xa, false>(v);   // row_bcast:15
  if (L == 64) v = dpp_shifted_addi<0x143, 0xc, false>(v);   // row_bcast:31
  return v;
}

// A chosen expert's score up to a factor common to the row, so that
// renormalized weights stay right where every score underflows: softmax
// e^(l - m), sigmoid e^(l - min(m, 0)) / (1 + e^l) (or its mirror for l >= 0),
// with m the largest chosen logit.  Without such a one: 0, NaN for NaN.
__device__ __forceinline__ float shifted_score(float l, float m, bool sigmoid) {
  if (m == -INFINITY) return l != l ? l : 0.f;
  if (!sigmoid) return expf(l - m);
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - fminf(m, 0.f)) / (1.f + expf(l));
}

__device__ __forceinline__ float sigmoid_f32(float l) {
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l) / (1.f + expf(l));
}

constexpr float kLog2e = 1.44269504f;

// The same on the hardware's exponential (one ulp; the rounding of its
// argument adds |x| 2^-24 relative): shift is m for the softmax, min(m, 0)
// for a sigmoid, and finite.
__device__ __forceinline__ float hw_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float hw_sigmoid(float l) {
  const float t = hw_exp(-fabsf(l));
  return (l >= 0.f ? 1.f : t) * __builtin_amdgcn_rcpf(1.f + t);
}
__device__ __forceinline__ float fast_score(float l, float shift, bool sigmoid) {
  const float e = hw_exp(l >= 0.f && sigmoid ? 0.f : l - shift);
  return sigmoid ? e * __builtin_amdgcn_rcpf(1.f + hw_exp(-fabsf(l))) : e;
}

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
// E doubles of this wave.  Kept small (no unrolled element loops), so that it
// takes no registers from that pass; how often it runs depends on the rule and
// the logits (below).
__device__ __forceinline__ void select_exactly(const SelectParams& a, int t, double* c) {
  int lane = threadIdx.x & 63, E = a.E, G = a.n_group;
  const int k = a.top_k;
  // opaque here, so that nothing computed from them is held in registers
  // through the fp32 pass
  asm volatile("" : "+v"(lane));
  asm volatile("" : "+s"(E), "+s"(G));
  const float* row = a.logits + (size_t)t * E;
  float mx = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < E; e += 64) mx = fmaxf(mx, row[e]);
  mx = wave_max(mx);
  const bool scored = a.bias != nullptr || (G > 1 && a.group_top == 2);
  if (scored) {
    // sigmoid: e^-l, softmax: e^(l - mx), summed
    const double sign = a.sigmoid ? -1.0 : 1.0, shift = a.sigmoid ? 0.0 : (double)mx;
    double z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      const double v = exp_f64(sign * ((double)row[e] - shift));
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
  const int gs = E / G;
  if (G > 1) {
    // 64 / n_group lanes scan a group (n_group <= 64) and join their two best
    const int lpg = 64 / G;
    const int g = min(lane / lpg, G - 1), sub = lane - g * lpg;
    uint64_t k1 = 0ull, k2 = 0ull;   // keys order as the values do
#pragma unroll 1
    for (int j = sub; j < gs && sub < lpg; j += lpg) {
      const uint64_t q = choice_key(c[g * gs + j]);
      k2 = max(k2, min(k1, q));
      k1 = max(k1, q);
    }
    const uint64_t o1 = k1, o2 = k2;
#pragma unroll 1
    for (int o = 1; o < lpg; ++o) {
      const int src = sub < lpg ? g * lpg + (sub + o) % lpg : lane;
      const uint64_t p1 = __shfl(o1, src, kWave), p2 = __shfl(o2, src, kWave);
      k2 = max(max(k2, p2), min(k1, p1));
      k1 = max(k1, p1);
    }
    if (a.group_top == 2) k1 = choice_key(key_value(k1) + key_value(k2));
    int rank = 0;
#pragma unroll 2
    for (int o = 0; o < G; ++o) {
      const uint64_t other = __shfl(k1, o * lpg, kWave);
      rank += (other > k1) | ((other == k1) & (o < g));
    }
    // bit g: group g stays
    const unsigned long long m = __ballot(rank < a.topk_group && sub == 0);
    kept = 0ull;
#pragma unroll 1
    for (int o = 0; o < G; ++o) kept |= ((m >> (o * lpg)) & 1ull) << o;
  }
  // without a bias the order is the logits'
  constexpr int kPer = kSelMaxE / 64;
  uint32_t hi[kPer], lo[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    uint64_t q = 0ull;
    if (e < E && (G == 1 || ((kept >> (e / gs)) & 1ull)))
      q = choice_key(a.bias != nullptr ? c[e] : (double)row[e]);
    hi[i] = (uint32_t)(q >> 32);
    lo[i] = (uint32_t)q;
  }
  // top_k times the largest key, the lowest expert id among equals: the
  // largest upper half, then the largest lower half of those, then the id
  int my_id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t h = hi[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) h = max(h, hi[i]);
    h = wave_umax(h);
    uint32_t v = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v = max(v, hi[i] == h ? lo[i] : 0u);
    v = wave_umax(v);
    uint32_t first = 0u;   // kSelMaxE - id, the largest for the lowest id
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (hi[i] == h && lo[i] == v) first = kSelMaxE - (lane + 64 * i);
    const int at = kSelMaxE - (int)wave_umax(first);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (at == lane + 64 * i) hi[i] = lo[i] = 0u;
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
//    into LDS and ranked against each other; where two neighbours in a biased
//    sigmoid's order are closer than the error of c, again with choice scores
//    in double precision.
// 4. A row that this cannot decide is done over in double precision by the
//    whole wave: two groups, or two neighbours in a biased softmax's order,
//    closer than the error of c; a sigmoid's closer than double precision's;
//    -inf or NaN among the chosen; more than kCands candidates (rows of ties).
//
//    One such row takes its wave 3 to 4 us, several are done in turn.  A
//    biased sigmoid without groups has next to none (65536 x 512, two batches
//    of logits in turn, std 0.9, 4 and 6: 42, 43, 44 us).  A biased softmax
//    has many where one probability stands far above those at the border (the
//    same: 48, 179, 292 us; 8192 x 256, by the biases drawn: 12, 13 to 26, 12
//    to 28), a sum of two a few where the border of the groups lies close (8192
//    x 256 in 8 groups: none 9 us, a few 13 to 17; softmax with a bias, std 6:
//    20 to 39).  Rows whose choice reaches masked experts (a bias or logits of
//    -inf) are all done over, and where top_k is more than the lanes that are
//    open, with more than kCands experts in them.
//
// Error of c: sigmoid 2^-22 (its slope times the exponent's rounding, two
// hardware transcendentals, two roundings), softmax 2^-19 of the largest
// probability (the common sum of C / 4 + 6 terms in a row, each rounding
// once), and 2^-24 |c| for the bias.
//
// Bound by vector instructions (72 to 75 % of the time), two transcendentals
// per expert among them, the rest loads that few waves per SIMD do not hide,
// and, for few tokens, by the chain of steps: 65536 x 512, sigmoid with a
// bias, top_k 10, in 47 us (2.9 TB/s of logits; 33 us without one), 8192 x 256
// in 8 groups in 9.1 (3 the launch; 6.6 by the logits alone, 7.7 with scores
// and bias), one token in 5.5.  A wave per token with every comparison in
// double precision, the simplest form, took 192 and 37 us for the first two.
template <int L, int C, int V>
__global__ __launch_bounds__(64 * kSelWaves) void select_kernel(SelectParams a, int lpg) {
  constexpr int T = 64 / L;                    // tokens per wave
  constexpr int kList = 64;                    // rows to do over, per wave
  constexpr int kCands = kSelCands;
  struct TokenLds {
    uint64_t cand[kCands];                     // candidates' keys
    uint64_t top[34];                          // by rank
    float lm[L];                               // lane maxima
    uint16_t id[kCands];
  };
  union WaveLds {
    TokenLds tok[T];
    double c[kSelMaxE];
  };
  __shared__ __attribute__((aligned(16))) WaveLds s_all[kSelWaves];
  __shared__ int s_list[kSelWaves][kList];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int li = lane % L, base = lane - li;         // lane within its token
  TokenLds& s = s_all[w].tok[lane / L];
  const int E = a.E, k = a.top_k, G = a.n_group;
  const int gs = E / G;
  const int grp = li / lpg, sub = li - grp * lpg;
  const bool scored = a.bias != nullptr || (G > 1 && a.group_top == 2);
  const bool by_logit = a.bias == nullptr;     // the order of experts is exact
  const bool refine = !by_logit && a.sigmoid;  // candidates evaluated again
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
      // opaque in each turn, so that what is computed from them (the index of
      // each expert, addresses) is not held in registers of its own
      asm volatile("" : "+v"(lane_e0), "+v"(li), "+v"(base));
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
      float mx = -INFINITY, z = 0.f, rz = 0.f;
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
      // error of a difference of two c (the softmax's is relative to its
      // largest probability, 1 / z)
      const float eps = a.sigmoid ? 0x1p-21f : 0x1p-18f * __builtin_amdgcn_rcpf(z);
      if (scored) {
        if (a.sigmoid) {
#pragma unroll
          for (int i = 0; i < C; ++i)
            c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * l[i]));
        } else {
          rz = __builtin_amdgcn_rcpf(z);
#pragma unroll
          for (int i = 0; i < C; ++i) c[i] *= rz;
        }
        // experts that are not there: -inf for their bias
#pragma unroll
        for (int i = 0; i < C; i += V) {
          const int e = expert(i);
          const float none = e < lane_end ? 0.f : -INFINITY;
          if constexpr (V == 4) {
            f32x4 b = {none, none, none, none};
            if (a.bias != nullptr && e < lane_end) b = *reinterpret_cast<const f32x4*>(a.bias + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i + j] += b[j];
          } else {
            c[i] += a.bias != nullptr && e < lane_end ? a.bias[e] : none;
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
          // The worst group that stays and the best that does not, each moved
          // by the error that its c have from their own magnitudes (a sum of a
          // large positive and a large negative c keeps the error of both).
          // -inf: masked by the bias, behind every finite sum; a sum past the
          // type's range counts as its end.
          const float last = a.group_top == 2 ? m2 : m1;
          const float by = 0x1p-22f * fabsf(m1) + (a.group_top == 2 ? 0x1p-22f * fabsf(m2) : 0.f);
          const bool some = last > -INFINITY;
          const float sum = fminf(fmaxf(score, -3.4028235e38f), 3.4028235e38f);
          const float lo = -lanes_max<L>(!open ? -INFINITY : some ? by - sum : INFINITY);
          const float hi = lanes_max<L>(!open && grp < G && some ? sum + by : -INFINITY);
          unsure = !(lo - hi > 2.f * eps);
        } else {
          // a group of -inf (or NaN) alone among those that stay
          unsure = lanes_max<L>(open && !(score > -INFINITY) ? 1.f : 0.f) > 0.f;
        }
        if (scored && by_logit) {
#pragma unroll
          for (int i = 0; i < C; ++i) c[i] = l[i];
        }
      }
      // the bound
      float lmax = c[0];
#pragma unroll
      for (int i = 1; i < C; ++i) lmax = fmaxf(lmax, c[i]);
      if (lmax != lmax || !open) lmax = -INFINITY;
      s.lm[li] = lmax;
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
      // Never -inf, which experts that are not there have for their c: fewer
      // than top_k lanes hold anything, or a bias of the type's lowest value
      // is the bound, whose difference overflows.
      const float cut = open ? fmaxf(bound - tol, -3.4028235e38f) : INFINITY;
      // this lane's candidates, expert i at bit C - 1 - i
      uint32_t mask = 0u;
#pragma unroll
      for (int i = 0; i < C; ++i) mask = 2u * mask + (c[i] >= cut ? 1u : 0u);
      if (!open) mask = 0u;   // +inf is no candidate either
      const int n = __popc(mask);
      const int upto = lanes_scan<L>(n);
      const int total = (int)lanes_max<L>((float)upto);
      unsure = unsure || total < k || total > kCands;
      const int most = min(kCands, (int)lanes_max<64>((float)total));
      int pos = upto - n;
      while (__any(mask != 0u)) {
        if (mask != 0u) {
          const int i = C - 32 + __clz(mask);
          if (pos < kCands) s.id[pos] = (uint16_t)expert(i);
          mask &= ~(0x80000000u >> __clz(mask));
          ++pos;
        }
      }
      __builtin_amdgcn_wave_barrier();
      // lane j: slot j, after a second turn with a sigmoid's keys in double
      // precision if any token of the wave needs one
      int id = 0;
      float lj = -INFINITY;
      bool fine = false, close;
#pragma unroll 1
      for (;;) {
#pragma unroll 1
        for (int q = li; q < most; q += L) {
          uint64_t key = 0ull;
          if (q < total) {
            const int id = s.id[q];
            const float v = row[id];
            if (fine) {
              const double u = 1.0 + exp_f64(-(double)v);
              key = (choice_key(1.0 / u + (double)a.bias[id]) & ~(uint64_t)(kSelMaxE - 1)) |
                    (uint64_t)(kSelMaxE - 1 - id);
            } else if (by_logit) {
              key = cand_key(v, id);
            } else {
              const float e = __builtin_amdgcn_exp2f(kLog2e * (a.sigmoid ? -v : v - mx));
              key = cand_key((a.sigmoid ? __builtin_amdgcn_rcpf(1.f + e) : e * rz) + a.bias[id], id);
            }
          }
          s.cand[q] = key;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = li; q < most; q += L) {
          const uint64_t my = s.cand[q];
          int rank = 0;
#pragma unroll 4
          for (int o = 0; o < most; ++o) rank += s.cand[o] > my;
          if (q < total && rank <= k) s.top[rank] = my;
        }
        __builtin_amdgcn_wave_barrier();
        close = false;
        if (li < k) {
          const uint64_t my = s.top[li];
          id = min(cand_id(my), E - 1);   // unset in a row that is done over
          lj = by_logit ? cand_value(my) : row[id];
          if (!by_logit && li + 1 < total) {
            const uint64_t nx = s.top[li + 1];
            if (fine) {
              // the keys dropped the last nine bits, and the doubles are an
              // ulp or two off
              close = my - nx < 2ull * kSelMaxE;
            } else {
              const float x = cand_value(my), y = cand_value(nx);
              close = !(x - y > eps + 0x1p-22f * fmaxf(fabsf(x), fabsf(y)));
            }
          }
        }
        if (!refine || fine || !__any(close)) break;
        fine = true;
      }
      unsure = unsure || close;
      if (!by_logit) unsure = lanes_max<L>(unsure ? 1.f : 0.f) > 0.f;
      float wt;
      if (a.renormalize) {
        const float m = lanes_max<L>(lj);
        // a bias may choose experts whose logits are -inf, and those alone
        const float sh = li < k && m > -INFINITY
                             ? fast_score(lj, a.sigmoid ? fminf(m, 0.f) : m, a.sigmoid) : 0.f;
        const float sum = lanes_sum<L>(sh);
        wt = sum == 0.f ? 0.f : a.scale * (sh * __builtin_amdgcn_rcpf(sum));
      } else if (a.sigmoid) {
        wt = a.scale * hw_sigmoid(lj);
      } else {
        wt = a.scale * (hw_exp(lj - mx) * __builtin_amdgcn_rcpf(z));
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

// Gradient of the weights to the logits, L lanes per token, slot j on lane j.
// With s^ the renormalized scores and d_j = scale * g_j:
//   renormalize   s_j (dL/ds_j) = s^_j (d_j - sum_i d_i s^_i)
//   else          s_j (dL/ds_j) = s_j d_j
//   sigmoid       dL/dl_j = (1 - s_j) * that, 0 for the other experts
//   softmax       renormalize: dL/dl_j = that (the sum over j is zero), 0 for
//                 the others; else dL/dl_e = that - p_e sum_j p_j d_j
// An id outside [0, E) takes no part; an id that a row holds twice gets both
// slots' gradients, added in slot order.
//
// The slots' values go through a row of LDS that is zero elsewhere: it is
// read in pieces of V experts, stored, and cleared again at the slots alone.
// Bound by the stores of [M, E] (non-temporal: 65536 x 512 in 33 us, 44 with
// plain stores, which push the logits' lines out) and by the lines that the
// top_k gathered logits bring in.
template <int L, int V>
__global__ __launch_bounds__(64 * kSelWaves) void select_backward_kernel(
    SelectParams a, const float* __restrict__ grad_weights, float* __restrict__ grad_logits) {
  constexpr int T = 64 / L;
  __shared__ __attribute__((aligned(16))) float s_row[kSelWaves][T][kSelMaxE];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int li = lane % L, base = lane - li;
  const int E = a.E, k = a.top_k;
  const bool sigmoid = a.sigmoid != 0, dense = !sigmoid && !a.renormalize;
  float* r = s_row[w][lane / L];
  for (int e = li; e < E; e += L) r[e] = 0.f;
  __builtin_amdgcn_wave_barrier();
  const int step = (int)gridDim.x * kSelWaves * T;
#pragma unroll 1
  for (int t0 = ((int)blockIdx.x * kSelWaves + w) * T; t0 < a.M; t0 += step) {
    const bool live = t0 + lane / L < a.M;
    const int t = live ? t0 + lane / L : a.M - 1;
    const float* row = a.logits + (size_t)t * E;
    int id = -1;
    float d = 0.f;
    if (li < k) {
      id = a.ids[(size_t)t * k + li];
      d = a.scale * grad_weights[(size_t)t * k + li];
    }
    const bool used = id >= 0 && id < E;
    const float l = used ? row[id] : -INFINITY;
    if (!used) d = 0.f;
    float mx = -INFINITY, rz = 0.f;
    if (dense) {
      // maximum, then sum of exponentials of the row (from the cache)
      float z = 0.f;
#pragma unroll 4
      for (int e = V * li; e < E; e += V * L) {
        if constexpr (V == 4) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(row + e);
          mx = fmaxf(mx, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
        } else {
          mx = fmaxf(mx, row[e]);
        }
      }
      mx = lanes_max<L>(mx);
#pragma unroll 4
      for (int e = V * li; e < E; e += V * L) {
        if constexpr (V == 4) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(row + e);
          z += (hw_exp(x[0] - mx) + hw_exp(x[1] - mx)) + (hw_exp(x[2] - mx) + hw_exp(x[3] - mx));
        } else {
          z += hw_exp(row[e] - mx);
        }
      }
      z = lanes_sum<L>(z);
      rz = mx == -INFINITY ? 0.f : __builtin_amdgcn_rcpf(z);
      if (mx == -INFINITY) mx = 0.f;
    }
    float g;
    if (a.renormalize) {
      const float m = lanes_max<L>(l);
      // no logit above -inf: 0, NaN for NaN
      const float none = l != l ? l : 0.f;
      const float sh = !used ? 0.f : m > -INFINITY
                           ? fast_score(l, sigmoid ? fminf(m, 0.f) : m, sigmoid) : none;
      const float total = lanes_sum<L>(sh);
      // a true quotient: one weight alone is 1 and its gradient exactly 0
      const float hat = total == 0.f ? 0.f : sh / total;
      g = hat * (d - lanes_sum<L>(hat * d));
    } else if (sigmoid) {
      g = hw_sigmoid(l) * d;
    } else {
      g = hw_exp(l - mx) * rz * d;
    }
    if (sigmoid) g *= hw_sigmoid(-l);
    if (!used) g = 0.f;
    const float all = dense ? lanes_sum<L>(g) : 0.f;
    // a slot that finds another's mark shares its id
    if (used) r[id] = __int_as_float(li);
    __builtin_amdgcn_wave_barrier();
    const bool shared = used && __float_as_int(r[id]) != li;
    if (__any(shared)) {
      float sum = 0.f;
      for (int j = 0; j < k; ++j) {
        const int oj = __shfl(id, base + j, kWave);
        const float gj = __shfl(g, base + j, kWave);
        if (oj == id) sum += gj;
      }
      g = sum;
    }
    __builtin_amdgcn_wave_barrier();
    if (used) r[id] = g;
    __builtin_amdgcn_wave_barrier();
    float* out = grad_logits + (size_t)t * E;
    if (live) {
#pragma unroll 4
      for (int e = V * li; e < E; e += V * L) {
        if constexpr (V == 4) {
          f32x4 v = *reinterpret_cast<const f32x4*>(r + e);
          if (dense) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] -= hw_exp(x[j] - mx) * rz * all;
          }
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(out + e));
        } else {
          out[e] = dense ? r[e] - hw_exp(row[e] - mx) * rz * all : r[e];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (used) r[id] = 0.f;
    __builtin_amdgcn_wave_barrier();
  }
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
  // waves of a large batch take several turns: two rounds of the workgroups
  // that a CU holds (five; three with 32 experts a lane).  Eight for all took
  // 50.7 us where this takes 47.2 (65536 x 512), 17.4 against 15.9 (65536 x 128)
  const int wgs = ceil_div_host(a.M, per), most = (C == 32 ? 6 : 10) * device_cu_count();
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
  // Sixteen lanes a token where a lane has at most four experts, or where the
  // batch fills the chip all the same; else 32, as far as the lane maxima
  // bound top_k well.  Measured us, 16 / 32 / 64 lanes: 60 experts, 4096
  // tokens 4.7 / 5.2 / 6.9; 128 experts, 1024 tokens 5.1 / 4.5 / 4.8, 65536
  // 16.8 / 26.1 / 54.2; 512 experts, 8192 tokens 11.6 / 9.9 / 13.1, 65536
  // 47.5 / 48.8 / 78.5; 256 experts in 8 groups, 64 tokens 8.8 / 6.0 / 6.5,
  // 65536 40 / 49 / 97; 256 experts, top_k 16, 65536 tokens 77 / 39 / 67.
  auto bounds = [&](int lanes) {
    // else every expert of the groups that stay is a candidate
    return lanes / G * a.topk_group >= a.top_k || a.topk_group * gs <= kSelCands;
  };
  const int n16 = per_lane(16, V, G, gs);
  int L = 64;
  if (a.top_k <= 12 && n16 <= 32 && bounds(16) &&
      (n16 <= 4 || a.M > 4 * device_cu_count() * n16)) L = 16;
  else if (a.top_k <= 26 && per_lane(32, V, G, gs) <= 16 && bounds(32)) L = 32;
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

namespace {

template <int L, int V>
hipError_t go_backward(const SelectArgs& a, const float* grad_weights, float* grad_logits,
                       hipStream_t s) {
  const SelectParams p{a.logits, nullptr, a.M, a.E, a.top_k, a.sigmoid, a.renormalize, a.n_group,
                       a.topk_group, a.group_top, a.scale, a.topk_ids, nullptr};
  const int wgs = ceil_div_host(a.M, kSelWaves * 64 / L), most = 8 * device_cu_count();
  hipLaunchKernelGGL((select_backward_kernel<L, V>), dim3(wgs < most ? wgs : most),
                     dim3(64 * kSelWaves), 0, s, p, grad_weights, grad_logits);
  return hipGetLastError();
}

template <int V>
hipError_t launch_backward_v(const SelectArgs& a, const float* grad_weights, float* grad_logits,
                             hipStream_t s) {
  // As launch_select.  Measured us, 16 / 32 lanes a token: 60 experts, 8192
  // tokens 3.5 / 3.9; 128 experts, 1024 tokens 3.7 / 3.3, 16384 4.2 / 4.8; 512
  // experts, 8192 tokens 5.8 / 5.5, 65536 34 / 38.  With a gradient for every
  // logit, 128 experts, 65536 tokens 17.4 / 14.9.  (64 lanes: 512 experts, 1024
  // tokens 3.4 against 3.5 with 32, 65536 tokens 41.)
  const bool dense = !a.sigmoid && !a.renormalize;
  const bool many = a.M > 4 * device_cu_count() * ceil_div_host(a.E, 16);
  if (a.top_k <= 16 && (a.E <= 64 || (!dense && many)))
    return go_backward<16, V>(a, grad_weights, grad_logits, s);
  return go_backward<32, V>(a, grad_weights, grad_logits, s);
}

}  // namespace

hipError_t launch_select_backward(const SelectArgs& a, const float* grad_weights,
                                  float* grad_logits, hipStream_t s) {
  return a.E % 4 == 0 ? launch_backward_v<4>(a, grad_weights, grad_logits, s)
                      : launch_backward_v<1>(a, grad_weights, grad_logits, s);
}

}  // namespace moe_host
