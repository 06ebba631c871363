// Token log probabilities over rows of logits l[0 .. V):
//   m = max l,  z = sum e^(l - m),  lse = m + log z
//   logprob of a token = l[token] - lse
//   entropy = log z - sum (l - m) e^(l - m) / z
//   the `top` largest logits, in descending order, ties to the lower id
// and the gradient of the first two with respect to the logits.
//
// One pass over the logits.  A thread keeps a running anchor (its largest
// logit so far) and forms each exponent as one FMA, y = l log2 e - m2 with
// m2 = fp32(m log2 e); what m2 is off by is taken back from the sums at the
// end.  Sums are fp32: of 16 or 32 logits first, then of a thread's such
// groups, of lanes, waves and chunks, in a fixed order (bitwise repeatable).
// Where a chunk's largest logit lies beyond +-kFar (a mask throughout,
// infinities) that would be too much; its sums are formed again from the
// differences l - m.
//
// Alternatives: a wave collects the logits that reach a threshold in LDS.  The
// threshold is the top-th largest of the lanes' maxima so far (at least `top`
// logits reach it), taken again after 1, 2, 4 ... groups, at first the best of
// the four waves', and rises to the top-th largest so far whenever the list is
// cut back; a logit is looked at singly only in a 16-byte block whose
// maximum reaches the threshold.  Lists that grow are cut by a bitwise search for
// a key that exactly `top` entries reach (wave ballots), equal keys by their ids;
// the last 64 entries or fewer are ranked against each other.
//
// 2048 rows of 131072 bf16 logits: 104 to 108 us without alternatives (5.1 TB/s,
// what a large copy reaches), 110 to 121 with 5, 154 with 20, 184 with 32; of fp32
// 191, 199, 215 and 222 us.  One row 5.4 to 7, 11 to 13, 18 to 19.5 and 21 us, two
// launches and the searches' chains.  From 20 on the lists take vector instructions,
// which 5 alternatives keep busy for 90 % of the time already.  A threshold taken
// from the first group alone: 136 us with 5, 166 with 20.  Without a prefetch a wave
// takes 64 registers and a SIMD holds 8 of them, which hide the loads (4 waves at
// the least: 5 % more).
#include <algorithm>

#include "dense.h"

using namespace moe;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kFar = 16777216.f;  // 2^24: fp32(m log2 e) is off by less than 2
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kLoads = 4;           // 16-byte blocks of a thread's group
constexpr int kGroup = kThreads * kLoads;
constexpr int kMaxTop = 32;
constexpr int kMinWaves = 8;        // waves of a SIMD: 64 registers a wave
constexpr int kMaxChunks = 64;
constexpr int kFill = 2048;         // workgroups that fill the chip: no more chunks than that
constexpr int kKeep = 64;           // a longer list is cut back before it takes more
constexpr int kList = kKeep + 64;
constexpr int kFewLanes = 6;        // with a hit: their logits are dealt out, a lane's at a time

typedef unsigned long long u64;

constexpr uint32_t kLeastKey = 0x007fffffu;   // the order key of -inf

// (ids have kIdBits bits: the low words differ in no others)
constexpr int kIdBits = 19;

// One logit's place in the order: larger logits first, then lower ids.  NaN
// comes after -inf, 0 after everything (no logit).
__device__ __forceinline__ u64 order_of(float v, int id) {
  const uint32_t k = v != v ? 1u : topk_detail::order_key(v);
  return ((u64)k << 32) | (uint32_t)~id;
}
__device__ __forceinline__ int id_of(u64 o) { return (int)~(uint32_t)o; }
__device__ __forceinline__ float logit_of(u64 o) {
  const uint32_t k = (uint32_t)(o >> 32);
  return k == 1u ? __builtin_nanf("") : topk_detail::key_logit(k);
}

// The 16-byte blocks that a row of V elements of a dense [M, V] tensor
// touches: block b holds elements b * kPer - lead ...  Rows need not start on
// a 16-byte border; a block that two rows share belongs to both.
template <bool kBf16>
struct Row {
  static constexpr int kPer = kBf16 ? 8 : 4;
  const uint8_t* base;   // first block
  size_t left;           // elements of the tensor from the first block on
  int lead, V, blocks;
  __device__ __forceinline__ Row(const void* t, size_t M, int V_, int m) : V(V_) {
    const size_t at = (size_t)m * V;
    lead = (int)(at % kPer);
    base = static_cast<const uint8_t*>(t) + (at - lead) * (16 / kPer);
    left = M * V - (at - lead);
    blocks = (lead + V + kPer - 1) / kPer;
  }
  // Block b; only a tensor's very last block can be cut short.
  __device__ __forceinline__ u32x4 load(int b) const {
    if ((size_t)(b + 1) * kPer <= left) return load16(base + (size_t)b * 16);
    u32x4 r = {0u, 0u, 0u, 0u};
    const int n = (int)(left - (size_t)b * kPer);
    for (int j = 0; j < n; ++j) {
      if (kBf16) {
        const uint32_t v = reinterpret_cast<const uint16_t*>(base)[(size_t)b * 8 + j];
        r[j >> 1] |= v << (16 * (j & 1));
      } else {
        r[j] = reinterpret_cast<const uint32_t*>(base)[(size_t)b * 4 + j];
      }
    }
    return r;
  }
  __device__ __forceinline__ int first(int b) const { return b * kPer - lead; }
  __device__ __forceinline__ bool whole(int b) const {
    return first(b) >= 0 && first(b) + kPer <= V;
  }
};

template <bool kBf16>
__device__ __forceinline__ float element(const u32x4& w, int j) {
  if (!kBf16) return __uint_as_float(w[j]);
  return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
}
// -inf in an element's place
template <bool kBf16>
__device__ __forceinline__ void drop(u32x4& w, int j) {
  if (!kBf16)
    w[j] = 0xFF800000u;
  else
    w[j >> 1] = j & 1 ? (w[j >> 1] & 0xFFFFu) | 0xFF800000u : (w[j >> 1] & 0xFFFF0000u) | 0xFF80u;
}

// A key that exactly n of the wave's keys reach, or, where equal keys leave
// none, the largest that at least n reach: T, whose bits kFrom .. kTo are 0,
// and those bits.  `reach`: how many keys reach T, then how many reach the
// result.
template <int kFrom, int kTo, int NB>
__device__ __forceinline__ uint32_t nth_key(const uint32_t (&key)[NB], int n, uint32_t T,
                                            int& reach) {
  for (int bit = kFrom; bit >= kTo && reach != n; --bit) {
    const uint32_t t = T | (1u << bit);
    const int c = topk_detail::count_ge(key, t);
    if (c >= n) {
      T = t;
      reach = c;
    }
  }
  return T;
}

__device__ __forceinline__ void lds_order() {   // of one wave's LDS accesses
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// Keeps the n largest of the wave's entries (0: none), in no order, in `to`;
// returns how many there are.  `least`: a key that they all reach and, if
// `strict`, that later entries (of higher ids) have to pass to replace one;
// at most -inf's key if fewer than n are kept.  kLoose: up to 64 entries that
// reach the n-th largest key are all kept.
template <bool kBf16, bool kLoose, int NB>
__device__ __forceinline__ int cut(const u64 (&o)[NB], u64* to, int n, uint32_t& least,
                                   bool& strict) {
  const int lane = threadIdx.x & 63;
  uint32_t key[NB], low[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    key[i] = (uint32_t)(o[i] >> 32);
    low[i] = (uint32_t)o[i];
  }
  // of bf16 logits the key's upper half decides; the lower one is all 0, or
  // all 1 below 0
  int reach = topk_detail::count_ge(key, 1u);
  uint32_t T = nth_key<31, kBf16 ? 16 : 0>(key, n, 0u, reach);
  uint32_t low_least = 0u;
  strict = reach > n && !(kLoose && reach <= 64);
  if (strict) {
    if (kBf16 && !(T & 0x80000000u)) T |= 0xFFFFu;
    // of the entries that equal T the lower ids, which are the larger low words
    const int above = topk_detail::count_ge(key, T + 1u);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (key[i] != T) low[i] = 0u;
    low_least = nth_key<kIdBits - 1, 0>(low, n - above, ~0u << kIdBits, reach = NB * 64);
  }
  least = max(T, kLeastKey);
  const unsigned long long below = (1ull << lane) - 1ull;
  int at = 0;
  lds_order();
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const bool keep = key[i] >= max(T, 1u) && (!strict || key[i] != T || low[i] >= low_least);
    const unsigned long long m = __ballot(keep);
    if (keep) to[at + __popcll(m & below)] = o[i];
    at += __popcll(m);
  }
  lds_order();
  return at;
}

// The place of an entry among `count` different ones in LDS: 0 for the largest.
__device__ __forceinline__ int rank_of(const u64* list, int count, u64 o) {
  int r = 0;
#pragma unroll 8
  for (int i = 0; i < count; ++i) r += list[i] > o;
  return r;
}

// What a chunk of a row leaves for the row's join, kFill of them at most; then
// the lists, `top` entries a chunk (0: none).
struct Partial {
  float m;       // largest logit (NaN aside)
  float z, s;    // sums of e = 2^y and y e, y = (l - m) log2 e (m = -inf: of l)
  float pad;
};
__host__ __device__ inline u64* lists_of(void* partial) {
  return reinterpret_cast<u64*>(static_cast<uint8_t*>(partial) + kFill * sizeof(Partial));
}

// A logit of a row, and that of its token.
template <bool kBf16>
__device__ __forceinline__ float logit_at(const moe_host::LogprobArgs& a, int m, int v) {
  const size_t at = (size_t)m * a.V + v;
  return kBf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[at] << 16)
               : static_cast<const float*>(a.logits)[at];
}
struct Asked {
  bool is;       // the token is one of the row's
  float l;
};
template <bool kBf16>
__device__ __forceinline__ Asked asked_of(const moe_host::LogprobArgs& a, int m) {
  const int t = a.tokens[m];
  Asked k{t >= 0 && t < a.V, 0.f};
  if (k.is) k.l = logit_at<kBf16>(a, m, t);
  return k;
}

// A row's results, by one wave: its largest logit, sums, and `count` entries in
// LDS (at most 64, in no order) that hold its alternatives.
template <bool kBf16>
__device__ __forceinline__ void finish(const moe_host::LogprobArgs& a, int m, const Asked& asked,
                                       float M, float z, float s, const u64* list, int count) {
  const int lane = threadIdx.x & 63;
  // no logit above -inf: nothing is likely, nothing uncertain
  const bool none = z == 0.f;
  const float lz = logf(z);
  auto logprob = [&](float l) { return none ? -INFINITY : l - M - lz; };
  if (lane == 0) {
    a.logprobs[m] = asked.is ? logprob(asked.l) : 0.f;
    a.entropy[m] = none ? 0.f : lz - kLn2 * (s / z);
    a.lse[m] = none ? -INFINITY : M + lz;
  }
  if (a.top == 0) return;
  const size_t to = (size_t)m * a.top;
  if (lane < count) {
    const u64 o = list[lane];
    const int r = rank_of(list, count, o);
    if (r < a.top) {
      a.top_ids[to + r] = id_of(o);
      a.top_logprobs[to + r] = logprob(logit_of(o));
    }
  }
  // fewer than `top` logits are numbers: NaN follows, by id
  const unsigned long long below = (1ull << lane) - 1ull;
  for (int v0 = 0; v0 < a.V && count < a.top; v0 += 64) {
    const float l = v0 + lane < a.V ? logit_at<kBf16>(a, m, v0 + lane) : 0.f;
    const unsigned long long nan = __ballot(l != l);
    const int at = count + __popcll(nan & below);
    if (l != l && at < a.top) {
      a.top_ids[to + at] = v0 + lane;
      a.top_logprobs[to + at] = __builtin_nanf("");
    }
    count += __popcll(nan);
  }
}

// ---- one chunk of a row ----
template <bool kBf16, bool kTop>
__global__ __launch_bounds__(kThreads, kMinWaves) void logprob_kernel(
    moe_host::LogprobArgs a, int chunks, int chunk_blocks) {
#pragma clang fp contract(off)      // an anchor's product is the rounded one wherever it is used
  constexpr int kPer = Row<kBf16>::kPer;
  __shared__ float s_m[kWaves], s_a[kWaves], s_z[kWaves], s_s[kWaves];
  __shared__ float s_t[kTop ? kWaves : 1];
  __shared__ int s_count[kWaves];
  __shared__ u64 s_list[kTop ? kWaves : 1][kTop ? kList : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const Row<kBf16> row(a.logits, a.M, a.V, m);
  const int b0 = c * chunk_blocks, b1 = min(row.blocks, b0 + chunk_blocks);

  // A wave's group g: 64 kLoads consecutive blocks.  `inner`: all of them are
  // there, whole, and not the tensor's last.
  auto start = [&](int g) { return b0 + (g * kWaves + wave) * (64 * kLoads); };
  auto inner = [&](int g) {
    const int b = start(g);
    return b + 64 * kLoads <= b1 && b + 64 * kLoads < row.blocks && (b > 0 || row.lead == 0);
  };
  auto load = [&](int g, u32x4 (&w)[kLoads]) {
    const int b = start(g) + lane;
    if (inner(g)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) w[i] = load16(row.base + (size_t)(b + 64 * i) * 16);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        w[i] = u32x4{0u, 0u, 0u, 0u};
        if (b + 64 * i < b1) w[i] = row.load(b + 64 * i);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int e = row.first(b + 64 * i) + j;
          if (e < 0 || e >= a.V || b + 64 * i >= b1) drop<kBf16>(w[i], j);
        }
      }
    }
  };
  Asked asked{false, 0.f};
  if (chunks == 1 && wave == 0) asked = asked_of<kBf16>(a, m);
  const int groups = ceil_div(b1 - b0, kGroup);
  float mx = -INFINITY, from = -kFar, m2 = -kFar * kLog2e, z = 0.f, s = 0.f;
  float T = -INFINITY;
  int count = 0;
  u64* list = s_list[kTop ? wave : 0];
  const unsigned long long below = (1ull << lane) - 1ull;
  bool strict = false;
  auto cut_back = [&] {
    uint32_t least;
    u64 o[kList / 64];
    lds_order();
#pragma unroll
    for (int i = 0; i < kList / 64; ++i) o[i] = 64 * i + lane < count ? list[64 * i + lane] : 0ull;
    count = cut<kBf16, false>(o, list, a.top, least, strict);
    if (count == a.top) T = topk_detail::key_logit(least);
  };
  // cut lists raise the threshold: soon where few alternatives are wanted
  const int keep = min(kKeep, 2 * a.top + 32);
  auto push = [&](bool hit, float l, int e) {
    const unsigned long long hits = __ballot(hit);
    if (hits == 0ull) return;
    if (count > keep) cut_back();
    if (hit) list[count + __popcll(hits & below)] = order_of(l, e);
    count += __popcll(hits);
  };
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    u32x4 w[kLoads];
    load(g, w);
    float bm[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      bm[i] = -INFINITY;                               // NaN aside
#pragma unroll
      for (int j = 0; j < kPer; ++j) bm[i] = fmaxf(bm[i], element<kBf16>(w[i], j));
    }
    // (widened again below: 32 fp32 registers fewer)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) asm("" : "+v"(w[i]));
    const float gm = fmaxf(fmaxf(bm[0], bm[1]), fmaxf(bm[2], bm[3]));
    mx = fmaxf(mx, gm);
    from = fmaxf(from, gm);
    const float to = from * kLog2e, d = m2 - to, f = __builtin_amdgcn_exp2f(d);
    m2 = to;
    float gz = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float y = __builtin_fmaf(element<kBf16>(w[i], j), kLog2e, -m2);
        const float e = __builtin_amdgcn_exp2f(y);
        gz += e;
        gs = __builtin_fmaf(fmaxf(y, -200.f), e, gs);   // -inf * 0 is 0 here
      }
    s = __builtin_fmaf(f, __builtin_fmaf(d, z, s), gs);
    z = __builtin_fmaf(f, z, gz);
    if (kTop) {
      if ((g & (g + 1)) == 0) {          // 0, 1, 3, 7, ...
        const uint32_t key[1] = {topk_detail::order_key(mx)};
        int reach = 64;
        const uint32_t k = nth_key<31, kBf16 ? 16 : 0>(key, a.top, 0u, reach);
        T = fmaxf(T, topk_detail::key_logit(max(k, kLeastKey)));
        if (g == 0) {                    // the best of the waves' serves them all
          if (lane == 0) s_t[wave] = T;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kWaves; ++i) T = fmaxf(T, s_t[i]);
        }
      }
      if (__ballot(gm >= T) != 0ull) {
        const bool whole = inner(g);
#pragma unroll 1
        for (int i = 0; i < kLoads; ++i) {
          const float top = i == 0 ? bm[0] : i == 1 ? bm[1] : i == 2 ? bm[2] : bm[3];
          unsigned long long lanes = __ballot(top >= T);
          if (lanes == 0ull) continue;
          const u32x4 v = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
          const int b = start(g) + 64 * i, e = row.first(b + lane);
          if (whole && __popcll(lanes) <= kFewLanes) {
            // one lane's logits at a time, dealt to the first lanes
            const int q = kBf16 ? lane >> 1 : lane;
            for (; lanes != 0ull; lanes &= lanes - 1ull) {
              const int L = __builtin_ctzll(lanes);
              uint32_t x = (uint32_t)__builtin_amdgcn_readlane((int)v[0], L);
#pragma unroll
              for (int k = 1; k < 4; ++k) {
                const uint32_t y = (uint32_t)__builtin_amdgcn_readlane((int)v[k], L);
                x = q == k ? y : x;
              }
              const float l =
                  kBf16 ? (lane & 1 ? bf16_hi(x) : bf16_lo(x)) : __uint_as_float(x);
              push(lane < kPer && l >= T, l, row.first(b + L) + lane);
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < kPer; ++j) {
              const int q = kBf16 ? j >> 1 : j;
              const uint32_t x = q == 0 ? v[0] : q == 1 ? v[1] : q == 2 ? v[2] : v[3];
              const float l = kBf16 ? (j & 1 ? bf16_hi(x) : bf16_lo(x)) : __uint_as_float(x);
              push(l >= T && (whole || (b + lane < b1 && e + j >= 0 && e + j < a.V)), l, e + j);
            }
          }
          // the logits of later blocks have higher ids: an equal one does not count
          if (strict) {
            T = topk_detail::key_logit(topk_detail::order_key(T) + 1u);
            strict = false;
          }
        }
      }
    }
  }
  if (kTop) {
    if (count > kKeep) cut_back();
    lds_order();
    if (lane == 0) s_count[wave] = count;
  }

  const float wm = wave_max(mx), wa = wave_max(from);
  if (lane == 0) {
    s_m[wave] = wm;
    s_a[wave] = wa;
  }
  __syncthreads();
  float M = s_m[0], A = s_a[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    M = fmaxf(M, s_m[i]);
    A = fmaxf(A, s_a[i]);
  }
  if (__builtin_fabsf(M) <= kFar || M == -INFINITY) {
    const float M2 = A * kLog2e, d = m2 - M2, f = __builtin_amdgcn_exp2f(d);
    s = f * __builtin_fmaf(d, z, s);
    z = f * z;
  } else {
    z = s = 0.f;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      u32x4 w[kLoads];
      load(g, w);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float y = (element<kBf16>(w[i], j) - M) * kLog2e;
          const float e = __builtin_amdgcn_exp2f(y);
          z += e;
          s = __builtin_fmaf(fmaxf(y, -200.f), e, s);
        }
    }
    A = M;
  }
  z = wave_sum(z);
  s = wave_sum(s);
  if (lane == 0) {
    s_z[wave] = z;
    s_s[wave] = s;
  }
  __syncthreads();
  if (wave != 0) return;
  z = s_z[0];
  s = s_s[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    z += s_z[i];
    s += s_s[i];
  }
  if (A != M || __builtin_fabsf(M) <= kFar) {
    // to the anchor itself, from fp32(A log2 e)
    const float off = __builtin_fmaf(A, kLog2e, -(A * kLog2e));
    const float f = __builtin_amdgcn_exp2f(-off);
    s = f * __builtin_fmaf(-off, z, s);
    z = f * z;
  }
  int kept = 0;
  if (kTop) {
    // the waves' lists, each at most kKeep long, one after another
    int total = 0, from_wave = 0, from_at = lane;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = s_count[w];
      if (lane >= total + n && w + 1 < kWaves) {
        from_wave = w + 1;
        from_at = lane - total - n;
      }
      total += n;
    }
    if (total <= 64) {
      const u64 o = lane < total ? s_list[kTop ? from_wave : 0][kTop ? from_at : 0] : 0ull;
      lds_order();
      if (lane < total) list[lane] = o;
      lds_order();
      kept = total;
    } else {
      u64 o[kWaves];
      uint32_t least;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        o[w] = lane < s_count[w] ? s_list[kTop ? w : 0][kTop ? lane : 0] : 0ull;
      kept = cut<kBf16, true>(o, list, a.top, least, strict);
    }
  }
  if (chunks == 1) {
    finish<kBf16>(a, m, asked, M, z, s, list, kept);
    return;
  }
  if (lane == 0) static_cast<Partial*>(a.partial)[blockIdx.x] = Partial{M, z, s, 0.f};
  if (kTop) {
    u64* to = lists_of(a.partial) + (size_t)blockIdx.x * a.top;
    if (lane < kept) {
      const u64 o = list[lane];
      const int r = rank_of(list, kept, o);
      if (r < a.top) to[r] = o;
    } else if (lane < a.top) {
      to[lane] = 0ull;
    }
  }
}

// ---- a row's chunks joined: one wave a row, lane c holding chunk c's sums ----
template <bool kBf16, int NB>
__global__ __launch_bounds__(64) void logprob_join_kernel(moe_host::LogprobArgs a, int chunks) {
  __shared__ u64 s_list[64];
  const int m = blockIdx.x, lane = threadIdx.x;
  const Asked asked = asked_of<kBf16>(a, m);
  Partial p{-INFINITY, 0.f, 0.f, 0.f};
  if (lane < chunks) p = static_cast<const Partial*>(a.partial)[(size_t)m * chunks + lane];
  int kept = 0;
  if (NB > 0) {
    u64 o[NB > 0 ? NB : 1];
    const int all = chunks * a.top;
    const u64* lists = lists_of(a.partial) + (size_t)m * all;
#pragma unroll
    for (int i = 0; i < NB; ++i) o[i] = i * 64 + lane < all ? lists[i * 64 + lane] : 0ull;
    uint32_t least;
    bool strict;
    kept = cut<kBf16, true>(o, s_list, a.top, least, strict);
  }
  const float M = wave_max(p.m);
  // a chunk without a logit above -inf adds 0 (or its NaN) as it is, one far
  // below the row's largest logit nothing
  const float d = p.m == -INFINITY ? 0.f : (p.m - M) * kLog2e;
  const float f = __builtin_amdgcn_exp2f(d);
  const float z = wave_sum(p.z * f);
  const float s = wave_sum(f > 0.f ? f * __builtin_fmaf(d, p.z, p.s) : 0.f * p.z);
  finish<kBf16>(a, m, asked, M, z, s, s_list, kept);
}

// Blocks of 16 bytes that a row touches at most, and the length of a chunk:
// whole groups of a workgroup's loads, as many chunks as fill the chip.
int row_blocks(int V, int bf16) {
  const int per = bf16 ? 8 : 4;
  return V % per == 0 ? V / per : (V + 2 * (per - 1)) / per;
}
int chunk_blocks_of(int M, int V, int bf16) {
  const int groups = moe_host::ceil_div_host(row_blocks(V, bf16), kGroup);
  const int want = std::min(kMaxChunks, std::max(1, kFill / std::max(M, 1)));
  return moe_host::ceil_div_host(groups, want) * kGroup;
}
int chunks_of(int M, int V, int bf16) {
  return moe_host::ceil_div_host(row_blocks(V, bf16), chunk_blocks_of(M, V, bf16));
}

template <bool kBf16>
void launch_rows(const moe_host::LogprobArgs& a, hipStream_t s) {
  const int length = chunk_blocks_of(a.M, a.V, a.bf16), chunks = chunks_of(a.M, a.V, a.bf16);
  const unsigned grid = (unsigned)a.M * chunks;
  if (a.top > 0)
    logprob_kernel<kBf16, true><<<grid, kThreads, 0, s>>>(a, chunks, length);
  else
    logprob_kernel<kBf16, false><<<grid, kThreads, 0, s>>>(a, chunks, length);
  if (chunks == 1) return;
  const int lists = chunks * a.top;
  if (lists == 0)
    logprob_join_kernel<kBf16, 0><<<a.M, 64, 0, s>>>(a, chunks);
  else if (lists <= 256)
    logprob_join_kernel<kBf16, 4><<<a.M, 64, 0, s>>>(a, chunks);
  else if (lists <= 768)
    logprob_join_kernel<kBf16, 12><<<a.M, 64, 0, s>>>(a, chunks);
  else
    logprob_join_kernel<kBf16, kMaxChunks * kMaxTop / 64><<<a.M, 64, 0, s>>>(a, chunks);
}

// ---- gradient ----
//
// log p = l - lse; d = -p (g + h (log p + H)), g more at the token.  A row
// whose lse is below kNone is ruled out from end to end (by -inf, the type's
// lowest value or -1e9): fp32's step there is 2 or more, lse does not tell how
// many logits share it, and p would be 1 for each of them.  Its gradient is 0.
constexpr float kNone = -kFar;
constexpr int kGradLoads = 4;       // blocks a thread

template <bool kBf16>
__global__ __launch_bounds__(256) void logprob_backward_kernel(moe_host::LogprobGradArgs a,
                                                               int chunks) {
  constexpr int kPer = Row<kBf16>::kPer;
  const int m = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const Row<kBf16> row(a.logits, a.M, a.V, m);
  uint8_t* out = static_cast<uint8_t*>(a.grad_logits) +
                 (row.base - static_cast<const uint8_t*>(a.logits));
  const int t = a.tokens[m];
  const float lse = a.lse[m];
  const bool none = lse < kNone;
  const float g = t >= 0 && t < a.V && !none ? a.grad_logprobs[m] : 0.f;
  const float h = a.grad_entropy != nullptr && !none ? a.grad_entropy[m] : 0.f;
  const float H = a.grad_entropy != nullptr && !none ? a.entropy[m] : 0.f;
  u32x4 w[kGradLoads];
#pragma unroll
  for (int i = 0; i < kGradLoads; ++i) {
    const int b = (c * kGradLoads + i) * 256 + (int)threadIdx.x;
    w[i] = u32x4{0u, 0u, 0u, 0u};
    if (b < row.blocks) w[i] = row.load(b);
  }
#pragma unroll
  for (int i = 0; i < kGradLoads; ++i) {
    const int b = (c * kGradLoads + i) * 256 + (int)threadIdx.x;
    if (b >= row.blocks) continue;
    float d[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float lp = element<kBf16>(w[i], j) - lse;
      const float p = none ? 0.f : __builtin_amdgcn_exp2f(lp * kLog2e);
      // -inf * 0 is 0 here: a token ruled out has no gradient
      const float inner = __builtin_fmaf(h, fmaxf(lp, -200.f) + H, g);
      d[j] = -p * inner + (row.first(b) + j == t ? g : 0.f);
    }
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = kBf16 ? pack_bf16x2(d[(2 * j) % kPer], d[(2 * j + 1) % kPer])
                   : __float_as_uint(d[j % kPer]);
    if (row.whole(b)) {
      *reinterpret_cast<u32x4*>(out + (size_t)b * 16) = o;
    } else {
      for (int j = 0; j < kPer; ++j) {
        const int e = row.first(b) + j;
        if (e < 0 || e >= a.V) continue;
        if (kBf16)
          reinterpret_cast<uint16_t*>(out)[(size_t)b * 8 + j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
        else
          reinterpret_cast<uint32_t*>(out)[(size_t)b * 4 + j] = o[j % 4];
      }
    }
  }
}

}  // namespace

namespace moe_host {

size_t logprob_partial_bytes(int top) {
  return (size_t)kFill * (sizeof(Partial) + (size_t)top * sizeof(u64));
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.bf16)
    launch_rows<true>(a, s);
  else
    launch_rows<false>(a, s);
  return hipGetLastError();
}

hipError_t launch_token_logprobs_backward(const LogprobGradArgs& a, hipStream_t s) {
  const int chunks = ceil_div_host(row_blocks(a.V, a.bf16), 256 * kGradLoads);
  const unsigned grid = (unsigned)(a.M * chunks);
  if (a.bf16)
    logprob_backward_kernel<true><<<grid, 256, 0, s>>>(a, chunks);
  else
    logprob_backward_kernel<false><<<grid, 256, 0, s>>>(a, chunks);
  return hipGetLastError();
}

}  // namespace moe_host
