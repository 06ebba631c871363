// Token log probabilities over rows of logits l[0 .. V):
//   m = max l,  z = sum e^(l - m),  lse = m + log z
//   logprob of a token = l[token] - lse
//   entropy = log z - sum (l - m) e^(l - m) / z
//   the `top` largest logits, in descending order, ties to the lower id
// and the gradient of the first two with respect to the logits.
//
// Differences l - m are formed before anything is multiplied, so that a row
// of the type's lowest value (a mask) is as exact as any other; sums are fp32,
// of one register's logits first, then of lanes, waves and chunks in a fixed
// order (bitwise repeatable).
#include <algorithm>

#include "dense.h"

using namespace moe;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 64;      // the join keeps one chunk's list per lane
constexpr int kFill = 512;          // workgroups that fill the chip
constexpr int kMaxCand = 512;       // candidates of a chunk that are ranked in LDS

typedef unsigned long long u64;

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

__device__ __forceinline__ u64 wave_max64(u64 v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const u64 o = __shfl_xor(v, d, kWave);
    v = o > v ? o : v;
  }
  return v;
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

// What a chunk of a row leaves for the row's join.
struct Partial {
  float m;       // largest logit (NaN aside)
  float z, s;    // sums of e = 2^y and y e, y = (l - m) log2 e (m = -inf: of l)
  float pad;
};
__host__ __device__ inline size_t partial_stride(int top) {
  return sizeof(Partial) + (size_t)((top + 1) & ~1) * 8;
}

// ---- one chunk of a row: kThreads * kLoads blocks, held in registers ----
template <bool kBf16, int kLoads, bool kTop>
__global__ __launch_bounds__(kThreads) void logprob_chunk_kernel(moe_host::LogprobArgs a,
                                                                 int chunks) {
  constexpr int kPer = Row<kBf16>::kPer;
  __shared__ float s_m[kWaves], s_z[kWaves], s_s[kWaves], s_t[kWaves];
  __shared__ u64 s_cand[kMaxCand];
  __shared__ u64 s_best[kWaves];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const Row<kBf16> row(a.logits, a.M, a.V, m);
  const int b0 = c * kThreads * kLoads;

  u32x4 w[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int b = b0 + i * kThreads + tid;
    w[i] = u32x4{0u, 0u, 0u, 0u};
    if (b < row.blocks) w[i] = row.load(b);
  }
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int b = b0 + i * kThreads + tid;
    if (!row.whole(b)) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = row.first(b) + j;
        if (e < 0 || e >= a.V) drop<kBf16>(w[i], j);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) mx = fmaxf(mx, element<kBf16>(w[i], j));
  }
  const float wmx = wave_max(mx);
  if (lane == 0) s_m[wave] = wmx;
  if (kTop) {
    // the top-th largest of the wave's lane maxima bounds the row's from below
    const uint32_t key = topk_detail::order_key(mx);
    const uint32_t k1[1] = {key};
    uint32_t T = 0u;
#pragma unroll
    for (int bit = 31; bit >= (kBf16 ? 16 : 0); --bit) {
      const uint32_t t = T | (1u << bit);
      if (topk_detail::count_ge(k1, t) >= a.top) T = t;
    }
    // bf16: the low 16 key bits are all 0 (positive) or all 1 (negative)
    if (kBf16 && !(T & 0x80000000u)) T |= 0xFFFFu;
    if (lane == 0) s_t[wave] = T >= 0x007fffffu ? topk_detail::key_logit(T) : -INFINITY;
    if (tid == 0) s_count = 0;
  }
  __syncthreads();
  float M = s_m[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) M = fmaxf(M, s_m[i]);
  const float from = M == -INFINITY ? 0.f : M;

  float z = 0.f, s = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float y = (element<kBf16>(w[i], j) - from) * kLog2e;
      const float e = __builtin_amdgcn_exp2f(y);
      z += e;
      s = __builtin_fmaf(fmaxf(y, -200.f), e, s);   // -inf * 0 is 0 here
    }
  z = wave_sum(z);
  s = wave_sum(s);
  if (lane == 0) {
    s_z[wave] = z;
    s_s[wave] = s;
  }

  uint8_t* part = static_cast<uint8_t*>(a.partial) + (size_t)blockIdx.x * partial_stride(a.top);
  u64* list = reinterpret_cast<u64*>(part + sizeof(Partial));
  if (kTop) {
    float T = s_t[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) T = fmaxf(T, s_t[i]);
    if (mx >= T && T > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float v = element<kBf16>(w[i], j);
          if (v >= T) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kMaxCand)
              s_cand[at] = order_of(v, row.first(b0 + i * kThreads + tid) + j);
          }
        }
    }
    __syncthreads();
    const int n = s_count;
    if (T > -INFINITY && n >= a.top && n <= kMaxCand) {
      // ranks among the candidates (their order in the list does not matter)
      for (int q = tid; q < n; q += kThreads) {
        const u64 o = s_cand[q];
        int r = 0;
        for (int i = 0; i < n; ++i) r += s_cand[i] > o;
        if (r < a.top) list[r] = o;
      }
    } else {
      // many equal logits, or few at all: the next largest, one after another
      u64 last = ~0ull;
      for (int k = 0; k < a.top; ++k) {
        u64 best = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int e = row.first(b0 + i * kThreads + tid) + j;
            const u64 o = e >= 0 && e < a.V ? order_of(element<kBf16>(w[i], j), e) : 0ull;
            if (o < last && o > best) best = o;
          }
        best = wave_max64(best);
        if (lane == 0) s_best[wave] = best;
        __syncthreads();
        best = s_best[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) best = s_best[i] > best ? s_best[i] : best;
        __syncthreads();
        if (tid == 0) list[k] = best;
        last = best;
      }
    }
  } else {
    __syncthreads();
  }
  if (tid == 0) {
    float zs = s_z[0], ss = s_s[0];
    for (int i = 1; i < kWaves; ++i) {
      zs += s_z[i];
      ss += s_s[i];
    }
    *reinterpret_cast<Partial*>(part) = Partial{M, zs, ss, 0.f};
  }
}

// ---- a row's chunks joined: one wave a row, lane c holding chunk c ----
__global__ __launch_bounds__(64) void logprob_join_kernel(moe_host::LogprobArgs a, int chunks) {
  const int m = blockIdx.x, lane = threadIdx.x;
  const size_t stride = partial_stride(a.top);
  const uint8_t* part = static_cast<const uint8_t*>(a.partial) + ((size_t)m * chunks + lane) * stride;
  Partial p{-INFINITY, 0.f, 0.f, 0.f};
  if (lane < chunks) p = *reinterpret_cast<const Partial*>(part);
  const float M = wave_max(p.m);
  // a chunk without a logit above -inf adds 0 (or its NaN) as it is
  const float d = p.m == -INFINITY ? 0.f : (p.m - M) * kLog2e;
  const float f = __builtin_amdgcn_exp2f(d);
  // a chunk far below the row's largest logit adds nothing
  const float z = wave_sum(p.z * f);
  const float s = wave_sum(f > 0.f ? f * __builtin_fmaf(d, p.z, p.s) : 0.f * p.z);
  // no logit above -inf: nothing is likely, nothing uncertain
  const bool none = z == 0.f;
  const float lz = logf(z);
  auto logprob = [&](float l) {
    if (none) return -INFINITY;
    return l - M - lz;
  };
  if (lane == 0) {
    const int t = a.tokens[m];
    float lp = 0.f;
    if (t >= 0 && t < a.V) {
      const size_t at = (size_t)m * a.V + t;
      const float l = a.bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[at]
                                               << 16)
                             : static_cast<const float*>(a.logits)[at];
      lp = logprob(l);
    }
    a.logprobs[m] = lp;
    a.entropy[m] = none ? 0.f : lz - kLn2 * (s / z);
    a.lse[m] = none ? -INFINITY : M + lz;
  }
  // the lists' heads, one a lane; the largest is the next alternative
  const u64* list = reinterpret_cast<const u64*>(part + sizeof(Partial));
  u64 head = lane < chunks && a.top > 0 ? list[0] : 0ull;
  int at = 0;
  for (int k = 0; k < a.top; ++k) {
    const u64 best = wave_max64(head);
    if (lane == 0) {
      a.top_ids[(size_t)m * a.top + k] = id_of(best);
      a.top_logprobs[(size_t)m * a.top + k] = logprob(logit_of(best));
    }
    if (head == best && lane < chunks) {
      ++at;
      head = at < a.top ? list[at] : 0ull;
    }
  }
}

// Blocks of 16 bytes that a row touches at most, and chunks of `loads` blocks
// a thread.
int row_blocks(int V, int bf16) {
  const int per = bf16 ? 8 : 4;
  return (V + 2 * (per - 1)) / per;
}
int chunks_of(int V, int bf16, int loads) {
  return moe_host::ceil_div_host(row_blocks(V, bf16), kThreads * loads);
}
// Whole registers of logits a thread where the rows fill the chip, else
// smaller chunks, so that more CUs read.
int loads_of(int M, int V, int bf16) {
  int loads = 8;
  while (loads > 1 && (long long)M * chunks_of(V, bf16, loads) < kFill &&
         chunks_of(V, bf16, loads / 2) <= kMaxChunks)
    loads /= 2;
  return loads;
}

template <bool kBf16, bool kTop>
void launch_chunks(const moe_host::LogprobArgs& a, int loads, int chunks, hipStream_t s) {
  const dim3 grid((unsigned)(a.M * chunks));
  switch (loads) {
    case 1: logprob_chunk_kernel<kBf16, 1, kTop><<<grid, kThreads, 0, s>>>(a, chunks); break;
    case 2: logprob_chunk_kernel<kBf16, 2, kTop><<<grid, kThreads, 0, s>>>(a, chunks); break;
    case 4: logprob_chunk_kernel<kBf16, 4, kTop><<<grid, kThreads, 0, s>>>(a, chunks); break;
    default: logprob_chunk_kernel<kBf16, 8, kTop><<<grid, kThreads, 0, s>>>(a, chunks); break;
  }
}

// ---- gradient ----
//
// log p = l - lse; d = -p (g + h (log p + H)), g more at the token.  A row
// whose lse is below kNone has no logit that fp32 can tell from its lse (all
// are -inf or a mask's lowest value): its gradient is 0.
constexpr float kNone = -1e30f;
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
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[m] : 0.f;
  const float H = a.grad_entropy != nullptr ? a.entropy[m] : 0.f;
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

size_t logprob_partial_bytes(int M, int V, int top, int bf16) {
  // halved chunks are fewer than 2 * kFill; so sized, a workspace serves fewer
  // rows as well
  return std::max<size_t>((size_t)M * chunks_of(V, bf16, 8), 2 * kFill) * partial_stride(top);
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  const int loads = loads_of(a.M, a.V, a.bf16), chunks = chunks_of(a.V, a.bf16, loads);
  if (a.bf16)
    a.top > 0 ? launch_chunks<true, true>(a, loads, chunks, s)
              : launch_chunks<true, false>(a, loads, chunks, s);
  else
    a.top > 0 ? launch_chunks<false, true>(a, loads, chunks, s)
              : launch_chunks<false, false>(a, loads, chunks, s);
  logprob_join_kernel<<<a.M, 64, 0, s>>>(a, chunks);
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
