// Low-rank adapters of many requests beside a shared projection:
//   y[m] = addend[m] + scale[s] (x[m] A_s^T) B_s^T,   s = slots[m]
//   out = bf16(y), or with `gated` SiLU(first half of y) * second half
// A_s [R, K], B_s [N, R]; a token whose slot is outside [0, S) has no adapter.
//
// Two steps, t = scale (x A^T) and y = addend + t B^T.  Few tokens: each reads
// its adapter by itself (GEMVs, t in fp32).  More: tokens are grouped by slot
// first (a counting sort; the groups' order does not reach any sum), 64 to a
// unit, and both steps run on the matrix cores; t is kept as the sum of two
// bf16 numbers, so that it loses less than 2^-16 of itself.
#include <algorithm>

#include "dense.h"

using namespace moe;
using moe_host::AdapterArgs;

namespace {

constexpr int kUnit = 64;              // tokens of a unit at most
constexpr int kWindow = 8192;          // tokens that one workgroup groups
constexpr int kPlanThreads = 1024;
constexpr int kPlanTokens = kWindow / kPlanThreads;
constexpr int kMaxSlots = 4096;
constexpr int kMaxRank = 128;

struct Unit {
  int slot;      // S: no adapter
  int start;     // place of the first token in the order by slot
  int count;     // tokens; 0: no unit
  int pad;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// ---- few tokens ----

// t[m, r] = scale x[m] . A_s[r]: one wave for kR rows of A_s
template <int kR>
__global__ __launch_bounds__(256) void shrink_gemv_kernel(AdapterArgs a, float* __restrict__ t) {
  const int lane = threadIdx.x & 63;
  const int groups = a.R / kR;
  const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int m = w / groups, r0 = w % groups * kR;
  if (m >= a.M) return;
  const int s = a.slots[m];
  if (s < 0 || s >= a.S) return;
  const uint16_t* x = a.x + (size_t)m * a.K;
  const uint16_t* A = a.a + ((size_t)s * a.R + r0) * a.K;
  float sum[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) sum[r] = 0.f;
#pragma unroll 4
  for (int k = lane * 8; k < a.K; k += 512) {
    const u32x4 xv = load16(x + k);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const u32x4 av = load16(A + (size_t)r * a.K + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[r] = __builtin_fmaf(bf16_lo(xv[j]), bf16_lo(av[j]), sum[r]);
        sum[r] = __builtin_fmaf(bf16_hi(xv[j]), bf16_hi(av[j]), sum[r]);
      }
    }
  }
  const float scale = a.scales != nullptr ? a.scales[s] : 1.f;
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const float v = wave_sum(sum[r]);
    if (lane == 0) t[(size_t)m * a.R + r0 + r] = v * scale;
  }
}

// y of one token, one column a thread
template <bool kGated>
__global__ __launch_bounds__(256) void expand_gemv_kernel(AdapterArgs a,
                                                          const float* __restrict__ t) {
  const int n_out = kGated ? a.N / 2 : a.N;
  const int m = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= n_out) return;
  const int s = a.slots[m];
  float y[2] = {0.f, 0.f};
  if (s >= 0 && s < a.S) {
    const float* tm = t + (size_t)m * a.R;
#pragma unroll
    for (int h = 0; h < (kGated ? 2 : 1); ++h) {
      const uint16_t* b = a.b + ((size_t)s * a.N + n + h * n_out) * a.R;
#pragma unroll 4
      for (int r = 0; r < a.R; r += 8) {
        const u32x4 v = load16(b + r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[h] = __builtin_fmaf(tm[r + 2 * j], bf16_lo(v[j]), y[h]);
          y[h] = __builtin_fmaf(tm[r + 2 * j + 1], bf16_hi(v[j]), y[h]);
        }
      }
    }
  }
  if (a.addend != nullptr) {
    const uint16_t* p = a.addend + (size_t)m * a.N + n;
    y[0] += bf16_at(p);
    if (kGated) y[1] += bf16_at(p + n_out);
  }
  a.out[(size_t)m * n_out + n] = (uint16_t)f32_to_bf16(kGated ? silu_mul(y[0], y[1]) : y[0]);
}

// Both steps in one launch, with the same sums: each workgroup of 256 columns forms t by itself, B's
// first rows on their way meanwhile.
template <bool kGated>
__global__ __launch_bounds__(256) void adapters_gemv_kernel(AdapterArgs a) {
  constexpr int kHalves = kGated ? 2 : 1, kAhead = 4;
  __shared__ __attribute__((aligned(16))) float s_t[kMaxRank];
  const int n_out = kGated ? a.N / 2 : a.N;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  const int s = a.slots[m];
  float y[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) y[h] = 0.f;
  if (s >= 0 && s < a.S) {
    const uint16_t* b[kHalves];
    u32x4 first[kHalves][kAhead];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      b[h] = a.b + ((size_t)s * a.N + min(n, n_out - 1) + h * n_out) * a.R;
#pragma unroll
      for (int q = 0; q < kAhead; ++q) first[h][q] = load16_or_zero(b[h] + 8 * q, 8 * q < a.R);
    }
    const uint16_t* x = a.x + (size_t)m * a.K;
    const float scale = a.scales != nullptr ? a.scales[s] : 1.f;
    for (int r0 = wave * 4; r0 < a.R; r0 += 16) {
      const uint16_t* A = a.a + ((size_t)s * a.R + r0) * a.K;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int k = lane * 8; k < a.K; k += 512) {
        const u32x4 xv = load16(x + k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const u32x4 av = load16(A + (size_t)r * a.K + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum[r] = __builtin_fmaf(bf16_lo(xv[j]), bf16_lo(av[j]), sum[r]);
            sum[r] = __builtin_fmaf(bf16_hi(xv[j]), bf16_hi(av[j]), sum[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = wave_sum(sum[r]);
        if (lane == 0) s_t[r0 + r] = v * scale;
      }
    }
    __syncthreads();
    auto add = [&](int h, const u32x4& v, int r) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[h] = __builtin_fmaf(s_t[r + 2 * j], bf16_lo(v[j]), y[h]);
        y[h] = __builtin_fmaf(s_t[r + 2 * j + 1], bf16_hi(v[j]), y[h]);
      }
    };
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (8 * q < a.R) add(h, first[h][q], 8 * q);
      for (int r = 8 * kAhead; r < a.R; r += 8) add(h, load16(b[h] + r), r);
    }
  }
  if (n >= n_out) return;
  if (a.addend != nullptr) {
    const uint16_t* p = a.addend + (size_t)m * a.N + n;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) y[h] += bf16_at(p + h * n_out);
  }
  a.out[(size_t)m * n_out + n] =
      (uint16_t)f32_to_bf16(kGated ? silu_mul(y[0], y[kHalves - 1]) : y[0]);
}

// ---- tokens grouped by slot ----

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, kWave);
    if (lane >= d) v += o;
  }
  return v;
}

// Window blockIdx.x of kWindow tokens: order[place] = token, by slot, and the
// window's units (`cap` records, the last ones empty).
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(AdapterArgs a, int* __restrict__ order,
                                                            Unit* __restrict__ units, int cap) {
  __shared__ int s_count[kMaxSlots + 1], s_place[kMaxSlots + 1];
  __shared__ int s_wave[2][kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int base = blockIdx.x * kWindow, here = min(kWindow, a.M - base);
  const int bins = a.S + 1;
  for (int i = tid; i < bins; i += kPlanThreads) s_count[i] = 0;
  __syncthreads();
  int slot[kPlanTokens], rank[kPlanTokens];
#pragma unroll
  for (int i = 0; i < kPlanTokens; ++i) {
    const int at = i * kPlanThreads + tid;
    slot[i] = -1;
    if (at < here) {
      const int s = a.slots[base + at];
      slot[i] = s < 0 || s >= a.S ? a.S : s;
    }
  }
#pragma unroll
  for (int i = 0; i < kPlanTokens; ++i) {
    rank[i] = 0;
    if (i * kPlanThreads >= here) break;
    const int first = __builtin_amdgcn_readfirstlane(slot[i]);
    if (__ballot(slot[i] == first) == ~0ull && first >= 0) {
      int old = 0;
      if (lane == 0) old = atomicAdd(&s_count[first], 64);
      rank[i] = __builtin_amdgcn_readfirstlane(old) + lane;
    } else if (slot[i] >= 0) {
      rank[i] = atomicAdd(&s_count[slot[i]], 1);
    }
  }
  __syncthreads();
  // exclusive sums over the bins of tokens and units; a thread has `per` bins
  const int per = (bins + kPlanThreads - 1) / kPlanThreads;
  int tokens = 0, unit = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    const int c = b < bins ? s_count[b] : 0;
    tokens += c;
    unit += (c + kUnit - 1) / kUnit;
  }
  const int in_t = wave_scan(tokens, lane), in_u = wave_scan(unit, lane);
  if (lane == 63) {
    s_wave[0][wave] = in_t;
    s_wave[1][wave] = in_u;
  }
  __syncthreads();
  int t0 = in_t - tokens, u0 = in_u - unit, total = 0;
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    if (i < wave) {
      t0 += s_wave[0][i];
      u0 += s_wave[1][i];
    }
    total += s_wave[1][i];
  }
  units += (size_t)blockIdx.x * cap;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= bins) break;
    const int c = s_count[b];
    s_place[b] = t0;
    for (int q = 0; q < c; q += kUnit) units[u0++] = Unit{b, base + t0 + q, min(kUnit, c - q), 0};
    t0 += c;
  }
  for (int i = total + tid; i < cap; i += kPlanThreads) units[i] = Unit{0, 0, 0, 0};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanTokens; ++i)
    if (slot[i] >= 0) order[base + s_place[slot[i]] + rank[i]] = base + i * kPlanThreads + tid;
}

// t of 16 FT tokens of a unit (blockIdx.x: unit, part): eight waves, an eighth
// of K each, summed through LDS in wave order.  t[place] holds R high parts,
// then R low parts.
template <int FR, int FT>
__global__ __launch_bounds__(512) void shrink_kernel(AdapterArgs a, const int* __restrict__ order,
                                                     const Unit* __restrict__ units,
                                                     uint16_t* __restrict__ t) {
  __shared__ f32x4 red[8][FT * FR][64];
  constexpr int kParts = kUnit / (16 * FT);
  const Unit u = units[blockIdx.x / kParts];
  const int q = blockIdx.x % kParts * 16 * FT, n = u.count - q;
  if (n <= 0 || u.slot >= a.S) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int steps = ceil_div(a.K, 32), per = ceil_div(steps, 8);
  const int first = wave * per, last = min(steps, first + per);
  const uint16_t *x[FT], *A[FR];
#pragma unroll
  for (int j = 0; j < FT; ++j)
    x[j] = a.x + (size_t)order[u.start + q + min(16 * j + i, n - 1)] * a.K + 8 * g;
#pragma unroll
  for (int f = 0; f < FR; ++f)
    A[f] = a.a + ((size_t)u.slot * a.R + min(f * 16 + i, a.R - 1)) * a.K + 8 * g;
  f32x4 acc[FT][FR];
#pragma unroll
  for (int j = 0; j < FT; ++j)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  // kBatch steps at a time, all their loads in flight at once; past the end of
  // K zeros
  constexpr int kBatch = FR <= 4 ? 4 : 2;
  for (int k = first; k < last; k += kBatch) {
    u32x4 xv[kBatch][FT], av[kBatch][FR];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool ok = k + b < last && (k + b) * 32 + 8 * g < a.K;
#pragma unroll
      for (int j = 0; j < FT; ++j) xv[b][j] = load16_or_zero(x[j] + (k + b) * 32, ok);
#pragma unroll
      for (int f = 0; f < FR; ++f) av[b][f] = load16_or_zero(A[f] + (k + b) * 32, ok);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[j][f] = mfma_16x16x32(av[b][f], xv[b][j], acc[j][f]);
  }
#pragma unroll
  for (int j = 0; j < FT; ++j)
#pragma unroll
    for (int f = 0; f < FR; ++f) red[wave][j * FR + f][lane] = acc[j][f];
  __syncthreads();
  const float scale = a.scales != nullptr ? a.scales[u.slot] : 1.f;
  for (int e = threadIdx.x; e < FT * FR * 64; e += 512) {
    const int f = e >> 6, l = e & 63;
    const int r = f % FR * 16 + 4 * (l >> 4), tok = f / FR * 16 + (l & 15);
    f32x4 v = red[0][f][l];
#pragma unroll
    for (int w = 1; w < 8; ++w) v += red[w][f][l];
    if (tok >= n || r >= a.R) continue;
    float hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = v[j] * scale;
      hi[j] = __uint_as_float(f32_to_bf16(y) << 16);
      // not finite: the low part is 0
      lo[j] = __builtin_fabsf(hi[j]) < INFINITY ? y - hi[j] : 0.f;
    }
    uint16_t* p = t + (size_t)(u.start + q + tok) * 2 * a.R + r;
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
    *reinterpret_cast<u32x2*>(p + a.R) =
        u32x2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
  }
}

constexpr int kExpandWaves = 4;

// y of a unit: each of four waves has 16 of its tokens and walks over `steps`
// times 16 F columns (not gated: 128-byte lines).  The step's four fragments of
// B are read once, one by each wave, and shared through LDS (every wave for
// itself, B comes from L2 four times and bounds the kernel: 4096 tokens x 8192,
// rank 64); the next step's loads are in flight meanwhile.  The rows of the F
// fragments of B are dealt so that a lane holds 4 F consecutive columns.
template <int FK, bool kGated>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_kernel(
    AdapterArgs a, const int* __restrict__ order, const Unit* __restrict__ units,
    const uint16_t* __restrict__ t, int total, int steps) {
  constexpr int kHalves = kGated ? 2 : 1, F = kGated ? 2 : 4, kQ = F / 2;
  static_assert(kHalves * F == kExpandWaves, "a fragment a wave");
  __shared__ u32x4 s_b[2][kExpandWaves][FK][64];
  const int at_unit = blockIdx.y + blockIdx.z * gridDim.y;
  if (at_unit >= total) return;
  const Unit u = units[at_unit];
  const bool none = u.slot >= a.S;
  const int n_out = kGated ? a.N / 2 : a.N;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int c0 = blockIdx.x * steps * 16 * F, c1 = min(c0 + steps * 16 * F, n_out);
  const bool added = a.addend != nullptr;
  if (u.count == 0 || c0 >= c1 || (none && !kGated && a.addend == a.out)) return;
  // a wave past the unit's last token works for the others alone
  const int count = u.count - 16 * wave;
  const int place = u.start + min(16 * wave + i, u.count - 1), m = order[place];
  const uint16_t* addend = added ? a.addend + (size_t)m * a.N : nullptr;
  uint16_t* out = a.out + (size_t)m * n_out;
  const uint8_t* B = reinterpret_cast<const uint8_t*>(a.b + (size_t)(none ? 0 : u.slot) * a.N * a.R);
  constexpr u32x4 kZero = {0u, 0u, 0u, 0u};
  struct Loads {
    u32x4 add[kHalves][kQ], b[FK];
  };
  auto load = [&](int c, Loads& l) {
    if (added && count > 0) {
      // lanes past the last column read what is there and store nothing
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int q = 0; q < kQ; ++q)
          l.add[h][q] = load16(addend + h * n_out + min(c + 4 * F * g + 8 * q, n_out - 8));
    }
    if (!none) {
      // row i of fragment wave % F, of the half wave / F
      const int row = min(c + 4 * F * (i >> 2) + 4 * (wave % F) + (i & 3), n_out - 1) +
                      wave / F * n_out;
      const uint32_t at = (uint32_t)__umul24(row, 2 * a.R) + 16 * g;
#pragma unroll
      for (int k = 0; k < FK; ++k) l.b[k] = load16_or_zero(B + (at + 64 * k), 32 * k + 8 * g < a.R);
    }
  };
  Loads next;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int q = 0; q < kQ; ++q) next.add[h][q] = kZero;
#pragma unroll
  for (int k = 0; k < FK; ++k) next.b[k] = kZero;
  load(c0, next);
  u32x4 hi[FK], lo[FK];
#pragma unroll
  for (int k = 0; k < FK; ++k) {
    const uint16_t* p = t + (size_t)place * 2 * a.R + 32 * k + 8 * g;
    const bool ok = !none && 32 * k + 8 * g < a.R;
    hi[k] = load16_or_zero(p, ok);
    lo[k] = load16_or_zero(p + a.R, ok);
  }
  int buf = 0;
#pragma unroll 1
  for (int c = c0; c < c1; c += 16 * F, buf ^= 1) {
#pragma unroll
    for (int k = 0; k < FK; ++k) s_b[buf][wave][k][lane] = next.b[k];
    const Loads now = next;
    wait_lgkm0();
    barrier_nofence();
    if (c + 16 * F < c1) load(c + 16 * F, next);
    if (count <= 0) continue;
    f32x4 acc[kHalves][F];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        u32x4 b[FK];
#pragma unroll
        for (int k = 0; k < FK; ++k) b[k] = s_b[buf][h * F + f][k][lane];
        acc[h][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        // the smaller terms first
#pragma unroll
        for (int k = 0; k < FK; ++k) acc[h][f] = mfma_16x16x32(b[k], lo[k], acc[h][f]);
#pragma unroll
        for (int k = 0; k < FK; ++k) acc[h][f] = mfma_16x16x32(b[k], hi[k], acc[h][f]);
      }
    const int n = c + 4 * F * g;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (i >= count || n + 8 * q >= n_out) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        auto at = [&](int h) {
          const uint32_t w = now.add[h][q][e >> 1];
          return acc[h][2 * q + (e >> 2)][e & 3] + (e & 1 ? bf16_hi(w) : bf16_lo(w));
        };
        y[e] = kGated ? silu_mul(at(0), at(kHalves - 1)) : at(0);
      }
      *reinterpret_cast<u32x4*>(out + n + 8 * q) =
          u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                pack_bf16x2(y[6], y[7])};
    }
  }
}

using moe_host::ceil_div_host;

// Units enough to fill the chip with workgroups of 4 steps (8 and 16 steps: 43
// and 46 us against 41 for 4096 tokens, 8192 columns, rank 64).
constexpr int kManyTokens = 1024;

// Tokens up to which each reads its adapter by itself, whatever the rank: where the
// two meet depends little on how many adapters there are, more on rank and K.  2048
// -> 8192 columns, 16 adapters, each by itself and by units: rank 16, 128 tokens 9.7
// and 14.0 us, 256 13.6 and 15.2; rank 64, 100 tokens 20.6 and 23.5, 128 23.7 and
// 24.0, 192 32 and 25; rank 128, 64 tokens 23.6 and 33.4, 100 33.7 and 34.0, 128 41
// and 35, but 51 and 80 of 8192 -> 8192 columns.  One adapter for all: 7.7 and 12.6,
// 22.5 and 21.8, 39 and 31 at 128 tokens.
constexpr int kGemvTokens = 128;

// One launch where an adapter's A has at most kOneLaunchA bytes and all workgroups'
// reading of it is at most kOneLaunchAll.  It saves a launch's 2.7 us of the host
// (rank 16, 2048 -> 2048 columns, 1 to 64 tokens 8.7 us a call against 11.4) and
// costs time on the GPU, more with the passes of 16 rows over A.  -> 2048 columns, 1
// to 32 tokens, one launch and two: rank 16 x 2048 5.3 to 5.6 and 5.0 to 5.2 us, rank
// 32 x 1408 5.3 to 5.6 and 4.9 to 5.3, rank 128 x 256 9.4 to 9.9 and 6.1 to 6.4;
// larger A: rank 16 x 2560 5.7 to 5.9 and 5.1 to 5.4, x 4096 7.5 to 8.7 and 5.4 to
// 5.6, rank 64 x 1024 7.1 to 7.7 and 5.5 to 5.7; more reading: 64 tokens, rank 16,
// 2048 -> 8192 columns 13.6 and 6.0.
constexpr long long kOneLaunchA = 64 << 10, kOneLaunchAll = 64 << 20;

struct Layout {
  int windows, cap;        // of the grouping; units of a window
  size_t order, units, t, total;
};
Layout layout_of(int M, int R, int S) {
  Layout l;
  l.windows = ceil_div_host(M, kWindow);
  const int w = std::min(M, kWindow);
  l.cap = w / kUnit + std::min(S + 1, w);
  auto align = [](size_t v) { return (v + 255) & ~(size_t)255; };
  l.t = 0;
  l.order = align((size_t)M * R * 4);
  l.units = l.order + align((size_t)M * 4);
  l.total = l.units + align((size_t)l.windows * l.cap * sizeof(Unit));
  return l;
}

template <int FR>
void launch_shrink(const AdapterArgs& a, const Layout& l, const int* order, const Unit* units,
                   uint16_t* t, hipStream_t s) {
  // A of a high rank is read once for 32 tokens (64 adapters of rank 64, 4096 tokens
  // in any order: 69 us by 16, 60 by 32; rank 16: 14.2 and 15.6 for 1000)
  constexpr int FT = FR >= 4 ? 2 : 1;
  shrink_kernel<FR, FT>
      <<<l.windows * l.cap * (kUnit / (16 * FT)), 512, 0, s>>>(a, order, units, t);
}
template <int FK, bool kGated>
void launch_expand(const AdapterArgs& a, const Layout& l, const int* order, const Unit* units,
                   const uint16_t* t, hipStream_t s) {
  // the columns of one unit next to each other: the rows' lines, and with 8 XCDs
  // the same columns of B, meet in one L2
  const int units_all = l.windows * l.cap, high = std::min(units_all, 32768);
  const int steps = a.M >= kManyTokens ? 4 : 1;
  const dim3 grid((unsigned)ceil_div_host(kGated ? a.N / 2 : a.N, 16 * (kGated ? 2 : 4) * steps),
                  (unsigned)high, (unsigned)ceil_div_host(units_all, high));
  expand_kernel<FK, kGated><<<grid, 64 * kExpandWaves, 0, s>>>(a, order, units, t, units_all,
                                                               steps);
}

}  // namespace

namespace moe_host {

size_t adapters_bytes(int M, int R) {
  // any number of adapters up to the most
  return layout_of(M, R, kMaxSlots).total;
}

hipError_t launch_adapters(const AdapterArgs& a, hipStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const Layout l = layout_of(a.M, a.R, a.S);
  if (a.M <= kGemvTokens) {
    float* t = reinterpret_cast<float*>(ws + l.t);
    const int n_out = a.gated ? a.N / 2 : a.N;
    const dim3 grid((unsigned)ceil_div_host(n_out, 256), (unsigned)a.M);
    const long long bytes = (long long)a.R * a.K * 2;
    if (bytes <= kOneLaunchA && bytes * grid.x * a.M <= kOneLaunchAll) {
      if (a.gated)
        adapters_gemv_kernel<true><<<grid, 256, 0, s>>>(a);
      else
        adapters_gemv_kernel<false><<<grid, 256, 0, s>>>(a);
      return hipGetLastError();
    }
    shrink_gemv_kernel<2><<<ceil_div_host(a.M * (a.R / 2), 4), 256, 0, s>>>(a, t);
    if (a.gated)
      expand_gemv_kernel<true><<<grid, 256, 0, s>>>(a, t);
    else
      expand_gemv_kernel<false><<<grid, 256, 0, s>>>(a, t);
    return hipGetLastError();
  }
  int* order = reinterpret_cast<int*>(ws + l.order);
  Unit* units = reinterpret_cast<Unit*>(ws + l.units);
  uint16_t* t = reinterpret_cast<uint16_t*>(ws + l.t);
  plan_kernel<<<l.windows, kPlanThreads, 0, s>>>(a, order, units, l.cap);
  if (a.R <= 16)
    launch_shrink<1>(a, l, order, units, t, s);
  else if (a.R <= 32)
    launch_shrink<2>(a, l, order, units, t, s);
  else if (a.R <= 64)
    launch_shrink<4>(a, l, order, units, t, s);
  else
    launch_shrink<8>(a, l, order, units, t, s);
  if (a.gated) {
    if (a.R <= 32)
      launch_expand<1, true>(a, l, order, units, t, s);
    else if (a.R <= 64)
      launch_expand<2, true>(a, l, order, units, t, s);
    else
      launch_expand<4, true>(a, l, order, units, t, s);
  } else {
    if (a.R <= 32)
      launch_expand<1, false>(a, l, order, units, t, s);
    else if (a.R <= 64)
      launch_expand<2, false>(a, l, order, units, t, s);
    else
      launch_expand<4, false>(a, l, order, units, t, s);
  }
  return hipGetLastError();
}

}  // namespace moe_host
