// A gated feed-forward block in bf16 and its gradient:
//   gate = x Wg^T,  up = x Wu^T,  act = SiLU(gate) * up      w13 = [Wg; Wu]
//   s = 1 / (1 + e^-gate)
//   d_up = d_act * gate * s,  d_gate = d_act * up * s * (1 + gate (1 - s))
//   d_x = [d_gate d_up] w13,  d_w13 = [d_gate d_up]^T x
//
// Four products on one tile kernel; every sum is fp32.  d_gate and d_up are
// rounded to bf16, as the matrix cores take them: the gradients are then sqrt 2
// as far off as their own rounding leaves them.  Of kFewRows rows or fewer each
// is kept as two bf16 numbers, a high part and what it leaves, a row each: the
// tiles have room for them (5632 features x 2048, 1 to 16 rows: 48 to 51 us; with
// one number each it took as long).
#include <algorithm>
#include <type_traits>
#include <utility>

#include "dense.h"

using namespace moe;

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Which product a tile kernel forms.  n is the output's contiguous axis.
//   kAct, kGradAct: out[m, i] from gate and up, both [m, n] = x w13^T
//   kGradX:  out[m, n] = sum_k d[m, k] w13[k, n]
//   kGradW:  out[m, n] = sum_k d[k, m] x[k, n]
enum Op { kAct, kGradAct, kGradX, kGradW };

// One operand: its rows (the output's axis) by k.
//   across false: element (r, k) at p[r * ld + k];  true: at p[k * ld + r].
struct TileArgs {
  const uint16_t* m_side;
  const uint16_t* n_side;
  int m_ld, n_ld;
  int rows, cols, K;         // output rows and columns (gated: columns of out), summed length
  int tiles_m, tiles_n, splits, k_per;   // K split into `splits` ranges of k_per
  const uint16_t* grad_out;  // kGradAct: [rows, cols]
  uint16_t* out;             // [rows, out_ld]
  int out_ld;
  float* partial;            // splits * parts > 1: [splits, rows, cols]
  int parts;                 // gradients: 2 where d is [high parts; low parts]
};

// Swizzles of the LDS tiles, in 16-byte pieces.  Rows of kK k: piece c of row r
// lies at c ^ (r / 2 % pieces), c ^ (r % 16) where a row is 256 bytes, so that the
// rows of one beat of a 16-byte read lie in different banks.  Rows of R columns:
// the pairs of pieces are exchanged by the bits of k in which the lanes of a
// transposing read differ.
template <int kK>
__device__ __forceinline__ int along_swizzle(int r) {
  return kK < 128 ? (r >> 1) & (kK / 8 - 1) : r & 15;
}
__device__ __forceinline__ int across_swizzle(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

// load_lds16 whose completion the kernel waits for itself (wait_vmem): the
// compiler, which cannot tell the stages of the ring apart, would wait for
// every copy in flight before each read of LDS.  `lds` is a byte address in
// LDS, the same for the whole wave.  (m0 is reserved: nothing else in these
// kernels uses it.)
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(lds)
               : "memory");
}

// The loads of one operand's stages: R rows by kK k, by W waves.
template <int R, int kK, int W, bool kAcross>
struct Loader {
  static constexpr int kInstr = R * kK * 2 / 1024 / W;   // 1 KB each
  const uint8_t* src[kInstr];
  int k[kInstr];             // k of the lane's piece within a stage
  size_t step;
  // row(r): the operand's row of tile row r (clamped to one that exists);
  // across: the tile's first column and how many columns there are; k from `wrap`
  // on is k - wrap (one stage alone)
  template <class F>
  __device__ __forceinline__ void init(const uint16_t* p, int ld, int k0, F row, int c0, int ncols,
                                       int wave, int lane, int wrap = 0x7fffffff) {
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      const int q = wave * kInstr + i;
      if (kAcross) {
        constexpr int kPieces = R / 8;                    // per k
        k[i] = q * (64 / kPieces) + lane / kPieces;
        const int c = (lane % kPieces) ^ across_swizzle(k[i]);
        const int col = min(c0 + c * 8, ncols - 8);
        const int at = k0 + k[i] < wrap ? k0 + k[i] : k0 + k[i] - wrap;
        src[i] = reinterpret_cast<const uint8_t*>(p + (size_t)at * ld + col);
      } else {
        constexpr int kPieces = kK / 8;                   // per row
        const int r = q * (64 / kPieces) + lane / kPieces;
        const int c = (lane % kPieces) ^ along_swizzle<kK>(r);
        k[i] = c * 8;
        src[i] = reinterpret_cast<const uint8_t*>(p + (size_t)row(r) * ld + k0 + k[i]);
      }
    }
    step = kAcross ? (size_t)kK * ld * 2 : kK * 2;
  }
  // The next stage into LDS; `left` elements of k are there from its first on
  // (none or fewer: zeros).
  __device__ __forceinline__ void issue(uint32_t lds, int wave, int left) {
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      copy16(k[i] < left ? (const void*)src[i] : (const void*)kZeroPage,
             lds + (wave * kInstr + i) * 1024);
      src[i] += step;
    }
  }
};

// Fragments (16 rows by 32 k) of one operand's LDS tile.
template <int R, int kK, bool kAcross>
struct Reader {
  int base, col, swz;        // bytes
  __device__ __forceinline__ Reader(int row0, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if (kAcross) {
      const int k = 8 * g + (i >> 2);
      base = k * R * 2 + (i & 1) * 8;
      col = row0 * 2 + ((i & 2) << 3);
      swz = across_swizzle(k) * 16;
    } else {
      base = (row0 + i) * kK * 2;
      col = g * 16;
      swz = along_swizzle<kK>(i) * 16;
    }
  }
  // fragment f of rows, of the 32 k at 32 s
  __device__ __forceinline__ u32x4 read(const uint8_t* lds, int f, int s) const {
    if (kAcross) {
      const uint8_t* p = lds + base + s * 64 * R + ((col + f * 32) ^ swz);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * R * 2));
      const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
      return u32x4{x[0], x[1], y[0], y[1]};
    }
    return load16(lds + base + ((col + s * 64) ^ swz) + f * (32 * kK));
  }
};

// Derivatives of SiLU(g) u times d.
__device__ __forceinline__ void gated_grad(float g, float u, float d, float& dg, float& du) {
  const float s = 1.0f / (1.0f + __expf(-g));
  du = d * (g * s);
  dg = d * u * (s * (1.0f + g * (1.0f - s)));
}

// f(0), f(1), ... as constants
template <class F, int... i>
__device__ __forceinline__ void each(std::integer_sequence<int, i...>, const F& f) {
  (f(std::integral_constant<int, i>{}), ...);
}

constexpr int kFewRows = 16;

// What a bf16 number leaves of v (nothing where it is not finite).
__device__ __forceinline__ float left_of(float v, float high) {
  return __builtin_fabsf(high) < INFINITY ? v - high : 0.f;
}

// Tiles of BM x BN in stages of kK k, a ring of kStages; WM x WN waves, KS times:
// each such group takes its share of every stage's k.
template <int BM, int BN, int kK, int WM, int WN, int KS, int kStages, Op kOp>
__global__ __launch_bounds__(64 * WM * WN * KS, BM < 128 && WN == 1 ? 1 : 2) void tile_kernel(
    TileArgs a) {
  constexpr int W = WM * WN * KS, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool kGated = kOp == kAct || kOp == kGradAct;
  constexpr bool kMAcross = kOp == kGradW, kNAcross = kOp == kGradX || kOp == kGradW;
  constexpr int kMBytes = BM * kK * 2, kStage = (BM + BN) * kK * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;

  // tiles of one XCD are neighbours: columns of up to 8 tiles of m
  int t = xcd_contiguous_tile(blockIdx.x, a.tiles_m * a.tiles_n * a.splits);
  if (t < 0) return;
  const int split = t / (a.tiles_m * a.tiles_n);
  t %= a.tiles_m * a.tiles_n;
  const int band = t / (8 * a.tiles_n), high = min(8, a.tiles_m - band * 8);
  t -= band * 8 * a.tiles_n;
  const int m0 = (band * 8 + t % high) * BM, tn = t / high;
  const int n0 = tn * (kGated ? BN / 2 : BN);
  const int k0 = split * a.k_per, K = min(a.K - k0, a.k_per);

  Loader<BM, kK, W, kMAcross> lm;
  Loader<BN, kK, W, kNAcross> ln;
  lm.init(a.m_side, a.m_ld, k0, [&](int r) { return min(m0 + r, a.rows - 1); }, m0, a.rows, wave,
          lane);
  ln.init(a.n_side, a.n_ld, k0,
          [&](int r) {
            if (!kGated) return min(n0 + r, a.cols - 1);
            // a wave's TN rows: TN/2 gates, then their ups; row i of fragment h of a
            // half is feature 8 (i / 4) + 4 h + i % 4, so that a lane holds 8
            // consecutive ones
            const int q = r % TN, h = q % (TN / 2) / 16, i = q % 16;
            const int f = min(n0 + r / TN * (TN / 2) + 8 * (i >> 2) + 4 * h + (i & 3), a.cols - 1);
            return q < TN / 2 ? f : a.cols + f;
          },
          n0, a.cols, wave, lane, kOp == kGradW && a.parts == 2 ? a.K / 2 : 0x7fffffff);
  const Reader<BM, kK, kMAcross> rm(wm * TM, lane);
  const Reader<BN, kK, kNAcross> rn(wn * TN, lane);

  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Stage kt of K, while the stages behind it are on their way: fragments to
  // registers, the copies of stage kt + kStages - 1 sent into the LDS of stage
  // kt - 1, which every wave has read; then the products.  The last stages have
  // no copies to send and wait for fewer (copies of zeros past the end, so that
  // every stage is alike: 128 rows x 2048 x 5632 1.4 us, 4096 rows 3).  Eight
  // waves are two halves, half a stage apart, so that of the two waves of a SIMD
  // one multiplies while the other reads.
  constexpr bool kHalves = W == 8 && KS == 1;
  constexpr int kSteps = kK / 32 / KS, kRead = kHalves ? 1 : kSteps;   // a wave's of a stage
  constexpr int kCopies = Loader<BM, kK, W, kMAcross>::kInstr + Loader<BN, kK, W, kNAcross>::kInstr;
  const int nk = max(ceil_div(K, kK), kStages - 1);
  const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_void_t*)lds;
  auto issue = [&](int kt) {
    const uint32_t to = lds_at + (uint32_t)(kt % kStages) * kStage;
    lm.issue(to, wave, K - kt * kK);
    ln.issue(to + kMBytes, wave, K - kt * kK);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  wait_vmem<(kStages - 2) * kCopies>();
  barrier_nofence();
  if (kHalves && wave >= W / 2) barrier_nofence();
  auto step = [&](int kt, auto more, auto left) {
    const uint8_t* at = lds + (kt % kStages) * kStage;
#pragma unroll
    for (int s0 = 0; s0 < kSteps; s0 += kRead) {
      u32x4 fn[kRead][FN], fm[kRead][FM];
#pragma unroll
      for (int q = 0; q < kRead; ++q) {
#pragma unroll
        for (int i = 0; i < FN; ++i) fn[q][i] = rn.read(at + kMBytes, i, wk * kSteps + s0 + q);
#pragma unroll
        for (int j = 0; j < FM; ++j) fm[q][j] = rm.read(at, j, wk * kSteps + s0 + q);
      }
      if (more && s0 == 0) issue(kt + kStages - 1);
      wait_lgkm0();
      if (s0 + kRead == kSteps) wait_vmem<left * kCopies>();   // stage kt + 1 is there
      barrier_nofence();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int q = 0; q < kRead; ++q)
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) acc[i][j] = mfma_16x16x32(fn[q][i], fm[q][j], acc[i][j]);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      if (kHalves) barrier_nofence();
    }
  };
#pragma unroll 1
  for (int kt = 0; kt < nk - (kStages - 1); ++kt)
    step(kt, std::true_type{}, std::integral_constant<int, kStages - 2>{});
  each(std::make_integer_sequence<int, kStages - 1>{}, [&](auto i) {
    step(nk - (kStages - 1) + i, std::false_type{},
         std::integral_constant<int, (kStages - 3 - i > 0 ? kStages - 3 - i : 0)>{});
  });
  if (kHalves && wave < W / 2) barrier_nofence();

  // the groups' sums meet in LDS, in order, and each group finishes its rows
  constexpr int FE = FM > KS ? FM / KS : 1;
  if (KS > 1) {
    static_assert(KS == 1 || (W * FN * FM * 1024 <= sizeof(lds)), "the sums");
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) red[((wave * FN + i) * FM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wk * FE >= FM) return;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FE; ++j) {
        const f32x4* p = red + (((wave % (WM * WN)) * FN + i) * FM + wk * FE + j) * 64 + lane;
        acc[i][j] = p[0];
#pragma unroll
        for (int q = 1; q < KS; ++q) acc[i][j] += p[q * (WM * WN * FN * FM * 64)];
      }
  }
  // a lane holds 4 consecutive n of one m, gated 8 features
  const int ml = m0 + wm * TM + wk * FE * 16 + (lane & 15), nq = 4 * (lane >> 4);
#pragma unroll
  for (int j = 0; j < FE; ++j) {
    const int m = ml + j * 16;
    if (m >= a.rows) continue;
    if (kGated) {
      static_assert(!kGated || FN == 4, "two fragments of gates, two of ups");
      const int n = n0 + wn * (TN / 2) + 2 * nq;
      if (n >= a.cols) continue;
      const size_t at = (size_t)m * a.out_ld + n;
      if (kOp == kAct) {
        u32x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 g = acc[r >> 1][j], u = acc[2 + (r >> 1)][j];
          const int e = 2 * (r & 1);
          o[r] = pack_bf16x2(silu_mul(g[e], u[e]), silu_mul(g[e + 1], u[e + 1]));
        }
        *reinterpret_cast<u32x4*>(a.out + at) = o;
      } else {
        const u32x4 d = load16(a.grad_out + (size_t)m * a.cols + n);
        // a low part as well (a large batch's last rows have such tiles too, and none)
        const bool two = BM <= kFewRows && a.parts == 2;
        u32x4 og, ou, lg, lu;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 g = acc[r >> 1][j], u = acc[2 + (r >> 1)][j];
          const int e = 2 * (r & 1);
          float dg[2], du[2];
          gated_grad(g[e], u[e], bf16_lo(d[r]), dg[0], du[0]);
          gated_grad(g[e + 1], u[e + 1], bf16_hi(d[r]), dg[1], du[1]);
          og[r] = pack_bf16x2(dg[0], dg[1]);
          ou[r] = pack_bf16x2(du[0], du[1]);
          if (two) {
            lg[r] = pack_bf16x2(left_of(dg[0], bf16_lo(og[r])), left_of(dg[1], bf16_hi(og[r])));
            lu[r] = pack_bf16x2(left_of(du[0], bf16_lo(ou[r])), left_of(du[1], bf16_hi(ou[r])));
          }
        }
        *reinterpret_cast<u32x4*>(a.out + at) = og;
        *reinterpret_cast<u32x4*>(a.out + at + a.cols) = ou;
        if (two) {
          const size_t low = at + (size_t)a.rows * a.out_ld;
          *reinterpret_cast<u32x4*>(a.out + low) = lg;
          *reinterpret_cast<u32x4*>(a.out + low + a.cols) = lu;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int n = n0 + wn * TN + i * 16 + nq;
        if (n >= a.cols) continue;
        const f32x4 v = acc[i][j];
        if (a.splits > 1 || (kOp == kGradX && a.parts > 1))
          *reinterpret_cast<f32x4*>(a.partial + ((size_t)split * a.rows + m) * a.cols + n) = v;
        else
          *reinterpret_cast<u32x2*>(a.out + (size_t)m * a.out_ld + n) =
              u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
  }
}

// ---- one to four rows: a GEMV, a wave reads the gate and up row of one feature ----
//
// Four waves a workgroup, so that 5632 features are 5.5 of them on every CU
// (2048 x 5632, one row 9.7 us; eight waves of two features 11.6: 1.4 workgroups
// a CU).  Two to four rows 4.7 to 5.6 us (2048 x 1408), 6.4 to 7.5 (4096 x 1024),
// 28 to 32 (8192 x 4096); by tiles 6.9, 10.1 and 31.6.  2048 x 5632 is the one size
// measured where tiles are as fast: 10.1 to 10.6 and 9.8 to 10.0.
constexpr int kGemvRows = 4;
constexpr int kGemvWaves = 4;

template <int T>
__global__ __launch_bounds__(64 * kGemvWaves) void gated_gemv_kernel(moe_host::GatedArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f = blockIdx.x * kGemvWaves + wave;
  if (f >= a.I) return;
  const uint16_t* w[2] = {a.w13 + (size_t)f * a.H, a.w13 + (size_t)(a.I + f) * a.H};
  float sum[2][T];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < T; ++t) sum[h][t] = 0.f;
  auto step = [&](int k) {
    u32x4 x[T], v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h] = load16(w[h] + k);
#pragma unroll
    for (int t = 0; t < T; ++t) x[t] = load16(a.x + (size_t)t * a.H + k);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[h][t] = __builtin_fmaf(bf16_lo(x[t][j]), bf16_lo(v[h][j]), sum[h][t]);
          sum[h][t] = __builtin_fmaf(bf16_hi(x[t][j]), bf16_hi(v[h][j]), sum[h][t]);
        }
  };
  int k = 0;
#pragma unroll 4
  for (; k + 512 <= a.H; k += 512) step(k + lane * 8);
  if (k + lane * 8 < a.H) step(k + lane * 8);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const float g = wave_sum(sum[0][t]), u = wave_sum(sum[1][t]);
    if (lane == 0) a.out[(size_t)t * a.I + f] = (uint16_t)f32_to_bf16(silu_mul(g, u));
  }
}

// out = bf16(sum of the splits, and of a row's parts, in their order); n a multiple
// of 8
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int splits,
                                                   size_t n, uint16_t* __restrict__ out) {
  for (size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; at < n;
       at += (size_t)gridDim.x * 2048) {
    f32x4 s[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 8
    for (int i = 0; i < splits; ++i) {
      const f32x4* p = reinterpret_cast<const f32x4*>(partial + (size_t)i * n + at);
      s[0] += p[0];
      s[1] += p[1];
    }
    *reinterpret_cast<u32x4*>(out + at) =
        u32x4{pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
              pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
  }
}

__global__ __launch_bounds__(256) void zero_kernel(u32x4* p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    p[i] = u32x4{0u, 0u, 0u, 0u};
}

using moe_host::ceil_div_host;

constexpr int kTileCus = 256;          // CUs that tiles are counted for
constexpr int kMaxSplits = 16;
constexpr int kSplitTiles = 1024;
constexpr int kSmallSplitTiles = 256;   // 512 and 1024: 5 and 12 % slower at 509 x 2048 x 1408

// Tile size and ranges of K of one product.  Copies into LDS bound them all (9 to
// 12 TB/s from L2 over the chip), and what they cost follows the lines that they
// touch.
//
// Large: 256 x 256 where half the chip has one, however few the rows (16 rows'
// gradient, 40000 x 1408, 182 us with grad_x alone, by 128 x 128 176); whole
// 128-byte lines, two stages of 64 k, hold too little in flight (4096 rows x 2048 x
// 5632 175 us for 168).
// Sums of grad_x and grad_w13 shorter than kShortSum, which store more than they
// read, take 128 x 128 all the same.  grad_w13's are two workgroups to a CU: one
// stores while the other reads (200 rows' grad_w13 of 2 x 5632 x 2048 51 us for 55
// with gate and up before it); grad_x's, one to a CU, gain with few tiles and lose
// with many (4096 x 2048 x 248 33 us for 46, 4096 x 8192 x 200 100 for 81).
// 128 x 128, but for grad_w13: 64 x 64 a wave, four to each half of a stage's 64 k
// (900 rows x 2048 x 1408 20.4 us; four waves, stages of 32 k 23.7; 1500 x 2048 x
// 5632 gate, up and grad_x 168 for 193, the same with grad_w13 164 for 159).
//
// Gate and up of at most 64 rows, or where 128 x 128 would leave half the chip
// without: tiles of 64 rows or fewer whose waves are 64 rows of w13 wide (32 gates
// and their ups) and share out a stage of 128 k, 256-byte runs of every row.  So a
// fragment of x is read from LDS once a tile, or twice; the sums meet in LDS at
// the end.  Tiles 64 wide while the chip holds them at once, else 128.  2048 x
// 5632: 16 rows 11.0 us, 32 12.0, 64 14.0 (weights through LDS of each wave's own
// and x straight to registers 13.5, 15, 19), 128 rows 18.2; 200 x 2048 x 1408
// 10.3, 300 x 4096 x 1024 16.6, 509 x 2048 x 1408 14.3 (64 x 128 by waves side by
// side, stages of 64 k: 18.2, 16.2, 28.6, 16.3).
//
// A product whose sum is all it stores is cut along K until every CU has a tile,
// in ranges of at least 8 times 32 k; one that ends inside a tile's stage of 64 or
// 128 k is filled up with zeros.
// grad_x whose ranges would be kShortRange or less takes 64 x 128 and longer ones
// where 128 x 128 would leave half the chip without (with gate and up 300 x 4096 x
// 1024 30.2 us for 33.8, 509 x 2048 x 1408 30.2 for 31.7, 1000 x 2048 x 200 18.3 for
// 20.1; 5632 features, ranges of 2816, 85 for 82; more tiles than half the chip: 300 x
// 8192 x 248 40.0 for 37.2, 1800 x 2048 x 200 25.4 for 21.8, 4096 x 8192 x 200 132
// for 101).
constexpr int kShortSum = 512, kShortRange = 1024;

struct Plan {
  int bm, bn;                // tile
  int splits, k_per;
};
Plan plan_of(Op op, int rows, int n_rows, int K) {
  auto tiles = [&](int bm, int bn) {
    return (long long)ceil_div_host(rows, bm) * ceil_div_host(n_rows, bn);
  };
  const bool gated = op == kAct || op == kGradAct;
  const int cu = kTileCus, stages = ceil_div_host(K, 32);   // the shortest tiles' stages
  Plan p{128, 128, 1, K};
  if (gated && (rows <= 64 || tiles(128, 128) <= cu / 2)) {
    p.bm = rows <= kFewRows ? kFewRows : rows <= 32 ? 32 : 64;
    p.bn = p.bm == kFewRows || tiles(64, 64) <= cu ? 64 : 128;
    return p;
  }
  if (tiles(256, 256) >= cu / 2 && (gated || K >= kShortSum)) p.bm = p.bn = 256;
  auto cut = [&] {
    const long long all = tiles(p.bm, p.bn);
    if (all >= cu) return;
    const long long most = std::min(stages / 8, kMaxSplits);
    const long long room = p.bm == 256 ? kSplitTiles / 4 : kSmallSplitTiles;
    p.splits = (int)std::max<long long>(1, std::min(room / all, most));
    p.k_per = ceil_div_host(stages, p.splits) * 32;
    p.splits = ceil_div_host(K, p.k_per);
  };
  if (!gated) cut();
  if (op == kGradX && p.bm == 128 && p.k_per <= kShortRange && tiles(128, 128) <= cu / 2) {
    p = Plan{64, 128, 1, K};
    cut();
  }
  return p;
}

template <Op kOp>
hipError_t launch_tiles(TileArgs a, int n_rows, hipStream_t s) {
  constexpr bool kGated = kOp == kAct || kOp == kGradAct;
  const Plan p = plan_of(kOp, a.rows, n_rows, a.K);
  a.splits = p.splits;
  a.k_per = p.k_per;
  a.tiles_m = ceil_div_host(a.rows, p.bm);
  a.tiles_n = ceil_div_host(n_rows, p.bn);
  TileArgs rest = a;
  const int last = a.tiles_m * a.tiles_n % kTileCus;
  const int whole = a.tiles_m * a.tiles_n / kTileCus * kTileCus / a.tiles_n;   // rows of tiles
  if (p.bm == 256 && p.splits == 1 && whole > 0 && last > 0 && last <= kTileCus / 2) {
    // a last round that leaves half the chip idle: its rows are a product of
    // their own, of smaller tiles (4096 x 2048 x 5632, grad_w13: 352 tiles)
    a.tiles_m = whole;
    a.rows = whole * 256;
    const size_t down = (size_t)a.rows;
    rest.rows -= a.rows;
    rest.m_side += kOp == kGradW ? down : down * rest.m_ld;
    rest.out += down * rest.out_ld;
    if (rest.grad_out != nullptr) rest.grad_out += down * rest.cols;
  } else {
    rest.rows = 0;
  }
  const unsigned grid = (unsigned)ceil_div_host(a.tiles_m * a.tiles_n * a.splits, 8) * 8;
  auto run = [&](auto kernel, int waves) { kernel<<<grid, 64 * waves, 0, s>>>(a); };
  if (p.bm == 256) {
    run(tile_kernel<256, 256, 32, 2, 4, 1, 4, kOp>, 8);
  } else if constexpr (kGated) {
    if (p.bm == 128)
      run(tile_kernel<128, 128, 64, 2, 2, 2, 4, kOp>, 8);
    else if (p.bn == 128)
      p.bm == 64 ? run(tile_kernel<64, 128, 128, 1, 2, 4, 3, kOp>, 8)
                 : run(tile_kernel<32, 128, 128, 1, 2, 4, 3, kOp>, 8);
    else if (p.bm == 64)
      run(tile_kernel<64, 64, 128, 1, 1, 4, 4, kOp>, 4);
    else if (p.bm == 32)
      run(tile_kernel<32, 64, 128, 1, 1, 4, 4, kOp>, 4);
    else
      run(tile_kernel<kFewRows, 64, 128, 1, 1, 4, 4, kOp>, 4);
  } else if constexpr (kOp == kGradX) {
    if (p.bm == 128)
      run(tile_kernel<128, 128, 64, 2, 2, 2, 4, kOp>, 8);
    else
      run(tile_kernel<64, 128, 128, 1, 2, 4, 3, kOp>, 8);
  } else {
    run(tile_kernel<128, 128, 32, 2, 2, 1, 4, kOp>, 4);
  }
  const int parts = kOp == kGradX ? a.parts : 1;
  if (p.splits * parts > 1) {
    const size_t n = (size_t)a.rows / parts * a.cols;
    const unsigned g = (unsigned)std::min<size_t>((n / 8 + 255) / 256, 4096);
    join_kernel<<<g, 256, 0, s>>>(a.partial, p.splits * parts, n, a.out);
  }
  const hipError_t err = hipGetLastError();
  return err != hipSuccess || rest.rows == 0 ? err : launch_tiles<kOp>(rest, n_rows, s);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
// Room for the ranges' sums of any product with at most so many rows: a plan
// has at most kMaxSplits ranges and, where it has more than one, no more than
// kSplitTiles tiles of 128 x 128 over all of them.
size_t partial_bytes(int rows, int cols) {
  return std::min<size_t>((size_t)kMaxSplits * rows * cols * 4, (size_t)kSplitTiles * 128 * 128 * 4);
}

}  // namespace

namespace moe_host {

hipError_t launch_gated(const GatedArgs& a, hipStream_t s) {
  if (a.M <= kGemvRows) {
    const int grid = ceil_div_host(a.I, kGemvWaves);
    switch (a.M) {
      case 1: gated_gemv_kernel<1><<<grid, 64 * kGemvWaves, 0, s>>>(a); break;
      case 2: gated_gemv_kernel<2><<<grid, 64 * kGemvWaves, 0, s>>>(a); break;
      case 3: gated_gemv_kernel<3><<<grid, 64 * kGemvWaves, 0, s>>>(a); break;
      default: gated_gemv_kernel<4><<<grid, 64 * kGemvWaves, 0, s>>>(a); break;
    }
    return hipGetLastError();
  }
  TileArgs t{};
  t.m_side = a.x;
  t.n_side = a.w13;
  t.m_ld = t.n_ld = t.K = a.H;
  t.rows = a.M;
  t.cols = t.out_ld = a.I;
  t.out = a.out;
  return launch_tiles<kAct>(t, 2 * a.I, s);
}

hipError_t launch_zero(void* p, size_t bytes, hipStream_t s) {
  const size_t n = bytes / 16;
  zero_kernel<<<(unsigned)std::min<size_t>((n + 255) / 256, 4096), 256, 0, s>>>(
      static_cast<u32x4*>(p), n);
  return hipGetLastError();
}

// Rows of d: its parts, and no fewer than a smaller batch has.
static int rows_of_d(int M) { return std::max(M, std::min(2 * M, 2 * kFewRows)); }

// [d_gate d_up] [rows_of_d(M), 2I], then the larger of the two products' partial sums
size_t gated_backward_bytes(int M, int H, int I) {
  const int rows = rows_of_d(M);
  return align256((size_t)rows * 2 * I * 2) +
         std::max(partial_bytes(rows, H), partial_bytes(2 * I, H));
}

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s) {
  uint16_t* d = static_cast<uint16_t*>(a.workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                            align256((size_t)rows_of_d(a.M) * 2 * a.I * 2));
  const int parts = a.M <= kFewRows ? 2 : 1;
  TileArgs t{};
  t.m_side = a.x;
  t.n_side = a.w13;
  t.m_ld = t.n_ld = t.K = a.H;
  t.rows = a.M;
  t.cols = a.I;
  t.grad_out = a.grad_out;
  t.out = d;
  t.out_ld = 2 * a.I;
  t.parts = parts;
  hipError_t err = launch_tiles<kGradAct>(t, 2 * a.I, s);
  if (err == hipSuccess && a.grad_x != nullptr) {
    TileArgs g{};
    g.m_side = d;
    g.n_side = a.w13;
    g.m_ld = g.K = 2 * a.I;
    g.n_ld = g.cols = g.out_ld = a.H;
    g.rows = a.M * parts;
    g.out = a.grad_x;
    g.partial = partial;
    g.parts = parts;
    err = launch_tiles<kGradX>(g, a.H, s);
  }
  if (err == hipSuccess && a.grad_w13 != nullptr) {
    TileArgs g{};
    g.m_side = d;
    g.n_side = a.x;
    g.m_ld = g.rows = 2 * a.I;
    g.n_ld = g.cols = g.out_ld = a.H;
    g.K = a.M * parts;
    g.out = a.grad_w13;
    g.partial = partial;
    g.parts = parts;
    err = launch_tiles<kGradW>(g, a.H, s);
  }
  return err;
}

}  // namespace moe_host
