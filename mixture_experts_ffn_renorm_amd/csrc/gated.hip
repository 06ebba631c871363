// A gated feed-forward block in bf16 and its gradient:
//   gate = x Wg^T,  up = x Wu^T,  act = SiLU(gate) * up      w13 = [Wg; Wu]
//   s = 1 / (1 + e^-gate)
//   d_up = d_act * gate * s,  d_gate = d_act * up * s * (1 + gate (1 - s))
//   d_x = [d_gate d_up] w13,  d_w13 = [d_gate d_up]^T x
//
// Four products on one tile kernel.  d_gate and d_up are rounded to bf16 once,
// as the matrix cores take them; every sum is fp32.
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
  float* partial;            // splits > 1: [splits, rows, cols]
};

// Swizzles of the LDS tiles, in 16-byte pieces.  Rows of kK k: piece c of row r
// lies at c ^ (r / 2 % pieces), so that the rows of one beat of a 16-byte read
// lie in different banks.  Rows of R columns: the pairs of pieces are exchanged
// by the bits of k in which the lanes of a transposing read differ.
template <int kK>
__device__ __forceinline__ int along_swizzle(int r) {
  return (r >> 1) & (kK / 8 - 1);
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
  // across: the tile's first column and how many columns there are
  template <class F>
  __device__ __forceinline__ void init(const uint16_t* p, int ld, int k0, F row, int c0, int ncols,
                                       int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kInstr; ++i) {
      const int q = wave * kInstr + i;
      if (kAcross) {
        constexpr int kPieces = R / 8;                    // per k
        k[i] = q * (64 / kPieces) + lane / kPieces;
        const int c = (lane % kPieces) ^ across_swizzle(k[i]);
        const int col = min(c0 + c * 8, ncols - 8);
        src[i] = reinterpret_cast<const uint8_t*>(p + (size_t)(k0 + k[i]) * ld + col);
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

// Tiles of BM x BN in stages of kK k, a ring of kStages; WM x WN waves, KS times:
// each such group takes its share of every stage's k.
template <int BM, int BN, int kK, int WM, int WN, int KS, int kStages, Op kOp>
__global__ __launch_bounds__(64 * WM * WN * KS, KS == 1 ? 2 : 1) void tile_kernel(TileArgs a) {
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
          n0, a.cols, wave, lane);
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
  constexpr bool kHalves = W == 8;
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
  constexpr int FE = FM / KS;
  if (KS > 1) {
    static_assert(KS == 1 || (W * FN * FM * 1024 <= sizeof(lds) && FM % KS == 0), "the sums");
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) red[((wave * FN + i) * FM + j) * 64 + lane] = acc[i][j];
    __syncthreads();
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
        u32x4 og, ou;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 g = acc[r >> 1][j], u = acc[2 + (r >> 1)][j];
          const int e = 2 * (r & 1);
          float dg[2], du[2];
          gated_grad(g[e], u[e], bf16_lo(d[r]), dg[0], du[0]);
          gated_grad(g[e + 1], u[e + 1], bf16_hi(d[r]), dg[1], du[1]);
          og[r] = pack_bf16x2(dg[0], dg[1]);
          ou[r] = pack_bf16x2(du[0], du[1]);
        }
        *reinterpret_cast<u32x4*>(a.out + at) = og;
        *reinterpret_cast<u32x4*>(a.out + at + a.cols) = ou;
      }
    } else {
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int n = n0 + wn * TN + i * 16 + nq;
        if (n >= a.cols) continue;
        const f32x4 v = acc[i][j];
        if (a.splits > 1)
          *reinterpret_cast<f32x4*>(a.partial + ((size_t)split * a.rows + m) * a.cols + n) = v;
        else
          *reinterpret_cast<u32x2*>(a.out + (size_t)m * a.out_ld + n) =
              u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
  }
}

// ---- few rows: the weights are read once, as fast as memory gives them ----

constexpr int kGemvRows = 4;           // rows of the GEMVs
constexpr int kFewRows = 64;           // rows of the streaming products
constexpr int kGemvFeatures = 2;       // features of a wave

// One to four rows: a wave reads the gate and up rows of kGemvFeatures
// features, 1 KB of each at a time.
template <int T>
__global__ __launch_bounds__(512) void gated_gemv_kernel(moe_host::GatedArgs a) {
  constexpr int F = kGemvFeatures;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f0 = (blockIdx.x * 8 + wave) * F;
  if (f0 >= a.I) return;
  const uint16_t* w[2 * F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int i = min(f0 + f, a.I - 1);
    w[f] = a.w13 + (size_t)i * a.H;
    w[F + f] = a.w13 + (size_t)(a.I + i) * a.H;
  }
  float sum[2 * F][T];
#pragma unroll
  for (int f = 0; f < 2 * F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) sum[f][t] = 0.f;
  auto step = [&](int k) {
    u32x4 x[T], v[2 * F];
#pragma unroll
    for (int f = 0; f < 2 * F; ++f) v[f] = load16(w[f] + k);
#pragma unroll
    for (int t = 0; t < T; ++t) x[t] = load16(a.x + (size_t)t * a.H + k);
#pragma unroll
    for (int f = 0; f < 2 * F; ++f)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[f][t] = __builtin_fmaf(bf16_lo(x[t][j]), bf16_lo(v[f][j]), sum[f][t]);
          sum[f][t] = __builtin_fmaf(bf16_hi(x[t][j]), bf16_hi(v[f][j]), sum[f][t]);
        }
  };
  int k = 0;
#pragma unroll 4
  for (; k + 512 <= a.H; k += 512) step(k + lane * 8);
  if (k + lane * 8 < a.H) step(k + lane * 8);
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float g = wave_sum(sum[f][t]), u = wave_sum(sum[F + f][t]);
      if (lane == 0 && f0 + f < a.I)
        a.out[(size_t)t * a.I + f0 + f] = (uint16_t)f32_to_bf16(silu_mul(g, u));
    }
}

// Up to 16 FM rows: a workgroup takes 16 FF features, its four waves every
// fourth 128 elements of K each.  A wave copies its weight rows in runs of 256
// bytes into LDS of its own (no barriers), two pieces of K ahead, and reads them
// back as fragments; x comes from L2 straight into registers.  The waves' sums
// meet in LDS, in wave order.  (2048 x 5632: 16 rows 13.5 us, 32 15.3, 64 19.2;
// fragments straight from memory, 16 rows of 64 bytes an instruction: 16.7, 17.1
// and 21.4.)  More than 16 rows take 32 features, since x comes from L2 once for
// every workgroup: 64 rows 24.8 with 16.
constexpr int kRowsWaves = 4;
constexpr int kRowsK = 128;            // elements of K of a piece

template <int FM, int FF>
__global__ __launch_bounds__(64 * kRowsWaves, 1) void gated_rows_kernel(moe_host::GatedArgs a) {
  constexpr int kRows = 32 * FF;                 // gate rows, then up rows
  constexpr int kPiece = kRows * kRowsK * 2, kCopies = kRows / 4, kSteps = kRowsK / 32;
  constexpr int kSums = kRowsWaves * 2 * FF * FM * 1024;
  constexpr int kLds = kRowsWaves * 2 * kPiece;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds > kSums ? kLds : kSums];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int f0 = blockIdx.x * 16 * FF;
  // copy q takes rows 4 q .. 4 q + 3; 16-byte piece c of row r lies at c ^ (r & 15)
  const uint16_t* src[kCopies];
  int at_k[kCopies];
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int r = 4 * q + g, f = min(f0 + r % (16 * FF), a.I - 1);
    at_k[q] = 8 * (i ^ (r & 15));
    src[q] = a.w13 + (size_t)(r < 16 * FF ? f : a.I + f) * a.H + at_k[q];
  }
  const uint16_t* x[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) x[j] = a.x + (size_t)min(16 * j + i, a.M - 1) * a.H + 8 * g;
  uint8_t* mine = lds + wave * 2 * kPiece;
  const uint32_t mine_at = (uint32_t)(uintptr_t)(lds_void_t*)mine;
  const int pieces = ceil_div(a.H, kRowsK * kRowsWaves);
  // piece p of this wave; past the end of K zeros
  auto issue = [&](int p, u32x4 (&xv)[kSteps][FM]) {
    const int k0 = (p * kRowsWaves + wave) * kRowsK;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < FM; ++j)
        xv[s][j] = load16_or_zero(x[j] + k0 + 32 * s, k0 + 32 * s + 8 * g < a.H);
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      copy16(k0 + at_k[q] < a.H ? (const void*)(src[q] + k0) : (const void*)kZeroPage,
             mine_at + (p & 1) * kPiece + q * 1024);
  };
  f32x4 acc[2 * FF][FM];
#pragma unroll
  for (int f = 0; f < 2 * FF; ++f)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int p, const u32x4 (&xv)[kSteps][FM]) {
    // at most the next piece's copies are still on their way
    wait_vmem<kCopies>();
    asm volatile("" ::: "memory");
    const uint8_t* at = mine + (p & 1) * kPiece + i * 256;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 v[2 * FF];
#pragma unroll
      for (int f = 0; f < 2 * FF; ++f) v[f] = load16(at + f * 4096 + (((4 * s + g) ^ i) << 4));
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int f = 0; f < 2 * FF; ++f) acc[f][j] = mfma_16x16x32(v[f], xv[s][j], acc[f][j]);
    }
    wait_lgkm0();                                // the piece's LDS is free
    asm volatile("" ::: "memory");
  };
  u32x4 x0[kSteps][FM], x1[kSteps][FM];
  issue(0, x0);
  issue(1, x1);
#pragma unroll 1
  for (int p = 0; p < pieces; p += 2) {
    multiply(p, x0);
    issue(p + 2, x0);
    multiply(p + 1, x1);
    issue(p + 3, x1);
  }
  wait_vmem<0>();                                // the copies past the end
  __syncthreads();
  f32x4* red = reinterpret_cast<f32x4*>(lds);    // [wave][2 FF][FM][64]
#pragma unroll
  for (int f = 0; f < 2 * FF; ++f)
#pragma unroll
    for (int j = 0; j < FM; ++j)
      red[((wave * 2 * FF + f) * FM + j) * 64 + lane] = acc[f][j];
  __syncthreads();
#pragma unroll
  for (int e = wave; e < FF * FM; e += kRowsWaves) {
    const int f = e / FM, j = e % FM, m = 16 * j + i, n = f0 + f * 16 + 4 * g;
    f32x4 sg = red[(f * FM + j) * 64 + lane], su = red[((FF + f) * FM + j) * 64 + lane];
#pragma unroll
    for (int q = 1; q < kRowsWaves; ++q) {
      sg += red[((q * 2 * FF + f) * FM + j) * 64 + lane];
      su += red[((q * 2 * FF + FF + f) * FM + j) * 64 + lane];
    }
    if (m < a.M && n < a.I)
      *reinterpret_cast<u32x2*>(a.out + (size_t)m * a.I + n) =
          u32x2{pack_bf16x2(silu_mul(sg[0], su[0]), silu_mul(sg[1], su[1])),
                pack_bf16x2(silu_mul(sg[2], su[2]), silu_mul(sg[3], su[3]))};
  }
}

// out = bf16(sum of the splits, in their order); n a multiple of 8
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int splits,
                                                   size_t n, uint16_t* __restrict__ out) {
  for (size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; at < n;
       at += (size_t)gridDim.x * 2048) {
    f32x4 s[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
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

// Tile size and ranges of K of one product.  Tiles of 256 x 256 where half the
// chip has one (128 x 128 re-reads twice as much from L2 and LDS), 64 x 128 with
// stages of 64 k where 128 x 128 would leave half the chip without (2048 x 5632,
// 128 rows: 18 us against 27), and a product whose sum is all it stores is cut
// along K until every CU has a tile.  Stages of 64 k are whole 128-byte lines of
// the rows and half the barriers, but at 128 KB a CU the rings hold two to
// four of them: 64 x 128 tiles 18 us for 23 (eight stages of 32), 128 x 128 tiles
// slower (1000 rows x 1408 features 33 us for 23, four stages 25), 256 x 256 as
// well (4096 rows 175 for 168).  The waves of 64 x 128 are 64 x 64, two to each
// half of a stage's k: a third less of LDS is read than by 32 x 64 (509 rows x
// 1408 features 15.0 us for 16.3, 300 x 1024 of 4096 25.6 for 28.6;
// three stages 16.1 and 27.6).
struct Plan {
  bool big;                  // 256 x 256 tiles, else bm x 128
  int bm;
  int splits, k_per;
};
Plan plan_of(int rows, int n_rows, int K, bool can_split) {
  Plan p{true, 128, 1, 0};
  const int cu = kTileCus;
  const long long big = (long long)ceil_div_host(rows, 256) * ceil_div_host(n_rows, 256);
  p.big = big >= cu / 2;
  const long long tiles =
      p.big ? big : (long long)ceil_div_host(rows, 128) * ceil_div_host(n_rows, 128);
  const int stages = ceil_div_host(K, 32);
  if (can_split && tiles < cu) {
    // whole stages, at least 8 to a range
    const long long most = std::min(stages / 8, kMaxSplits), room = p.big ? kSplitTiles / 4 : kSmallSplitTiles;
    p.splits = (int)std::max<long long>(1, std::min(room / tiles, most));
  }
  p.k_per = ceil_div_host(stages, p.splits) * 32;
  p.splits = ceil_div_host(K, p.k_per);
  if (!can_split && !p.big && tiles <= cu / 2) p.bm = 64;
  return p;
}

template <Op kOp>
hipError_t launch_tiles(TileArgs a, int n_rows, bool can_split, hipStream_t s) {
  const Plan p = plan_of(a.rows, n_rows, a.K, can_split);
  a.splits = p.splits;
  a.k_per = p.k_per;
  a.tiles_m = ceil_div_host(a.rows, p.big ? 256 : p.bm);
  a.tiles_n = ceil_div_host(n_rows, p.big ? 256 : 128);
  TileArgs rest = a;
  const int last = a.tiles_m * a.tiles_n % kTileCus;
  const int whole = a.tiles_m * a.tiles_n / kTileCus * kTileCus / a.tiles_n;   // rows of tiles
  if (p.big && p.splits == 1 && whole > 0 && last > 0 && last <= kTileCus / 2) {
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
  if (p.big) {
    tile_kernel<256, 256, 32, 2, 4, 1, 4, kOp><<<grid, 512, 0, s>>>(a);
  } else if (p.bm == 64) {
    if constexpr (kOp == kAct || kOp == kGradAct)
      tile_kernel<64, 128, 64, 1, 2, 2, 4, kOp><<<grid, 256, 0, s>>>(a);
  } else {
    tile_kernel<128, 128, 32, 2, 2, 1, 4, kOp><<<grid, 256, 0, s>>>(a);
  }
  if (p.splits > 1) {
    const size_t n = (size_t)a.rows * a.cols;
    const unsigned g = (unsigned)std::min<size_t>((n / 8 + 255) / 256, 4096);
    join_kernel<<<g, 256, 0, s>>>(a.partial, p.splits, n, a.out);
  }
  const hipError_t err = hipGetLastError();
  return err != hipSuccess || rest.rows == 0 ? err : launch_tiles<kOp>(rest, n_rows, can_split, s);
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
    const int grid = ceil_div_host(a.I, 8 * kGemvFeatures);
    switch (a.M) {
      case 1: gated_gemv_kernel<1><<<grid, 512, 0, s>>>(a); break;
      case 2: gated_gemv_kernel<2><<<grid, 512, 0, s>>>(a); break;
      case 3: gated_gemv_kernel<3><<<grid, 512, 0, s>>>(a); break;
      default: gated_gemv_kernel<4><<<grid, 512, 0, s>>>(a); break;
    }
    return hipGetLastError();
  }
  if (a.M <= kFewRows) {
    if (a.M <= 16)
      gated_rows_kernel<1, 1><<<ceil_div_host(a.I, 16), 64 * kRowsWaves, 0, s>>>(a);
    else if (a.M <= 32)
      gated_rows_kernel<2, 2><<<ceil_div_host(a.I, 32), 64 * kRowsWaves, 0, s>>>(a);
    else
      gated_rows_kernel<4, 2><<<ceil_div_host(a.I, 32), 64 * kRowsWaves, 0, s>>>(a);
    return hipGetLastError();
  }
  TileArgs t{};
  t.m_side = a.x;
  t.n_side = a.w13;
  t.m_ld = t.n_ld = t.K = a.H;
  t.rows = a.M;
  t.cols = t.out_ld = a.I;
  t.out = a.out;
  return launch_tiles<kAct>(t, 2 * a.I, false, s);
}

hipError_t launch_zero(void* p, size_t bytes, hipStream_t s) {
  const size_t n = bytes / 16;
  zero_kernel<<<(unsigned)std::min<size_t>((n + 255) / 256, 4096), 256, 0, s>>>(
      static_cast<u32x4*>(p), n);
  return hipGetLastError();
}

// [d_gate d_up] [M, 2I], then the larger of the two products' partial sums
size_t gated_backward_bytes(int M, int H, int I) {
  return align256((size_t)M * 2 * I * 2) +
         std::max(partial_bytes(M, H), partial_bytes(2 * I, H));
}

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s) {
  uint16_t* d = static_cast<uint16_t*>(a.workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                            align256((size_t)a.M * 2 * a.I * 2));
  TileArgs t{};
  t.m_side = a.x;
  t.n_side = a.w13;
  t.m_ld = t.n_ld = t.K = a.H;
  t.rows = a.M;
  t.cols = a.I;
  t.grad_out = a.grad_out;
  t.out = d;
  t.out_ld = 2 * a.I;
  hipError_t err = launch_tiles<kGradAct>(t, 2 * a.I, false, s);
  if (err == hipSuccess && a.grad_x != nullptr) {
    TileArgs g{};
    g.m_side = d;
    g.n_side = a.w13;
    g.m_ld = g.K = 2 * a.I;
    g.n_ld = g.cols = g.out_ld = a.H;
    g.rows = a.M;
    g.out = a.grad_x;
    g.partial = partial;
    err = launch_tiles<kGradX>(g, a.H, true, s);
  }
  if (err == hipSuccess && a.grad_w13 != nullptr) {
    TileArgs g{};
    g.m_side = d;
    g.n_side = a.x;
    g.m_ld = g.rows = 2 * a.I;
    g.n_ld = g.cols = g.out_ld = a.H;
    g.K = a.M;
    g.out = a.grad_w13;
    g.partial = partial;
    err = launch_tiles<kGradW>(g, a.H, true, s);
  }
  return err;
}

}  // namespace moe_host
