// Dense products with 4-bit weights in affine groups:
//   y[m, n] = sum_k x[m, k] (s[n, k / g] q[n, k] + b[n, k / g])
//   out = bf16(addend + row_scale[m] * y), or with `gated` SiLU(y[m, f]) *
//   y[m, N / 2 + f] in y's place (rows 0 .. N/2 - 1 the gate).
// Codes as in the group-quantized experts (least significant first in 32-bit
// words), groups of 32, 64 or 128 elements.
//
// The codes are never rounded: a code q becomes the bf16 value 128 + q
// exactly (q in the low mantissa bits of 128), the matrix cores form
// acc = sum (128 + q) x and sx = sum x over one group in fp32, and
//   s * sum q x + b * sum x = s * acc + (b - 128 s) * sx
// is added to the output's fp32 sum, two FMAs per group and output.
#include <algorithm>

#include "moe_common.h"
#include "qunit.h"

using namespace moe;

namespace {

// A 16-byte unit holds 32 codes of one weight row; a "block" is 128 codes of
// each of 16 rows: lane (r = lane % 16, g = lane / 16) loads unit g of row r
// (64 contiguous bytes per row).  An MFMA sums over the four lanes of a row,
// so the codes it takes have to belong to one group: for groups of 64 and 32
// the words are exchanged between the lanes of a row so that each word
// register holds one group (two or four lane-swap instructions per block).
constexpr int kBlockK = 128;

// Words of a block so that words [j * G/32, (j + 1) * G/32) are group j's.
template <int G>
__device__ __forceinline__ void group_words(u32x4& w) {
  uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
  if (G <= 64) {
    swap32(a, c);
    swap32(b, d);
  }
  if (G == 32) {
    swap16(a, b);
    swap16(c, d);
  }
  w = u32x4{a, b, c, d};
}

// 4 word + lane group of the operand that takes piece c (8 elements) of a
// block: where group_words puts the codes of elements 8 c .. 8 c + 7.
template <int G>
__device__ __forceinline__ int word_slot(int c) {
  if (G == 128) return ((c & 3) << 2) | (c >> 2);
  if (G == 64) return (c & 8) | ((c & 1) << 2) | (c & 2) | ((c >> 2) & 1);
  return c;
}

// The four lanes' values of a row, each in every lane of that row.
__device__ __forceinline__ void row_values(uint32_t own, uint32_t (&p)[4]) {
  uint32_t other = own;
  p[0] = own;
  swap32(p[0], other);
  p[1] = p[0];
  p[2] = p[3] = other;
  swap16(p[0], p[1]);
  swap16(p[2], p[3]);
}

// 8 codes as bf16 values 128 + q, pairs (i, i + 4).  The constants are kept
// in a scalar and a vector register, so that each pair is one and-or (two
// literals would not fit one instruction).
struct WidenConst {
  uint32_t mask, magic;
  __device__ __forceinline__ WidenConst() : mask(0x000f000fu), magic(0x43004300u) {
    asm("" : "+s"(mask));
    asm("" : "+v"(magic));
  }
};
__device__ __forceinline__ u32x4 widen8(uint32_t w, const WidenConst& k) {
  return u32x4{(w & k.mask) | k.magic, ((w >> 4) & k.mask) | k.magic,
               ((w >> 8) & k.mask) | k.magic, ((w >> 12) & k.mask) | k.magic};
}

// 8 consecutive bf16 elements in the same pairs (i, i + 4).
__device__ __forceinline__ u32x4 pair8(u32x4 X) {
  const bf16x8 v = __builtin_bit_cast(bf16x8, X);
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(v, v, 0, 4, 1, 5, 2, 6, 3, 7));
}

// The epilogue of one output value.
__device__ __forceinline__ void store_out(const moe_host::QLinearArgs& a, float y, int m, int n,
                                          int n_out) {
  const size_t at = (size_t)m * n_out + n;
  if (a.row_scale != nullptr) y *= a.row_scale[m];
  if (a.addend != nullptr) y += bf16_load(a.addend + at);
  a.out[at] = (uint16_t)f32_to_bf16(y);
}

// ---- GEMV: one or two tokens ----
//
// A lane keeps one unit (32 elements) of each token's x in registers, as the
// pairs that the codes widen to, and walks over weight rows: four rows at a
// time, the next four in flight, 1 KB of codes per row and wave.  Rows longer
// than 64 units are cut into `ns` slices of at most 64 units, one per wave
// (more than kGemvWaves slices: in turns, x read again).  The four rows' sums
// over the lanes share their first two steps (lane swaps), and the sums wait
// in LDS until the workgroup's rows are done.
//
// Bound by the codes' bytes where there are many (131072 x 2048, one token:
// 29 us, 5.2 TB/s, what a large copy reaches) and by launch, load and join
// where there are few (2048 x 2048: 3.9 us, of which an empty kernel takes 3).
// Two tokens: N = K = 8192 13.2 us against 14.0 with the row tiles below,
// N = 2048, K = 5632 5.3 / 8.1; three are faster there (13.5 / 16.3).
constexpr int kGemvWaves = 8;
constexpr int kGemvMaxRows = 64;   // weight rows per wave group

template <int T, bool kGated>
__global__ __launch_bounds__(64 * kGemvWaves) void qlinear_gemv_kernel(moe_host::QLinearArgs a,
                                                                       int ns, int nw,
                                                                       int chunks) {
  __shared__ float red[kGemvWaves][kGemvMaxRows * T];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (blockDim.x >> 6) / nw;               // wave groups per workgroup
  const int grp = wave / nw, w = wave % nw;
  const int n_out = kGated ? a.N / 2 : a.N;
  constexpr int kOut = kGated ? 2 : 4;                     // outputs per chunk of four rows
  const int o0 = (blockIdx.x * groups + grp) * chunks * kOut;
  const int upr = a.K / 32, gpr = a.K / a.group, sh = a.group == 32 ? 0 : a.group == 64 ? 1 : 2;
  const int ulen = ceil_div(upr, ns);
  const u32x4* q = reinterpret_cast<const u32x4*>(a.q);

  // row i of chunk c; rows past the end read the last one
  auto row_of = [&](int c, int i) {
    const int o = min(o0 + c * kOut + (kGated ? i & 1 : i), n_out - 1);
    return kGated && i >= 2 ? o + n_out : o;
  };
  for (int sl = w; sl < ns; sl += nw) {
    const int u = sl * ulen + lane;
    const bool ok = lane < ulen && u < upr;
    const int uc = ok ? u : 0;
    u32x4 cw[4];
    uint32_t cs[4], cb[4];
    auto load = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t n = (size_t)row_of(c, i);
        cw[i] = __builtin_nontemporal_load(q + n * upr + uc);
        cs[i] = a.scales[n * gpr + (uc >> sh)];
        cb[i] = a.biases[n * gpr + (uc >> sh)];
      }
    };
    load(0);
    XPairs4 xp[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const u32x4* xr =
          reinterpret_cast<const u32x4*>(a.x + (size_t)min(t, a.M - 1) * a.K) + (size_t)uc * 4;
      u32x4 xv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xv[i] = xr[i];
        if (!ok) xv[i] = u32x4{0u, 0u, 0u, 0u};
      }
      xp[t] = regroup_x4(xv);
    }
    const WidenConst wc;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      float y[T][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = __uint_as_float(cs[i] << 16);
        const float k = __builtin_fmaf(-128.f, s, __uint_as_float(cb[i] << 16));
        float d[T];
#pragma unroll
        for (int t = 0; t < T; ++t) d[t] = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const u32x4 p = widen8(cw[i][v], wc);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < T; ++t) d[t] = dot2_bf16(p[j], xp[t].y[4 * v + j], d[t]);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) y[t][i] = __builtin_fmaf(s, d[t], k * xp[t].sx);
      }
      load(min(c + 1, chunks - 1));
#pragma unroll
      for (int t = 0; t < T; ++t) {
        // four sums over 64 lanes -> one register: row of 16 lanes i holds sum i
        uint32_t b0 = __float_as_uint(y[t][0]), b1 = __float_as_uint(y[t][1]);
        uint32_t b2 = __float_as_uint(y[t][2]), b3 = __float_as_uint(y[t][3]);
        swap32(b0, b2);
        swap32(b1, b3);
        uint32_t e = __float_as_uint(__uint_as_float(b0) + __uint_as_float(b2));
        uint32_t o = __float_as_uint(__uint_as_float(b1) + __uint_as_float(b3));
        swap16(e, o);
        const float v = group_sum_last<16>(__uint_as_float(e) + __uint_as_float(o));
        if ((lane & 15) == 15) {
          float* r = &red[wave][t * kGemvMaxRows + 4 * c + (lane >> 4)];
          *r = sl == w ? v : *r + v;
        }
      }
    }
  }
  __syncthreads();
  // outputs of this wave group, over its own threads
  const int no = chunks * kOut;
  for (int i = w * 64 + lane; i < no * T; i += 64 * nw) {
    const int t = i / no, o = i - t * no;
    if (t >= a.M || o0 + o >= n_out) continue;
    const int at = t * kGemvMaxRows + (kGated ? 4 * (o >> 1) + (o & 1) : o);
    float y = 0.f, up = 0.f;
    for (int p = 0; p < nw; ++p) {
      y += red[grp * nw + p][at];
      if (kGated) up += red[grp * nw + p][at + 2];
    }
    if (kGated) y = silu_mul(y, up);
    store_out(a, y, t, o0 + o, n_out);
  }
}

template <int T, bool kGated>
hipError_t launch_gemv(const moe_host::QLinearArgs& a, hipStream_t s) {
  using moe_host::ceil_div_host;
  const int n_out = kGated ? a.N / 2 : a.N;
  constexpr int kOut = kGated ? 2 : 4;
  const int ns = ceil_div_host(a.K / 32, 64);
  const int nw = ns < kGemvWaves ? ns : kGemvWaves;
  const int groups = nw >= 4 ? 1 : 4 / nw;
  // chunks per wave group: about six waves for every SIMD
  const long long total = ceil_div_host(n_out, kOut);
  const long long want = 24LL * moe_host::device_cu_count() / nw;
  long long chunks = (total + want - 1) / want;
  if (chunks > kGemvMaxRows / 4) chunks = kGemvMaxRows / 4;
  const dim3 grid((unsigned)ceil_div_host((int)((total + chunks - 1) / chunks), groups));
  hipLaunchKernelGGL((qlinear_gemv_kernel<T, kGated>), grid, dim3(64 * nw * groups), 0, s, a, ns,
                     nw, (int)chunks);
  return hipGetLastError();
}

// ---- row-tile kernel: 3 to 16 tokens, and more where use_rows says so ----
//
// A wave keeps the x of 16 TM tokens and NB blocks (its slice of K) in
// registers as MFMA operands and walks over tiles of 16 weight rows, one
// tile's codes in flight while another is multiplied; the `nw` waves of a
// workgroup hold the slices of one K (in turns where there are more slices
// than waves).  A tile's sums wait in LDS until the workgroup's tiles are
// done and are then added over the waves.
//
// Memory is read in runs of a row (x 256 NB bytes, codes 64 NB bytes at a
// time) and turned to operands through the wave's own LDS: loads in operand
// order touch 16 rows each and took three times as long.
//
// A group's sum of x is formed once per slice (a product with ones) and kept.
// The codes' loads are ordinary ones: token tiles of one N share them in the
// caches (64 tokens, N = K = 8192 30 us, non-temporal 35), and one token tile
// gains as well (16 tokens 13.8 / 15.1).
//
// Up to 16 tokens bound by the latency of its loads: a workgroup reads all of
// its tokens' x before the first product.  16 tokens, N = 11264 gated, K =
// 2048, groups of 32: 8.8 us (1.7 TB/s); N = K = 8192: 13.8 us (2.7 TB/s).
// Above, by vector instructions (55 % of the time, matrix ones 18 %): 512
// tokens, N = 2048, K = 5632 32 us (370 TFLOP/s); 64 tokens, N = K = 8192
// 29.4 us.  Each 32 tokens widen the codes again.  Two to four tiles' codes in
// flight in place of one changed nothing.
constexpr int kRowsWaves = 8;
constexpr int kRowsLds = 160 * 1024;   // a workgroup's LDS at most

template <int G, int TM, int NB>
__global__ __launch_bounds__(64 * kRowsWaves) void qlinear_rows_kernel(moe_host::QLinearArgs a,
                                                                       int ns, int tiles,
                                                                       int wgs) {
  constexpr int NG = 128 / G;        // groups per block
  constexpr int NS = G / 32;         // MFMA steps per group
  constexpr int NGT = NB * NG;       // groups per slice
  constexpr int kPairs = (16 * NGT + 63) / 64;   // loads of (scale, bias) pairs per tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  uint8_t* own = lds + w * (NB * 4096);          // x, then each tile's codes and pairs
  f32x4* sums = reinterpret_cast<f32x4*>(lds + nw * (NB * 4096));   // [nw][tiles][TM][64]
  const int r = lane & 15, g = lane >> 4;
  const int n_out = a.gated ? a.N / 2 : a.N;
  const int upr = a.K / 32, gpr = a.K / G;
  // gated: tiles 2 j and 2 j + 1 are the gate and up rows of the same outputs
  const int t0 = blockIdx.x % wgs * tiles, m0 = blockIdx.x / wgs * (16 * TM);
  auto row_of = [&](int tile, int i) {
    const int o = (a.gated ? tile >> 1 : tile) * 16 + i;
    return min(o, n_out - 1) + (a.gated && (tile & 1) ? n_out : 0);
  };
  // codes piece u of row i in LDS: distinct banks for the 16 rows of an operand
  auto code_at = [&](int i, int u) {
    const int f = NB == 1 ? (0x78 >> ((i >> 2) * 2)) & 3 : (i >> 1) & 7;   // 0 2 3 1
    return i * (NB * 64) + ((u ^ f) << 4);
  };
  const WidenConst wc;
  const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  u32x4 cw[NB];
  uint32_t cs[kPairs], cb[kPairs];
  // the next piece to load: slice, tile
  int lsl = w, ltile = 0;
  auto load = [&]() {
    const int sl = lsl, tile = ltile;
    if (++ltile == tiles) {
      ltile = 0;
      lsl = min(lsl + nw, ns - 1);   // past the last slice: not used
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int p = 64 * i + lane, u = sl * NB * 4 + p % (NB * 4);
      // a unit past the row's end is read as unit 0; its x is 0
      cw[i] = *(reinterpret_cast<const u32x4*>(a.q) +
          (size_t)row_of(t0 + tile, p / (NB * 4)) * upr + (u < upr ? u : 0));
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int e = (64 * i + lane) % (16 * NGT), gi = sl * NGT + e % NGT;
      const size_t at = (size_t)row_of(t0 + tile, e / NGT) * gpr + (gi < gpr ? gi : 0);
      cs[i] = a.scales[at];
      cb[i] = a.biases[at];
    }
  };
  u32x4 xv[TM][4 * NB];
  auto load_x = [&](int sl) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int i = 0; i < 4 * NB; ++i) {
        const int p = 64 * i + lane, m = p / (16 * NB);
        const int k = sl * NB * kBlockK + p % (16 * NB) * 8;
        xv[t][i] = load16_or_zero(a.x + (size_t)min(m0 + 16 * t + m, a.M - 1) * a.K + k, k < a.K);
      }
  };
  load_x(w);
  load();
  u32x4 xp[TM][NB][4];
  f32x4 sx[TM][NGT];   // each group's sums of x
  int sl = w, tile = 0;
  auto turn_x = [&]() {
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      // as in the tile kernel: piece of word st, lane group g at (4 st + g) ^ m
#pragma unroll
      for (int i = 0; i < 4 * NB; ++i) {
        const int p = 64 * i + lane, m = p / (16 * NB), c = p % (16 * NB);
        *reinterpret_cast<u32x4*>(own + m * (NB * 256) + (c >> 4) * 256 +
                                  ((word_slot<G>(c & 15) ^ m) << 4)) = pair8(xv[t][i]);
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int st = 0; st < 4; ++st)
          xp[t][b][st] = *reinterpret_cast<const u32x4*>(own + r * (NB * 256) + b * 256 +
                                                         (((4 * st + g) ^ r) << 4));
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int j = 0; j < NGT; ++j) {
        sx[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NS; ++i)
          sx[t][j] = mfma_16x16x32(xp[t][j / NG][j % NG * NS + i], ones, sx[t][j]);
      }
    // the next turn's x (past the last: not used)
    load_x(min(sl + nw, ns - 1));
  };
#pragma unroll 1
  while (sl < ns) {
    if (tile == 0) turn_x();
    uint32_t* pl = reinterpret_cast<uint32_t*>(own + NB * 1024);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int p = 64 * i + lane;
      *reinterpret_cast<u32x4*>(own + code_at(p / (NB * 4), p % (NB * 4))) = cw[i];
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) pl[(64 * i + lane) % (16 * NGT)] = cs[i] | (cb[i] << 16);
    __builtin_amdgcn_wave_barrier();
    u32x4 wd[NB];
    uint32_t pair[NGT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      wd[b] = *reinterpret_cast<const u32x4*>(own + code_at(r, 4 * b + g));
#pragma unroll
    for (int j = 0; j < NGT; ++j) pair[j] = pl[r * NGT + j];
    __builtin_amdgcn_wave_barrier();
    load();
    f32x4 tot[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) tot[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      group_words<G>(wd[b]);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        f32x4 acc[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const u32x4 wv = widen8(wd[b][j * NS + i], wc);
#pragma unroll
          for (int t = 0; t < TM; ++t) acc[t] = mfma_16x16x32(xp[t][b][j * NS + i], wv, acc[t]);
        }
        const float s = bf16_lo(pair[b * NG + j]);
        const float c = __builtin_fmaf(-128.f, s, bf16_hi(pair[b * NG + j]));
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            tot[t][q] = __builtin_fmaf(s, acc[t][q], __builtin_fmaf(c, sx[t][b * NG + j][q], tot[t][q]));
      }
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      f32x4* p = sums + ((size_t)(w * tiles + tile) * TM + t) * 64 + lane;
      *p = sl == w ? tot[t] : *p + tot[t];
    }
    if (++tile == tiles) {
      tile = 0;
      sl += nw;
    }
  }
  __syncthreads();
  // lane: weight row r of a tile, tokens 4 g .. 4 g + 3 of a token tile
  const int per = a.gated ? 2 : 1;
  for (int i = threadIdx.x; i < tiles / per * TM * 64; i += blockDim.x) {
    const int ln = i & 63, t = (i >> 6) % TM, tile = (i >> 6) / TM * per;
    f32x4 y = {0.f, 0.f, 0.f, 0.f}, up = y;
    for (int p = 0; p < nw; ++p) {
      y += sums[((p * tiles + tile) * TM + t) * 64 + ln];
      if (a.gated) up += sums[((p * tiles + tile + 1) * TM + t) * 64 + ln];
    }
    const int o = (t0 + tile) / per * 16 + (ln & 15);
    if (o >= n_out) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + 16 * t + 4 * (ln >> 4) + q;
      if (m < a.M) store_out(a, a.gated ? silu_mul(y[q], up[q]) : y[q], m, o, n_out);
    }
  }
}

template <int G, int TM, int NB>
hipError_t launch_rows_nb(const moe_host::QLinearArgs& a, hipStream_t s) {
  using moe_host::ceil_div_host;
  const int per = a.gated ? 2 : 1;
  const int total = ceil_div_host(a.gated ? a.N / 2 : a.N, 16) * per;
  const int ns = ceil_div_host(ceil_div_host(a.K, kBlockK), NB);
  const int nw = ns < kRowsWaves ? ns : kRowsWaves;
  // tiles per workgroup: about two waves for every SIMD, as far as LDS holds
  // the sums (gated: whole pairs of tiles)
  const int mtile = ceil_div_host(a.M, 16 * TM);
  const long long want = 8LL * moe_host::device_cu_count() / nw;
  int tiles = (int)(((long long)total * mtile + want - 1) / want);
  const int most = (kRowsLds - nw * NB * 4096) / (nw * TM * 1024) / per * per;
  // no more than there are: 65536 tokens, N = 16, K = 512 17 us, 101 with
  // tiles past the last row multiplied and dropped
  tiles = std::min((tiles + per - 1) / per * per, total);
  // as few full rounds of workgroups as LDS allows, and none nearly empty (64
  // tokens, N = 11264 gated, K = 2048: 13 us in one round, 19 in one and a half)
  const int turns = ceil_div_host(tiles, most);
  tiles = ceil_div_host(ceil_div_host(tiles, turns), per) * per;
  while ((long long)ceil_div_host(total, tiles) * mtile > want * turns &&
         tiles < std::min(most, total))
    tiles += per;
  static bool set[moe_host::kMaxDevices] = {};
  const hipError_t e = moe_host::ensure_dynamic_lds(
      reinterpret_cast<const void*>(&qlinear_rows_kernel<G, TM, NB>), kRowsLds, set);
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)nw * (NB * 4096 + tiles * TM * 1024);
  const int wgs = ceil_div_host(total, tiles);
  hipLaunchKernelGGL((qlinear_rows_kernel<G, TM, NB>), dim3((unsigned)wgs * mtile), dim3(64 * nw),
                     lds, s, a, ns, tiles, wgs);
  return hipGetLastError();
}

template <int G>
hipError_t launch_rows(const moe_host::QLinearArgs& a, hipStream_t s) {
  if (a.M > 16) return launch_rows_nb<G, 2, 1>(a, s);
  // One block per wave where eight waves hold all of K and a CU has few codes
  // to read.  Measured us, one / two blocks: K = 512, N = 8192 4.4 / 5.1,
  // 65536 9.0 / 8.7; K = 1024, N = 2048 4.3 / 4.4, 65536 14.7 / 12.0; K = 2048,
  // N = 11264 8.3 / 7.2; N = K = 8192 16.3 / 14.0.
  if (a.K <= kRowsWaves * kBlockK &&
      (long long)a.N * a.K <= 32768LL * moe_host::device_cu_count())
    return launch_rows_nb<G, 1, 1>(a, s);
  return launch_rows_nb<G, 1, 2>(a, s);
}

// ---- tile kernel: many tokens ----
//
// A workgroup owns 64 tokens and 32 weight rows per wave (gated: 16 gate rows
// and their 16 up rows); K goes by in stages of 256.  x passes through LDS
// once per workgroup: each 16-byte piece is put into the codes' pair order on
// the way and summed over its group.  The piece that word w of lane group g
// multiplies lies at slot (4 w + g) ^ (m & 15) of token m's half row: with g
// in the low bits, the lanes that one LDS cycle serves fall on distinct banks
// (with g in the high bits a sixth of the kernel's time went to conflicts).
// A wave's codes go from memory to registers one stage ahead.
//
// The group sums' term, sum_j b_j sx_j - 128 s_j sx_j, is a product over the
// groups of its own: sx in three bf16 parts (24 bits), against the bf16 b and
// s themselves, eight k slots per group [b b b s s s 0 0] x
// [h m l -128h -128m -128l 0 0], so one more MFMA step per four groups adds it
// to the fp32 sums, where FMAs would cost as much vector time as the scaling.
//
// 2048 tokens, N = 2048, K = 5632, groups of 128: 63 us (750 TFLOP/s; a
// large library product in bf16 reaches 1204), groups of 64 68 us, of 32 85.
// Bound by the two waves that a SIMD holds: matrix instructions fill 36 % of
// its time, vector ones (widening, scaling, staging) 51 %, and overlap them in
// part.  Tiles of 64 x 64 per wave, one wave a SIMD, took 95 us; 32 tokens per
// wave and four waves a SIMD 75; both blocks of a stage unrolled up to 2.4
// times.
constexpr int kTileM = 64;
constexpr int kTileK = 256;
constexpr int kTileX = kTileM * kTileK * 2;      // bytes of x per stage
constexpr int kTileOut = 36;                     // floats from token to token in the epilogue

template <int G, int W>
__global__ __launch_bounds__(64 * W) void qlinear_tile_kernel(moe_host::QLinearArgs a, int ntile) {
  constexpr int NG = kTileK / G;                  // groups per stage
  constexpr int NX = (NG + 3) / 4;                // steps of the sums' product
  constexpr int NS = G / 32;                      // MFMA steps per group
  constexpr int F = 2;                            // row fragments per wave
  constexpr int kSums = NX * 4 * kTileM * 16;     // bytes of sums per stage
  constexpr int kStage = kTileX + kSums;
  static_assert(W * kTileM * kTileOut * 4 <= 2 * kStage + W * 4096, "the epilogue's LDS");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n_out = a.gated ? a.N / 2 : a.N;
  const int wg_n = ceil_div(ntile, W);
  const int id = xcd_contiguous_tile(blockIdx.x, wg_n * ceil_div(a.M, kTileM));
  if (id < 0) return;                             // whole workgroup
  const int m0 = id / wg_n * kTileM;
  const int n0 = (id % wg_n * W + wave) * (a.gated ? 8 * F : 16 * F);   // past the end: not stored
  const int upr = a.K / 32, gpr = a.K / G;
  const int nstage = ceil_div(a.K, kTileK);

  // weight row i of this wave: row i % 16 of fragment i / 16 (gated: the
  // first half of the fragments gates, the second their up rows)
  auto row_of = [&](int i) {
    return min(n0 + (a.gated ? i % (8 * F) : i), n_out - 1) + (a.gated && i >= 8 * F ? n_out : 0);
  };
  // A stage holds 128 bytes of codes per row: eight lanes load a row's
  // (whole cache lines), and the operands are
  // read back from the wave's own LDS (piece c of row i at c ^ ((i >> 1) & 7):
  // 16 rows of an operand fall on distinct banks).  Scales and biases: four
  // lanes load a row's four groups.
  //
  // Addresses are a uniform base that moves with the stage and a 32-bit lane
  // offset that does not (a tile's rows span less than 4 GB).
  const int lrow = lane >> 3, lpc = lane & 7;
  const char *wbase[F], *sbase[F], *bbase[F];
  uint32_t woff[2 * F], soff[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const size_t row0 = (size_t)row_of(16 * f);
    wbase[f] = reinterpret_cast<const char*>(a.q) + row0 * upr * 16;
    sbase[f] = reinterpret_cast<const char*>(a.scales + row0 * gpr);
    bbase[f] = reinterpret_cast<const char*>(a.biases + row0 * gpr);
#pragma unroll
    for (int i = 2 * f; i < 2 * f + 2; ++i)
      woff[i] = ((uint32_t)(row_of(8 * i + lrow) - row_of(16 * f)) * upr + lpc) * 16;
    soff[f] = ((uint32_t)(row_of(16 * f + (lane >> 2)) - row_of(16 * f)) * gpr +
               (lane & (NG < 4 ? NG - 1 : 3))) * 2;
  }
  uint8_t* wl = lds + 2 * kStage + wave * (F * 2048);
  // x: 32 pieces of 8 elements per token and stage; a row of 16 lanes takes
  // half a token's, so a piece's group lies inside its row of lanes
  constexpr int kPer = kTileM * kTileK / 8 / (64 * W);   // pieces per thread
  const char* xbase = reinterpret_cast<const char*>(a.x + (size_t)m0 * a.K);
  uint32_t xoff[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = i * 64 * W + tid;
    xoff[i] = (uint32_t)min(p >> 5, a.M - 1 - m0) * (uint32_t)a.K * 2 + (p & 31) * 16;
  }
  u32x4 xr[kPer];
  u32x4 wn[2 * F];
  uint32_t sn[F][NX], bn[F][NX];
  auto load = [&](int st) {
    if ((st + 1) * kTileK <= a.K) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) xr[i] = load16(xbase + st * (kTileK * 2) + xoff[i]);
#pragma unroll
      for (int i = 0; i < 2 * F; ++i)
        wn[i] = load16(wbase[i / 2] + st * (kTileK / 2) + woff[i]);
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < NX; ++j) {
          sn[f][j] = *reinterpret_cast<const uint16_t*>(sbase[f] + (st * NG + 4 * j) * 2 + soff[f]);
          bn[f][j] = *reinterpret_cast<const uint16_t*>(bbase[f] + (st * NG + 4 * j) * 2 + soff[f]);
        }
    } else {
      // the last, shorter stage: x past K is 0, codes and groups past it are
      // read from the row's start
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = st * kTileK + ((i * 64 * W + tid) & 31) * 8 < a.K;
        xr[i] = load16_or_zero(xbase + (in ? (uint32_t)(st * (kTileK * 2)) + xoff[i] : 0u), in);
      }
      const uint32_t u = st * (kTileK / 32) + lpc < upr ? st * (kTileK / 2) : -lpc * 16;
#pragma unroll
      for (int i = 0; i < 2 * F; ++i) wn[i] = load16(wbase[i / 2] + (woff[i] + u));
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < NX; ++j) {
          const int gl = lane & (NG < 4 ? NG - 1 : 3);
          const uint32_t at = soff[f] + (uint32_t)(st * NG + 4 * j + gl < gpr
                                                       ? (st * NG + 4 * j) * 2 : -gl * 2);
          sn[f][j] = *reinterpret_cast<const uint16_t*>(sbase[f] + at);
          bn[f][j] = *reinterpret_cast<const uint16_t*>(bbase[f] + at);
        }
    }
  };
  auto store_w = [&]() {
#pragma unroll
    for (int i = 0; i < 2 * F; ++i) {
      const int row = 8 * i + lrow;
      *reinterpret_cast<u32x4*>(wl + row * 128 + ((lpc ^ ((row >> 1) & 7)) << 4)) = wn[i];
    }
  };
  auto store_x = [&](int st) {
    uint8_t* buf = lds + (st & 1) * kStage;
    // a piece's group sum is in every lane of the group; lane i of a group
    // keeps the i-th piece's, so that the parts are formed once
    constexpr int kLanes = G / 8;                 // lanes of a group: 4, 8 or 16
    const int mine = lane & (kLanes - 1);
    float sum[(kPer + kLanes - 1) / kLanes];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = i * 64 * W + tid, m = p >> 5, c = p & 31;
      *reinterpret_cast<u32x4*>(buf + m * 512 + (c >> 4) * 256 +
                                ((word_slot<G>(c & 15) ^ (m & 15)) << 4)) = pair8(xr[i]);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s = dot2_bf16(xr[i][j], 0x3f803f80u, s);
      s = dpp_add_with<0xb1>(s);                 // quad_perm [1, 0, 3, 2]
      s = dpp_add_with<0x4e>(s);                 // quad_perm [2, 3, 0, 1]
      if (G >= 64) s = dpp_add_with<0x141>(s);   // row_half_mirror
      if (G == 128) s = dpp_add_with<0x140>(s);  // row_mirror
      sum[i / kLanes] = i % kLanes == 0 || mine == i % kLanes ? s : sum[i / kLanes];
    }
#pragma unroll
    for (int v = 0; v < kPer; v += kLanes)
      if (v + mine < kPer) {
        const int p = (v + mine) * 64 * W + tid, m = p >> 5, c = p & 31;
        const float s = sum[v / kLanes];
        const float h = bf16_lo(f32_to_bf16(s));
        const float mid = bf16_lo(f32_to_bf16(s - h));
        const float lo = s - h - mid;
        *reinterpret_cast<u32x4*>(buf + kTileX + ((c / kLanes) * kTileM + m) * 16) =
            u32x4{pack_bf16x2(h, mid), pack_bf16x2(lo, -128.f * h),
                  pack_bf16x2(-128.f * mid, -128.f * lo), 0u};
      }
  };

  const WidenConst wc;
  f32x4 tot[F][4];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int t = 0; t < 4; ++t) tot[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // group slots that no group fills (G = 128): zero in both buffers
  if (NX * 4 > NG)
    for (int i = tid; i < 2 * (NX * 4 - NG) * kTileM; i += blockDim.x)
      *reinterpret_cast<u32x4*>(lds + (i & 1) * kStage + kTileX + (NG * kTileM + (i >> 1)) * 16) =
          u32x4{0u, 0u, 0u, 0u};

  load(0);
  store_x(0);
  store_w();
  __syncthreads();
#pragma unroll 1
  for (int st = 0; st < nstage; ++st) {
    const uint8_t* buf = lds + (st & 1) * kStage;
    u32x4 w[F][2];
    uint32_t pr[F][NX];
#pragma unroll
    for (int f = 0; f < F; ++f) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        w[f][b] = *reinterpret_cast<const u32x4*>(
            wl + (16 * f + r) * 128 + (((4 * b + g) ^ ((r >> 1) & 7)) << 4));
        group_words<G>(w[f][b]);
      }
      // from lane 4 r + g to lane r + 16 g
#pragma unroll
      for (int j = 0; j < NX; ++j)
        pr[f][j] = (uint32_t)__shfl((int)(sn[f][j] | (bn[f][j] << 16)), 4 * r + g, kWave);
    }
    const int next = min(st + 1, nstage - 1);
    load(next);
    uint32_t pair[F][NX * 4];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        uint32_t p[4];
        row_values(pr[f][j], p);
#pragma unroll
        for (int i = 0; i < 4; ++i) pair[f][4 * j + i] = p[i];
      }
    // the wave that multiplies goes before the one that stages (2%)
    __builtin_amdgcn_s_setprio(1);
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      if (NX == 2 || b == 0) {
        // the sums' product for four groups
        u32x4 bx[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const uint32_t p = pr[f][0];
          bx[f] = u32x4{__builtin_amdgcn_perm(p, p, 0x07060706u),    // b b
                        __builtin_amdgcn_perm(p, p, 0x05040706u),    // b s
                        __builtin_amdgcn_perm(p, p, 0x05040504u),    // s s
                        0u};
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const u32x4 ax = *reinterpret_cast<const u32x4*>(
              buf + kTileX + ((4 * b + g) * kTileM + 16 * t + r) * 16);
#pragma unroll
          for (int f = 0; f < F; ++f) tot[f][t] = mfma_16x16x32(ax, bx[f], tot[f][t]);
        }
      }
#pragma unroll
      for (int j = 0; j < NG / 2; ++j) {          // groups of this block
        f32x4 acc[F][4];
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int word = j * NS + i;
          u32x4 wv[F];
#pragma unroll
          for (int f = 0; f < F; ++f) wv[f] = widen8(w[f][0][word], wc);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const u32x4 ax = *reinterpret_cast<const u32x4*>(
                buf + (16 * t + r) * 512 + b * 256 + (((4 * word + g) ^ r) << 4));
#pragma unroll
            for (int f = 0; f < F; ++f) acc[f][t] = mfma_16x16x32(ax, wv[f], acc[f][t]);
          }
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const float s = bf16_lo(pair[f][j]);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) tot[f][t][q] = __builtin_fmaf(s, acc[f][t][q], tot[f][t][q]);
        }
      }
      // the second block in the first one's registers
#pragma unroll
      for (int f = 0; f < F; ++f) {
        w[f][0] = w[f][1];
        pr[f][0] = pr[f][NX - 1];
#pragma unroll
        for (int j = 0; j < NG / 2; ++j) pair[f][j] = pair[f][NG / 2 + j];
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (st + 1 < nstage) {
      store_x(st + 1);
      store_w();
    }
    __syncthreads();
  }
  // The sums go through LDS (every wave is past its last stage) to lanes that
  // hold eight consecutive outputs of a token: 16-byte loads and stores in
  // place of 2-byte ones (2048 x 8192 outputs, K = 512, with an addend: 41.4 us,
  // 43.8 before).
  float* yl = reinterpret_cast<float*>(lds) + wave * (kTileM * kTileOut);
#pragma unroll
  for (int f = 0; f < F; ++f) {
    if (a.gated && f >= F / 2) break;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        yl[(16 * t + 4 * g + q) * kTileOut + 16 * f + r] =
            a.gated ? silu_mul(tot[f][t][q], tot[f | (F / 2)][t][q]) : tot[f][t][q];
  }
  __builtin_amdgcn_wave_barrier();
  const int sh = a.gated ? 1 : 2;                 // pieces of a token: 2 or 4
  const bool whole = n_out % 8 == 0;
  u32x4 ad[4];
  float rs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 64 * i + lane, m = m0 + (p >> sh), n = n0 + (p & ((1 << sh) - 1)) * 8;
    const bool in = m < a.M && n < n_out && p < kTileM << sh;
    ad[i] = load16_or_zero(a.addend + (in ? (size_t)m * n_out + n : 0),
                           in && whole && a.addend != nullptr);
    rs[i] = in && a.row_scale != nullptr ? a.row_scale[m] : 1.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = 64 * i + lane, m = m0 + (p >> sh), n = n0 + (p & ((1 << sh) - 1)) * 8;
    if (m >= a.M || n >= n_out || p >= kTileM << sh) continue;
    const f32x4* from = reinterpret_cast<const f32x4*>(
        yl + (p >> sh) * kTileOut + (p & ((1 << sh) - 1)) * 8);
    const f32x4 y[2] = {from[0], from[1]};
    const size_t at = (size_t)m * n_out + n;
    if (whole) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v0 = y[j / 2][2 * (j % 2)] * rs[i], v1 = y[j / 2][2 * (j % 2) + 1] * rs[i];
        if (a.addend != nullptr) v0 += bf16_lo(ad[i][j]), v1 += bf16_hi(ad[i][j]);
        o[j] = pack_bf16x2(v0, v1);
      }
      *reinterpret_cast<u32x4*>(a.out + at) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < n_out) {
          float v = y[j / 4][j % 4] * rs[i];
          if (a.addend != nullptr) v += bf16_load(a.addend + at + j);
          a.out[at + j] = (uint16_t)f32_to_bf16(v);
        }
    }
  }
}

template <int G, int W>
hipError_t launch_tile_waves(const moe_host::QLinearArgs& a, hipStream_t s) {
  using moe_host::ceil_div_host;
  constexpr int NX = (kTileK / G + 3) / 4;
  constexpr int kLds = 2 * (kTileX + NX * 4 * kTileM * 16) + W * 4096;
  static bool set[moe_host::kMaxDevices] = {};
  const hipError_t e = moe_host::ensure_dynamic_lds(
      reinterpret_cast<const void*>(&qlinear_tile_kernel<G, W>), kLds, set);
  if (e != hipSuccess) return e;
  const int ntile = ceil_div_host(a.gated ? a.N / 2 : a.N, a.gated ? 16 : 32);
  const int tiles = ceil_div_host(ntile, W) * ceil_div_host(a.M, kTileM);
  hipLaunchKernelGGL((qlinear_tile_kernel<G, W>), dim3((unsigned)ceil_div_host(tiles, 8) * 8),
                     dim3(64 * W), kLds, s, a, ntile);
  return hipGetLastError();
}

// Eight waves share a stage of x; four where that leaves CUs without work
// (measured us, eight / four: 2048 tokens, N = 2048, K = 5632 69 / 122; 1024
// tokens 66 / 62; 256 tokens, N = K = 8192 96 / 88).
int tile_waves(const moe_host::QLinearArgs& a) {
  using moe_host::ceil_div_host;
  return ceil_div_host(a.N, 256) * ceil_div_host(a.M, kTileM) >= moe_host::device_cu_count() ? 8 : 4;
}

template <bool kGated>
hipError_t launch_few(const moe_host::QLinearArgs& a, hipStream_t s) {
  if (a.M == 1) return launch_gemv<1, kGated>(a, s);
  return launch_gemv<2, kGated>(a, s);
}

// The row tiles' time grows with 32-token tiles times rows, the LDS tiles'
// with rounds of workgroups over the CUs, one a CU; both with K.  One round
// takes as long as the row tiles need for about 200 rows per CU (measured us,
// row / LDS tiles, K = 5632, N = 2048: 128 tokens 15 / 61, 512 34 / 62, 768
// 59 / 63; N = K = 8192: 64 tokens 30 / 86, 128 48 / 87, 192 84 / 88, 256
// 92 / 89; K = 2048: 1024 tokens, N = 2048 30 / 26).
bool use_rows(const moe_host::QLinearArgs& a) {
  using moe_host::ceil_div_host;
  const int cus = moe_host::device_cu_count();
  const long long wgs =
      (long long)ceil_div_host(a.N, 32 * tile_waves(a)) * ceil_div_host(a.M, kTileM);
  const long long rounds = (wgs + cus - 1) / cus;
  return (long long)ceil_div_host(a.M, 32) * a.N < rounds * 200 * cus;
}

template <int G>
hipError_t launch_group(const moe_host::QLinearArgs& a, hipStream_t s) {
  if (a.M <= 16 || use_rows(a)) return launch_rows<G>(a, s);
  if (tile_waves(a) == 8) return launch_tile_waves<G, 8>(a, s);
  return launch_tile_waves<G, 4>(a, s);
}

}  // namespace

namespace moe_host {

hipError_t launch_qlinear(const QLinearArgs& a, hipStream_t s) {
  if (a.M <= 2) return a.gated ? launch_few<true>(a, s) : launch_few<false>(a, s);
  switch (a.group) {
    case 32: return launch_group<32>(a, s);
    case 64: return launch_group<64>(a, s);
    default: return launch_group<128>(a, s);
  }
}

}  // namespace moe_host
