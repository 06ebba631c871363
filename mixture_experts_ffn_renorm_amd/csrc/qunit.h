// Products of one 16-byte unit of packed 4-bit codes (32 elements, inside
// one group) with the matching bf16 elements, shared by the quantized GEMV
// kernels.
#pragma once

#include "moe_common.h"

namespace moe {

// 4-bit units on the bf16 dot-2 instruction: a code q in [0, 16) becomes the
// bf16 value 128 + q exactly (exponent of 128, q in the low mantissa bits),
// so a unit's codes turn into bf16 pairs with one shift and one and-or per
// pair, and sum (128 + q_i) x_i - 128 * sum x_i = sum q_i x_i.  Code word w
// holds elements 8w .. 8w + 7; its pair i (i < 4) takes elements i and
// i + 4 (bits 4i and 16 + 4i), and x is regrouped once per unit to match.

__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a),
                                         __builtin_bit_cast(bf16x2, b), c, false);
}

struct XPairs4 {
  uint32_t y[16];   // (x_i, x_{i+4}) of each 8-element word, as bf16 pairs
  float sx;         // sum of the unit's 32 x
};

__device__ __forceinline__ XPairs4 regroup_x4(const u32x4* xv) {
  XPairs4 r;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const u32x4 X = xv[w];   // (x0,x1) (x2,x3) (x4,x5) (x6,x7) of word w
    r.y[4 * w + 0] = __builtin_amdgcn_perm(X[2], X[0], 0x05040100u);   // (x0, x4)
    r.y[4 * w + 1] = __builtin_amdgcn_perm(X[2], X[0], 0x07060302u);   // (x1, x5)
    r.y[4 * w + 2] = __builtin_amdgcn_perm(X[3], X[1], 0x05040100u);   // (x2, x6)
    r.y[4 * w + 3] = __builtin_amdgcn_perm(X[3], X[1], 0x07060302u);   // (x3, x7)
#pragma unroll
    for (int j = 0; j < 4; ++j) s = dot2_bf16(X[j], 0x3f803f80u, s);   // (1, 1)
  }
  r.sx = s;
  return r;
}

// sum q_i x_i over one 4-bit unit
__device__ __forceinline__ float dot_unit4(const u32x4 codes, const XPairs4& xp) {
  float d = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d = dot2_bf16(((codes[w] >> (4 * i)) & 0x000f000fu) | 0x43004300u, xp.y[4 * w + i], d);
  return d - 128.f * xp.sx;
}

__device__ __forceinline__ float bf16_load(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

// 16 bytes at unit u of a row of units; past the row the load is clamped to
// unit 0 (in bounds; the caller drops that unit's contribution), so that all
// loads of a pass leave back to back with no branch between them
template <bool kStream>
__device__ __forceinline__ u32x4 load_unit(const u32x4* row, int u, int nunit) {
  const u32x4* p = row + (u < nunit ? u : 0);
  return kStream ? __builtin_nontemporal_load(p) : *p;
}

}  // namespace moe
