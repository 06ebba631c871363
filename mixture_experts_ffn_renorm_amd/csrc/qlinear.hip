// Dense products with 4-bit weights in affine groups:
//   y[m, n] = sum_k x[m, k] (s[n, k / g] q[n, k] + b[n, k / g])
//   out = bf16(addend + row_scale[m] * y), or with `gated` SiLU(y[m, f]) *
//   y[m, N / 2 + f] in y's place (rows 0 .. N/2 - 1 the gate).
// Codes as in the group-quantized experts (least significant first in 32-bit
// words), groups of 32, 64 or 128 elements; the codes are never rounded:
// sum_k x w = s * sum q x + b * sum x inside a group, accumulated in fp32.
#include "moe_common.h"
#include "qunit.h"

using namespace moe;

namespace {

constexpr int kLinWaves = 4;
constexpr int kLinTokens = 4;

// The epilogue of one output value.
__device__ __forceinline__ void store_out(float y, const float* row_scale, const uint16_t* addend,
                                          uint16_t* out, size_t m, size_t at) {
  if (row_scale != nullptr) y *= row_scale[m];
  if (addend != nullptr) y += bf16_load(addend + at);
  out[at] = (uint16_t)f32_to_bf16(y);
}

// One output column (a row of W, or a gate row and its up row) per wave, up
// to kLinTokens tokens; lane l takes units l, l + 64, ...
template <bool kGated>
__global__ __launch_bounds__(64 * kLinWaves) void qlinear_gemv_kernel(moe_host::QLinearArgs a) {
  const int lane = threadIdx.x & 63;
  const int n_out = kGated ? a.N / 2 : a.N;
  const int ncol = ceil_div(n_out, kLinWaves);
  const int bx = blockIdx.x % ncol;
  const int m0 = blockIdx.x / ncol * kLinTokens;
  const int f = bx * kLinWaves + (threadIdx.x >> 6);
  if (f >= n_out) return;   // whole wave; no barrier follows
  constexpr int R = kGated ? 2 : 1;
  const int nunit = a.K / 32, ng = a.K / a.group, upg = a.group / 32;
  float acc[R][kLinTokens];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int u = 0; u < kLinTokens; ++u) acc[r][u] = 0.f;
  for (int u = lane; u < nunit; u += 64) {
    XPairs4 xp[kLinTokens];
#pragma unroll
    for (int v = 0; v < kLinTokens; ++v) {
      const int m = m0 + v < a.M ? m0 + v : 0;
      const u32x4* xr = reinterpret_cast<const u32x4*>(a.x + (size_t)m * a.K) + (size_t)u * 4;
      u32x4 xv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = xr[i];
      xp[v] = regroup_x4(xv);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const size_t row = (size_t)f + (size_t)r * n_out;
      const u32x4 c = reinterpret_cast<const u32x4*>(a.q)[row * nunit + u];
      const float s = bf16_load(a.scales + row * ng + u / upg);
      const float b = bf16_load(a.biases + row * ng + u / upg);
#pragma unroll
      for (int v = 0; v < kLinTokens; ++v) acc[r][v] += s * dot_unit4(c, xp[v]) + b * xp[v].sx;
    }
  }
#pragma unroll
  for (int v = 0; v < kLinTokens; ++v) {
    float y = wave_sum(acc[0][v]);
    if (kGated) y = silu_mul(y, wave_sum(acc[R - 1][v]));
    if (lane == 0 && m0 + v < a.M)
      store_out(y, a.row_scale, a.addend, a.out, m0 + v, (size_t)(m0 + v) * n_out + f);
  }
}

}  // namespace

namespace moe_host {

hipError_t launch_qlinear(const QLinearArgs& a, hipStream_t s) {
  const int n_out = a.gated ? a.N / 2 : a.N;
  const dim3 grid((unsigned)ceil_div_host(n_out, kLinWaves) * ceil_div_host(a.M, kLinTokens));
  if (a.gated)
    hipLaunchKernelGGL(qlinear_gemv_kernel<true>, grid, dim3(64 * kLinWaves), 0, s, a);
  else
    hipLaunchKernelGGL(qlinear_gemv_kernel<false>, grid, dim3(64 * kLinWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe_host
