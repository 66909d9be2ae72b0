// The product with its epilogue, in its simplest form: a workgroup of four
// waves owns a 64 x 64 output tile and walks k in slices of 32 through one LDS
// stage, converting operands to bf16 on the way in (exact for e4m3).
#include "layer_device.hpp"

namespace ptg {

__device__ __forceinline__ float ep_load(const void *p, int32_t type, int64_t i) {
  return type == kTypeF32 ? ((const float *)p)[i] : (float)((const __bf16 *)p)[i];
}

template <int FORM>
__global__ __launch_bounds__(256) void ptg_product_simple_kernel(const ProductArgs g) {
  constexpr bool AT = FORM == kFormTN, BT = FORM == kFormNT || FORM == kFormNTE4m3, E8 = FORM == kFormNTE4m3;
  __shared__ __attribute__((aligned(16))) __bf16 sa[64][40], sb[64][40];
  const int32_t tid = (int32_t)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
  auto element = [&](const void *p, bool k_major, int64_t ld, int64_t row, int64_t rows, int32_t k) -> __bf16 {
    if (row >= rows || k >= g.k) return (__bf16)0.0f;
    const int64_t i = k_major ? (int64_t)k * ld + row : row * ld + k;
    if constexpr (E8) return (__bf16)__builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t *)p)[i], 0);
    return ((const __bf16 *)p)[i];
  };
  f32x4 acc[4] = {};
  for (int32_t k0 = 0; k0 < g.k; k0 += 32) {
    for (int i = tid; i < 64 * 32; i += 256) {
      sa[i & 63][i >> 6] = element(g.a, AT, g.lda, m0 + (i & 63), g.m, k0 + (i >> 6));
      sb[i & 63][i >> 6] = element(g.b, !BT, g.ldb, n0 + (i & 63), g.n, k0 + (i >> 6));
    }
    __syncthreads();
    const bf16x8 af = *(const bf16x8 *)&sa[wave * 16 + (lane & 15)][8 * (lane >> 4)];
    for (int q = 0; q < 4; ++q)
      acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8 *)&sb[q * 16 + (lane & 15)][8 * (lane >> 4)], af, acc[q], 0, 0, 0);
    __syncthreads();
  }
  const EpilogueArgs &e = g.ep;
  const int64_t m = m0 + wave * 16 + (lane & 15);
  for (int q = 0; q < 4; ++q)
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + q * 16 + 4 * (lane >> 4) + i;
      if (m >= g.m || n >= g.n) continue;
      float z = acc[q][i];
      if (e.row_scale) z *= e.row_scale[m];
      if (e.col_scale) z *= e.col_scale[n];
      if (e.bias) z += ep_load(e.bias, e.bias_type, n);
      if (e.pre) ((__bf16 *)e.pre)[m * e.ldp + n] = (__bf16)z;
      float y = act_f32(e.act, z);
      if (e.residual) y += ep_load(e.residual, e.residual_type, m * e.ldr + n);
      if (e.out_type == kTypeF32) ((float *)e.out)[m * e.ldo + n] = y;
      else ((__bf16 *)e.out)[m * e.ldo + n] = (__bf16)y;
    }
}

hipError_t launch_product_simple(const ProductArgs &a, int form, hipStream_t s) {
  const dim3 grid((uint32_t)(((int64_t)a.m + 63) / 64), (uint32_t)((a.n + 63) / 64)), block(256);
  if (form == kFormNT) hipLaunchKernelGGL(ptg_product_simple_kernel<kFormNT>, grid, block, 0, s, a);
  else if (form == kFormNN) hipLaunchKernelGGL(ptg_product_simple_kernel<kFormNN>, grid, block, 0, s, a);
  else if (form == kFormTN) hipLaunchKernelGGL(ptg_product_simple_kernel<kFormTN>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(ptg_product_simple_kernel<kFormNTE4m3>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace ptg
