// The activation's gradient: dpre = dout act'(pre), and its column sums (the
// bias's gradient). Bound by memory: 6 bytes an element (8191 x 8192, gelu_tanh:
// 79 us, 5.1 TB/s; with the column sums' launch 83.5. One row at a time: 90).
//
// A workgroup covers 512 columns (64 threads of eight, so a wave reads 1 KiB of
// a row) and a range of rows, one row per wave at a time. A thread's columns do
// not change, so its share of the bias's gradient stays in registers; the four
// waves join in LDS and the workgroup leaves one partial row.
#include "layer_device.hpp"

namespace ptg {

template <int ACT>
__global__ __launch_bounds__(256) void ptg_activation_backward_kernel(const ActGradArgs a) {
  __shared__ f32x8 lds[4][64];
  const int32_t lane = (int32_t)threadIdx.x & 63, wave = (int32_t)threadIdx.x >> 6;
  const int32_t j = ((int32_t)blockIdx.x * 64 + lane) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_group;
  const int64_t r1 = r0 + a.rows_per_group < a.m ? r0 + a.rows_per_group : a.m;
  f32x8 sum = {};
  if (j < a.n) {
    // four rows at a time: their loads are all under way before the first is used
    for (int64_t row = r0 + wave; row < r1; row += 16) {
      bf16x8 d[4], z[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t m = row + 4 * u;
        if (m >= r1) continue;
        d[u] = *(const bf16x8 *)((const __bf16 *)a.dout + m * a.lddo + j);
        if constexpr (ACT != kActNone) z[u] = *(const bf16x8 *)((const __bf16 *)a.pre + m * a.ldp + j);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t m = row + 4 * u;
        if (m >= r1) continue;
        f32x8 g = widen(d[u]);
        if constexpr (ACT != kActNone) {
          const f32x8 v = widen(z[u]);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= act_grad_f32(ACT, v[e]);
        }
        if (a.dpre) store8_nt((__bf16 *)a.dpre + m * a.lddp + j, g);
        sum += g;
      }
    }
  }
  if (a.partial) {
    lds[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && j < a.n)
      store8(a.partial + (int64_t)blockIdx.y * a.n + j, ((lds[0][lane] + lds[1][lane]) + lds[2][lane]) + lds[3][lane]);
  }
}

hipError_t launch_activation_backward(const ActGradArgs &a, int row_groups, hipStream_t s) {
  const dim3 grid((uint32_t)((a.n + 511) / 512), (uint32_t)row_groups), block(256);
  switch (a.act) {
    case kActRelu: hipLaunchKernelGGL(ptg_activation_backward_kernel<kActRelu>, grid, block, 0, s, a); break;
    case kActGelu: hipLaunchKernelGGL(ptg_activation_backward_kernel<kActGelu>, grid, block, 0, s, a); break;
    case kActGeluTanh: hipLaunchKernelGGL(ptg_activation_backward_kernel<kActGeluTanh>, grid, block, 0, s, a); break;
    case kActSilu: hipLaunchKernelGGL(ptg_activation_backward_kernel<kActSilu>, grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL(ptg_activation_backward_kernel<kActNone>, grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace ptg
