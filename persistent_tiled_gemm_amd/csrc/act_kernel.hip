// The activation's gradient: dpre = dout act'(pre), and its column sums (the
// bias's gradient). Bound by memory: 6 bytes an element.
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
    for (int64_t row = r0 + wave; row < r1; row += 4) {
      f32x8 d = load8((const __bf16 *)a.dout + row * a.lddo + j);
      if constexpr (ACT != kActNone) {
        const f32x8 z = load8((const __bf16 *)a.pre + row * a.ldp + j);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= act_grad_f32(ACT, z[e]);
      }
      if (a.dpre) store8((__bf16 *)a.dpre + row * a.lddp + j, d);
      sum += d;
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
