// The products of a linear layer's gradient (NN, TN) with one factor for all sums,
// read from the device when a tile is finished: the incoming gradient of a loss, which
// then stays out of the operands' rounding. Bound as the products of product_kernel.hip are: 4096 x
// 16384 x 4096, NN 360 us (1530 TFLOP/s), TN 389.
#include "product_op.hpp"

namespace ptg {

template <int EDGE, int FORM, int STAGES, int MODE>
__global__ __launch_bounds__(256, stages_workgroups(EDGE, STAGES)) void ptg_product_scaled_kernel(const ProductKernelArgs a) {
  gemm_body<EDGE, EDGE, MODE, false, ProductOp<FORM, STAGES>>(a.gemm, a.op);
}

template <int EDGE>
__global__ __launch_bounds__(256) void ptg_product_scaled_reduce_kernel(const ReduceArgs a) {
  reduce_tiles<EDGE, kScalesOne, false, true>(a);
}

hipError_t launch_reduce_scaled(int tile_edge, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t super_rows, int32_t first,
                                int32_t tiles, int32_t chunks, hipStream_t s) {
  const ReduceArgs a = {op.ep, ws, m, n, (n + tile_edge - 1) / tile_edge, first, chunks, (m + tile_edge - 1) / tile_edge, super_rows};
  if (tile_edge == 256) hipLaunchKernelGGL(ptg_product_scaled_reduce_kernel<256>, dim3(reduce_grid<256>(tiles)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(ptg_product_scaled_reduce_kernel<128>, dim3(reduce_grid<128>(tiles)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int EDGE, int FORM, int STAGES, int MODE>
static hipError_t launch_one(const ProductKernelArgs &a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((ptg_product_scaled_kernel<EDGE, FORM, STAGES, MODE>), dim3((uint32_t)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int EDGE, int FORM>
static hipError_t launch_form(int mode, const ProductKernelArgs &a, int grid, hipStream_t s) {
  return mode == kDynamic ? launch_one<EDGE, FORM, 4, kDynamic>(a, grid, s) : launch_one<EDGE, FORM, 4, kNonPersistent>(a, grid, s);
}

hipError_t launch_product_scaled(int tile_edge, int form, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op, int grid,
                                 hipStream_t s) {
  const ProductKernelArgs a = {args, op};
  if (tile_edge == 256)
    return form == kFormNNScaled ? launch_form<256, kFormNNScaled>(mode, a, grid, s) : launch_form<256, kFormTNScaled>(mode, a, grid, s);
  if (form == kFormTNScaled) return launch_form<128, kFormTNScaled>(mode, a, grid, s);
  return alone ? launch_one<128, kFormNNScaled, 8, kNonPersistent>(a, grid, s) : launch_form<128, kFormNNScaled>(mode, a, grid, s);
}

}  // namespace ptg
