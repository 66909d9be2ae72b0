// The int8 product as tiles: the bf16 one's main loop, byte for byte, with the
// 16 x 16 x 64 int8 MFMA, which multiplies twice as many values in the same time and
// adds them in 32-bit integers: sums are exact (k is limited so that they fit) and are
// rounded once, on their way into the epilogue.
//
// Bound by power and MFMA issue where there are tiles enough (8192^3 with a residual 444 us,
// 2476 TOP/s; bare 407 to 448, by the bits of the operands, and the vendor library's 520); few
// tiles by their fill, drain and epilogue (1000 x 4104 x 2064: 23 us bare, 36 with bias, gelu,
// its kept argument and a residual).
#include "product_op.hpp"

namespace ptg {

template <int EDGE, int STAGES, int MODE>
__global__ __launch_bounds__(256, stages_workgroups(EDGE, STAGES)) void ptg_product_i8_kernel(const ProductKernelArgs a) {
  gemm_body<EDGE, EDGE, MODE, false, ProductOp<kFormNTI8, STAGES>>(a.gemm, a.op);
}

template <int EDGE>
__global__ __launch_bounds__(256) void ptg_product_i8_reduce_kernel(const ReduceArgs a) {
  reduce_tiles<EDGE, kScalesRowCol, true, true>(a);
}

hipError_t launch_reduce_i8(int tile_edge, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t super_rows, int32_t first,
                            int32_t tiles, int32_t chunks, hipStream_t s) {
  const ReduceArgs a = {op.ep, ws, m, n, (n + tile_edge - 1) / tile_edge, first, chunks, (m + tile_edge - 1) / tile_edge, super_rows};
  if (tile_edge == 256) hipLaunchKernelGGL(ptg_product_i8_reduce_kernel<256>, dim3(reduce_grid<256>(tiles)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(ptg_product_i8_reduce_kernel<128>, dim3(reduce_grid<128>(tiles)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int EDGE, int STAGES, int MODE>
static hipError_t launch_one(const ProductKernelArgs &a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((ptg_product_i8_kernel<EDGE, STAGES, MODE>), dim3((uint32_t)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_product_i8(int tile_edge, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  const ProductKernelArgs a = {args, op};
  if (tile_edge == 256) return mode == kDynamic ? launch_one<256, 4, kDynamic>(a, grid, s) : launch_one<256, 4, kNonPersistent>(a, grid, s);
  if (alone) return launch_one<128, 8, kNonPersistent>(a, grid, s);
  return mode == kDynamic ? launch_one<128, 4, kDynamic>(a, grid, s) : launch_one<128, 4, kNonPersistent>(a, grid, s);
}

}  // namespace ptg
