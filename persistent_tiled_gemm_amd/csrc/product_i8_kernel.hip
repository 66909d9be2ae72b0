// The int8 product as tiles: the bf16 one's main loop, byte for byte, with the
// 16 x 16 x 64 int8 MFMA, which multiplies twice as many values in the same time and
// adds them in 32-bit integers: sums are exact (k is limited so that they fit) and are
// rounded once, on their way into the epilogue.
//
// 8192^3 with a residual takes 446 us (2465 TOP/s; bare 391 to 446, by the bits of the operands,
// and the vendor library's 519 to 538): some 350 by power and MFMA issue, and some 100 (75 bare)
// of fill, drain and epilogue, four tiles a CU with nothing beside them (k = 2048 and 4096: 176
// and 260 us, bare 152 and 229). Few tiles are bound by those (1000 x 4104 x 2064: 23 us bare, 36
// with bias, gelu, its kept argument and a residual).
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
