// The product of the layer operators as tiles: gemm_body.hpp (dynamic scheduler)
// with strided operands in the layouts a linear layer and its gradients need,
// bf16 or e4m3, and the epilogue that turns z = sum_k a b into
// out = act(z scales + bias) + residual. Bound by MFMA issue and power, then by the
// epilogue. 8192^3 to bf16: NT 716 us (1535 TFLOP/s; the vendor library's 689), and 8
// more with pre, 17 with gelu_tanh, 19 with silu, 51 with gelu, 38 with a residual; both
// gradients (NN, TN) 1459 to 1468; e4m3 with a residual 678 to 686.
#include "product_op.hpp"

namespace ptg {

// MODE: kDynamic, or kNonPersistent where every unit's workgroup is resident at
// once: there is then nothing to claim, and the first claim's round trip is saved
// (1024^3 in 128 x 128 tiles 13.6 -> 11.3 us).
template <int EDGE, int FORM, int MODE>
__global__ __launch_bounds__(256, product_workgroups(EDGE, FORM)) void ptg_product_kernel(const ProductKernelArgs a) {
  gemm_body<EDGE, EDGE, MODE, false, ProductOp<FORM>>(a.gemm, a.op);
}

template <int EDGE, bool E8>
__global__ __launch_bounds__(256) void ptg_product_reduce_kernel(const ReduceArgs a) {
  reduce_tiles<EDGE, E8 ? kScalesRowCol : kScalesNone, false, false>(a);
}

template <int EDGE>
static hipError_t launch_reduce_edge(const ReduceArgs &a, int tiles, bool e8, hipStream_t s) {
  const dim3 grid((uint32_t)tiles * (EDGE / (256 / (EDGE / 8))));
  if (e8) hipLaunchKernelGGL((ptg_product_reduce_kernel<EDGE, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((ptg_product_reduce_kernel<EDGE, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_product_reduce(int tile_edge, int form, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t first,
                                 int32_t tiles, int32_t chunks, hipStream_t s) {
  const ReduceArgs a = {op.ep, ws, m, n, (n + tile_edge - 1) / tile_edge, first, chunks, (m + tile_edge - 1) / tile_edge, 0};
  return tile_edge == 256 ? launch_reduce_edge<256>(a, tiles, form == kFormNTE4m3, s) : launch_reduce_edge<128>(a, tiles, form == kFormNTE4m3, s);
}

template <int EDGE, int MODE>
static hipError_t launch_mode(int form, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  const dim3 g((uint32_t)grid), b(256);
  const ProductKernelArgs a = {args, op};
  switch (form) {
    case kFormNT: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNT, MODE>), g, b, 0, s, a); break;
    case kFormNN: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNN, MODE>), g, b, 0, s, a); break;
    case kFormTN: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormTN, MODE>), g, b, 0, s, a); break;
    case kFormNTE4m3: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNTE4m3, MODE>), g, b, 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int EDGE>
static hipError_t launch_edge(int form, int mode, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  return mode == kDynamic ? launch_mode<EDGE, kDynamic>(form, args, op, grid, s) : launch_mode<EDGE, kNonPersistent>(form, args, op, grid, s);
}

hipError_t launch_product(int tile_edge, int form, int mode, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  return tile_edge == 256 ? launch_edge<256>(form, mode, args, op, grid, s) : launch_edge<128>(form, mode, args, op, grid, s);
}

}  // namespace ptg
