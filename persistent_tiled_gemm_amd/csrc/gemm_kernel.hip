// The plain GEMM's kernels and their launches: gemm_body.hpp with fp32 C for every
// tile edge, scheduler, grouping and layout of B.
#include "gemm_body.hpp"

namespace ptg {

template <int BM, int BN, int MODE, bool GROUPED, bool BT>
__global__ __launch_bounds__(TileCfg<BM>::type::THREADS, 1) void ptg_gemm_kernel(const KernelArgs args) {
  gemm_body<BM, BN, MODE, GROUPED, PlainOp<BT>>(args, typename PlainOp<BT>::Args{});
}

template <int BM, int BN, int MODE, bool GROUPED, bool BT>
static hipError_t launch_one(const KernelArgs &args, int grid, int dyn_lds, hipStream_t stream) {
  hipLaunchKernelGGL((ptg_gemm_kernel<BM, BN, MODE, GROUPED, BT>), dim3(grid), dim3(TileCfg<BM>::type::THREADS),
                     dyn_lds, stream, args);
  return hipGetLastError();
}

template <int BM, int BN, bool BT>
static hipError_t launch_tile(int mode, bool grouped, const KernelArgs &args, int grid, int dyn_lds,
                              hipStream_t stream) {
  switch (mode) {
    case kNonPersistent:
      return grouped ? launch_one<BM, BN, kNonPersistent, true, BT>(args, grid, dyn_lds, stream)
                     : launch_one<BM, BN, kNonPersistent, false, BT>(args, grid, dyn_lds, stream);
    case kStatic:
      return grouped ? launch_one<BM, BN, kStatic, true, BT>(args, grid, dyn_lds, stream)
                     : launch_one<BM, BN, kStatic, false, BT>(args, grid, dyn_lds, stream);
    case kDynamic:
      return grouped ? launch_one<BM, BN, kDynamic, true, BT>(args, grid, dyn_lds, stream)
                     : launch_one<BM, BN, kDynamic, false, BT>(args, grid, dyn_lds, stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm(int tile_edge, int mode, bool grouped, bool b_transposed, const KernelArgs &args, int grid,
                       int dyn_lds, hipStream_t stream) {
  if (tile_edge == 256)
    return b_transposed ? launch_tile<256, 256, true>(mode, grouped, args, grid, dyn_lds, stream)
                        : launch_tile<256, 256, false>(mode, grouped, args, grid, dyn_lds, stream);
  if (tile_edge == 128)
    return b_transposed ? launch_tile<128, 128, true>(mode, grouped, args, grid, dyn_lds, stream)
                        : launch_tile<128, 128, false>(mode, grouped, args, grid, dyn_lds, stream);
  return hipErrorInvalidValue;
}

hipError_t gemm_occupancy(int tile_edge, int dyn_lds, int *blocks_per_cu) {
  if (tile_edge == 256)
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(
        blocks_per_cu, reinterpret_cast<const void *>(&ptg_gemm_kernel<256, 256, kDynamic, false, false>),
        TileCfg<256>::type::THREADS, dyn_lds);
  if (tile_edge == 128)
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(
        blocks_per_cu, reinterpret_cast<const void *>(&ptg_gemm_kernel<128, 128, kDynamic, false, false>),
        TileCfg<128>::type::THREADS, dyn_lds);
  return hipErrorInvalidValue;
}

int gemm_static_lds_bytes(int tile_edge) {
  if (tile_edge == 256) return TileCfg<256>::type::LDS + (int)sizeof(RingRec) * kRingDepth + 4;
  if (tile_edge == 128) return TileCfg<128>::type::LDS + (int)sizeof(RingRec) * kRingDepth + 4;
  return 0;
}

}  // namespace ptg
