// The product of the layer operators as tiles: gemm_body.hpp (dynamic scheduler)
// with strided operands in the layouts a linear layer and its gradients need,
// bf16 or e4m3, and the epilogue that turns z = sum_k a b into
// out = act(z scales + bias) + residual.
#include "gemm_body.hpp"
#include "layer_device.hpp"

namespace ptg {

struct ProductKernelArgs {
  KernelArgs gemm;
  ProductOpArgs op;
};

// The epilogue's arguments, read from the kernel's argument block when a tile is
// finished. Read through the parameter they would be loaded at the start and
// held in scalar registers over the main loop, which has none to spare: the
// tile pointers then move to vector registers and every k-step copies them back.
__device__ __forceinline__ EpilogueArgs epilogue_args() {
  constexpr size_t kWords = sizeof(EpilogueArgs) / 8;
  static_assert(sizeof(EpilogueArgs) % 8 == 0 && alignof(EpilogueArgs) == 8, "read as 64-bit words");
  typedef const __attribute__((address_space(4))) uint64_t *words;
  words p = (words)__builtin_amdgcn_kernarg_segment_ptr() + (offsetof(ProductKernelArgs, op) + offsetof(ProductOpArgs, ep)) / 8;
  asm volatile("" : "+s"(p));
  uint64_t w[kWords];
#pragma unroll
  for (size_t i = 0; i < kWords; ++i) w[i] = p[i];
  EpilogueArgs e;
  __builtin_memcpy(&e, w, sizeof(e));
  return e;
}

template <int FORM>
struct ProductOp {
  using Args = ProductOpArgs;
  static constexpr bool AT = FORM == kFormTN, E8 = FORM == kFormNTE4m3, BT = FORM == kFormNT || E8, kPlain = false;
  // e4m3: 16 x 16 blocks for both tile edges
  template <int EDGE> using Tile = typename std::conditional<E8, Cfg<EDGE, EDGE, 2, 2, 16>, typename TileCfg<EDGE>::type>::type;
  static __device__ __forceinline__ int32_t lda(const KernelProblem &, const Args &op) { return op.lda; }
  static __device__ __forceinline__ int32_t ldb(const KernelProblem &, const Args &op) { return op.ldb; }

  // RP staged rows of ROW_B bytes (16-byte chunk c of row r in slot c ^ (r mod
  // 16)) to memory, first row m_base, first column n_base. A lane takes eight
  // consecutive columns, so a bf16 row leaves as whole 16-byte stores (256
  // contiguous bytes a row for the 256 x 256 tile) and the columns' bias and
  // scale stay in registers. A lane's rows follow each other through one copy of
  // the code (five activations of eight values: unrolled over the rows they
  // outgrow the instruction cache and the registers), with the residuals and row
  // scales of the next kAhead rows under way.
  template <int RP, int ROW_B>
  static __device__ __forceinline__ void flush(const Args &, const unsigned char *wl, uint32_t lane, int32_t m_base, int32_t n_base,
                                               int32_t M, int32_t N) {
    constexpr int LPR = ROW_B / 32, RPI = 64 / LPR, kRows = RP / RPI, kAhead = 4;
    static_assert(kRows >= kAhead && (LPR == 16 || LPR == 8), "epilogue");
    const EpilogueArgs e = epilogue_args();
    // the lane's offsets are computed here, not kept over the main loop
    asm volatile("" : "+v"(lane));
    const uint32_t q = lane % LPR, r0 = lane / LPR;
    const int32_t n = n_base + (int32_t)(8u * q);
    if (n >= N) return;
    f32x8 bias = {}, cs = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (e.bias) bias = load8_as(e.bias, e.bias_type, n);
    if (E8 && e.col_scale) cs = load8(e.col_scale + n);
    struct Ahead { i32x4 lo, hi; float rs; };  // a row's residual as loaded, and its scale
    auto ask = [&](int i) -> Ahead {
      Ahead a = {{0, 0, 0, 0}, {0, 0, 0, 0}, 1.0f};
      const int64_t m = (int64_t)m_base + (uint32_t)(i * RPI) + r0;
      if (i < kRows && m < M) {
        if (e.residual) {
          const int64_t at = m * e.ldr + n;
          if (e.residual_type == kTypeF32) {
            a.lo = *(const i32x4 *)((const float *)e.residual + at);
            a.hi = *(const i32x4 *)((const float *)e.residual + at + 4);
          } else {
            a.lo = *(const i32x4 *)((const __bf16 *)e.residual + at);
          }
        }
        if (E8 && e.row_scale) a.rs = e.row_scale[m];
      }
      return a;
    };
    Ahead ahead[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) ahead[u] = ask(u);
    // 16 lanes a row (32 chunks): lanes 8..15 read their odd chunk first, which
    // spreads a read's 16 chunks over all banks; 8 lanes a row do so by the swizzle
    const uint32_t odd = LPR == 16 ? q >> 3 : 0u;
#pragma unroll 1
    for (int i = 0; i < kRows; ++i) {
      const uint32_t row = (uint32_t)(i * RPI) + r0;
      const int64_t m = (int64_t)m_base + row;
      const f32x4 v0 = *(const f32x4 *)(wl + row * ROW_B + (((2u * q + odd) ^ (row & 15u)) << 4));
      const f32x4 v1 = *(const f32x4 *)(wl + row * ROW_B + (((2u * q + 1u - odd) ^ (row & 15u)) << 4));
      const f32x4 lo = odd ? v1 : v0, hi = odd ? v0 : v1;
      f32x8 z = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      const Ahead now = ahead[0];
#pragma unroll
      for (int u = 0; u + 1 < kAhead; ++u) ahead[u] = ahead[u + 1];
      ahead[kAhead - 1] = ask(i + kAhead);
      if (m >= M) continue;
      if constexpr (E8) z = z * now.rs * cs;
      z += bias;
      if (e.pre) store8_nt((__bf16 *)e.pre + m * e.ldp + n, z);
      act8(e.act, z);
      if (e.residual) {
        if (e.residual_type == kTypeF32)
          z += __builtin_shufflevector(__builtin_bit_cast(f32x4, now.lo), __builtin_bit_cast(f32x4, now.hi), 0, 1, 2, 3, 4, 5, 6, 7);
        else
          z += __builtin_convertvector(__builtin_bit_cast(bf16x8, now.lo), f32x8);
      }
      if (e.out_type == kTypeF32) store8_nt((float *)e.out + m * e.ldo + n, z);
      else store8_nt((__bf16 *)e.out + m * e.ldo + n, z);
    }
  }
};

template <int EDGE, int FORM>
__global__ __launch_bounds__(256, EDGE == 128 ? 2 : 1) void ptg_product_kernel(const ProductKernelArgs a) {
  gemm_body<EDGE, EDGE, kDynamic, false, ProductOp<FORM>>(a.gemm, a.op);
}

template <int EDGE>
static hipError_t launch_edge(int form, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  const dim3 g((uint32_t)grid), b(256);
  const ProductKernelArgs a = {args, op};
  switch (form) {
    case kFormNT: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNT>), g, b, 0, s, a); break;
    case kFormNN: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNN>), g, b, 0, s, a); break;
    case kFormTN: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormTN>), g, b, 0, s, a); break;
    case kFormNTE4m3: hipLaunchKernelGGL((ptg_product_kernel<EDGE, kFormNTE4m3>), g, b, 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_product(int tile_edge, int form, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s) {
  return tile_edge == 256 ? launch_edge<256>(form, args, op, grid, s) : launch_edge<128>(form, args, op, grid, s);
}

}  // namespace ptg
