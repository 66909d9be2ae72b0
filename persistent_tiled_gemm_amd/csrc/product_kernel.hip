// The product of the layer operators as tiles: gemm_body.hpp (dynamic scheduler)
// with strided operands in the layouts a linear layer and its gradients need,
// bf16 or e4m3, and the epilogue that turns z = sum_k a b into
// out = act(z scales + bias) + residual. Bound by MFMA issue and power, then by the
// epilogue. 8192^3 to bf16: NT 716 us (1535 TFLOP/s; the vendor library's 689), and 8
// more with pre, 17 with gelu_tanh, 19 with silu, 51 with gelu, 38 with a residual; both
// gradients (NN, TN) 1459 to 1468; e4m3 with a residual 678 to 686.
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

// What the epilogue needs of one row's eight columns, as loaded: the residual's 16
// or 32 bytes and the row's scale.
struct RowTerms { i32x4 lo, hi; float scale; };
template <bool E8>
__device__ __forceinline__ RowTerms row_terms(const EpilogueArgs &e, int64_t m, int32_t n) {
  RowTerms t = {{0, 0, 0, 0}, {0, 0, 0, 0}, 1.0f};
  if (e.residual) {
    const int64_t at = m * e.ldr + n;
    if (e.residual_type == kTypeF32) {
      t.lo = *(const i32x4 *)((const float *)e.residual + at);
      t.hi = *(const i32x4 *)((const float *)e.residual + at + 4);
    } else {
      t.lo = *(const i32x4 *)((const __bf16 *)e.residual + at);
    }
  }
  if (E8 && e.row_scale) t.scale = e.row_scale[m];
  return t;
}

// Of eight columns, the same for every row.
struct ColumnTerms { f32x8 bias, scale; };
template <bool E8>
__device__ __forceinline__ ColumnTerms column_terms(const EpilogueArgs &e, int32_t n) {
  ColumnTerms t = {{}, {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}};
  if (e.bias) t.bias = load8_as(e.bias, e.bias_type, n);
  if (E8 && e.col_scale) t.scale = load8(e.col_scale + n);
  return t;
}

// z of rows m and (where `both`) m + step, columns n .. n + 7, to out (and pre).
// TERMS: there is a residual or a row scale.
template <bool E8, bool TERMS>
__device__ __forceinline__ void finish_rows(const EpilogueArgs &e, int64_t m, int32_t step, bool both, int32_t n, f32x8 z0, f32x8 z1,
                                            const ColumnTerms &col, const RowTerms &t0, const RowTerms &t1) {
  if constexpr (E8) {
    if constexpr (TERMS) {
      z0 *= t0.scale;
      z1 *= t1.scale;
    }
    z0 *= col.scale;
    z1 *= col.scale;
  }
  z0 += col.bias;
  z1 += col.bias;
  if (e.pre) {
    __bf16 *p = (__bf16 *)e.pre + m * e.ldp + n;
    store8_nt(p, z0);
    if (both) store8_nt(p + step * e.ldp, z1);
  }
  act16(e.act, z0, z1);
  if constexpr (TERMS) {
    if (e.residual) {
      if (e.residual_type == kTypeF32) {
        z0 += __builtin_shufflevector(__builtin_bit_cast(f32x4, t0.lo), __builtin_bit_cast(f32x4, t0.hi), 0, 1, 2, 3, 4, 5, 6, 7);
        z1 += __builtin_shufflevector(__builtin_bit_cast(f32x4, t1.lo), __builtin_bit_cast(f32x4, t1.hi), 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        z0 += __builtin_convertvector(__builtin_bit_cast(bf16x8, t0.lo), f32x8);
        z1 += __builtin_convertvector(__builtin_bit_cast(bf16x8, t1.lo), f32x8);
      }
    }
  }
  if (e.out_type == kTypeF32) {
    float *p = (float *)e.out + m * e.ldo + n;
    store8_nt(p, z0);
    if (both) store8_nt(p + step * e.ldo, z1);
  } else {
    __bf16 *p = (__bf16 *)e.out + m * e.ldo + n;
    store8_nt(p, z0);
    if (both) store8_nt(p + step * e.ldo, z1);
  }
}

template <int FORM>
struct ProductOp {
  using Args = ProductOpArgs;
  static constexpr bool AT = FORM == kFormTN, E8 = FORM == kFormNTE4m3, BT = FORM == kFormNT || E8, kPlain = false, kWide = !AT;
  // 16 x 16 blocks for both tile edges: a k-step's fragments are read a whole step
  // ahead of their MFMAs (the 128 x 128 tile's other form, 32 x 32 blocks read half
  // a step ahead, measured 160 us against 152 on 1024 x 8192 x 8192). k-contiguous
  // operands come two k-steps at a time (8192^3 NT 759 -> 742 us, and 785 -> 730 with
  // their loads spread over the step; NN 734 -> 700; 1000 x 4104 x 2056 61 -> 47); a
  // pair's loads then have one to two steps to land in a ring of four stages, enough
  // for the 256 x 256 tile's steps but not for the shorter ones of 128 x 128, which
  // get eight (and one workgroup a CU).
  template <int EDGE> using Tile = Cfg<EDGE, EDGE, 2, 2, 16, EDGE == 128 && !AT ? 8 : 4>;
  static __device__ __forceinline__ int32_t lda(const KernelProblem &, const Args &op) { return op.lda; }
  static __device__ __forceinline__ int32_t ldb(const KernelProblem &, const Args &op) { return op.ldb; }

  // RP staged rows of ROW_B bytes (16-byte chunk c of row r in slot c ^ (r mod
  // 16)) to memory, first row m_base, first column n_base. A lane takes eight
  // consecutive columns, so a bf16 row leaves as whole 16-byte stores (256
  // contiguous bytes a row for the 256 x 256 tile) and the columns' bias and
  // scale stay in registers. A lane's rows follow each other two at a time
  // through one copy of the code (five activations of 16 values: unrolled over all
  // rows they outgrow the instruction cache and the registers). One wave a SIMD
  // hides nothing by itself: the next two rows' sums are read from LDS, and with
  // residuals or row scales the next four rows' are asked for, before two rows are
  // finished.
  // slot: a K-chunk's sums go there unfinished, rows STRIDE floats apart.
  template <int RP, int ROW_B, int STRIDE>
  static __device__ __forceinline__ void flush(const Args &, const unsigned char *wl, uint32_t lane, int32_t m_base, int32_t n_base,
                                               int32_t M, int32_t N, float *slot) {
    constexpr int LPR = ROW_B / 32, RPI = 64 / LPR, kRows = RP / RPI;
    static_assert(kRows % 2 == 0 && (LPR == 16 || LPR == 8), "epilogue");
    const EpilogueArgs e = epilogue_args();
    // the lane's offsets are computed here, not kept over the main loop
    asm volatile("" : "+v"(lane));
    const uint32_t q = lane % LPR, r0 = lane / LPR;
    const int32_t n = n_base + (int32_t)(8u * q);
    const int32_t left = M - m_base - (int32_t)r0;  // rows from the lane's first on
    if (n >= N || left <= 0) return;
    const int rows = left >= RP ? kRows : (left + RPI - 1) / RPI;  // of the lane's, how many exist
    auto staged = [&](int i) -> f32x8 {
      const uint32_t row = (uint32_t)(i * RPI) + r0;
      const f32x4 lo = *(const f32x4 *)(wl + row * ROW_B + (((2u * q) ^ (row & 15u)) << 4));
      const f32x4 hi = *(const f32x4 *)(wl + row * ROW_B + (((2u * q + 1u) ^ (row & 15u)) << 4));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    if (slot) {
#pragma unroll 4
      for (int i = 0; i < rows; ++i) store8(slot + ((uint32_t)(i * RPI) + r0) * STRIDE + 8u * q, staged(i));
      return;
    }
    const ColumnTerms col = column_terms<E8>(e, n);
    const int64_t m0 = (int64_t)m_base + r0;
    auto finish = [&](auto terms) {
      constexpr bool kTerms = decltype(terms)::value;
      const RowTerms none = {{0, 0, 0, 0}, {0, 0, 0, 0}, 1.0f};
      auto ask = [&](int i) -> RowTerms { return i < rows ? row_terms<E8>(e, m0 + i * RPI, n) : none; };
      RowTerms t[4] = {none, none, none, none};
      if constexpr (kTerms) {
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] = ask(u);
      }
      f32x8 z0 = staged(0), z1 = staged(1);
#pragma unroll 1
      for (int i = 0; i < rows; i += 2) {
        const f32x8 a0 = z0, a1 = z1;
        if (i + 2 < kRows) {
          z0 = staged(i + 2);
          z1 = staged(i + 3);
        }
        const RowTerms t0 = t[0], t1 = t[1];
        if constexpr (kTerms) {
          t[0] = t[2];
          t[1] = t[3];
          t[2] = ask(i + 4);
          t[3] = ask(i + 5);
        }
        finish_rows<E8, kTerms>(e, m0 + i * RPI, RPI, i + 1 < rows, n, a0, a1, col, t0, t1);
      }
    };
    if (e.residual || (E8 && e.row_scale)) finish(std::true_type{});
    else finish(std::false_type{});
  }
};

// MODE: kDynamic, or kNonPersistent where every unit's workgroup is resident at
// once: there is then nothing to claim, and the first claim's round trip is saved
// (1024^3 in 128 x 128 tiles 13.6 -> 11.3 us).
template <int EDGE, int FORM, int MODE>
__global__ __launch_bounds__(256, product_workgroups(EDGE, FORM)) void ptg_product_kernel(const ProductKernelArgs a) {
  gemm_body<EDGE, EDGE, MODE, false, ProductOp<FORM>>(a.gemm, a.op);
}

// The tiles that were split along k: their chunks' sums, added in chunk order,
// through the epilogue. A second launch, so that the whole machine reads the
// sums: the workgroup that completes a tile, left to finish it alone (as the
// plain GEMM's split tail is), reads its S x 64 or 256 KiB at the 55 GB/s or so
// that one CU gets past its L2 (100 x 1024 x 8192, 8 tiles in 8 chunks: 24.8 us).
struct ReduceArgs {
  EpilogueArgs ep;
  const float *ws;
  int32_t m, n, tiles_n, first, chunks;  // first: the first split tile
};
template <int EDGE, bool E8>
__global__ __launch_bounds__(256) void ptg_product_reduce_kernel(const ReduceArgs a) {
  constexpr int LPR = EDGE / 8, kRows = 256 / LPR, kParts = EDGE / kRows;  // a workgroup: kRows rows of a tile
  const uint32_t q = threadIdx.x % LPR, r = blockIdx.x % kParts * kRows + threadIdx.x / LPR, tile = blockIdx.x / kParts;
  const int32_t t = a.first + (int32_t)tile;
  const int32_t m = t / a.tiles_n * EDGE + (int32_t)r, n = t % a.tiles_n * EDGE + (int32_t)(8u * q);
  if (m >= a.m || n >= a.n) return;
  const RowTerms row = row_terms<E8>(a.ep, m, n);
  const ColumnTerms col = column_terms<E8>(a.ep, n);
  const float *p = a.ws + (size_t)tile * a.chunks * (EDGE * EDGE) + r * EDGE + 8u * q;
  f32x8 z = load8(p);
  for (int32_t c = 1; c < a.chunks; ++c) z += load8(p + (size_t)c * (EDGE * EDGE));
  finish_rows<E8, true>(a.ep, m, 0, false, n, z, z, col, row, row);
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
  const ReduceArgs a = {op.ep, ws, m, n, (n + tile_edge - 1) / tile_edge, first, chunks};
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
