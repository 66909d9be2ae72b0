// The tiled products' operation types for gemm_body.hpp (strided operands, fused
// epilogue) and the kernel body that joins split tiles.
#pragma once

#include "gemm_body.hpp"
#include "layer_device.hpp"

namespace ptg {

struct ProductKernelArgs {
  KernelArgs gemm;
  ProductOpArgs op;
};

// Arguments read from the kernel's argument block, at byte OFFSET, when a tile is
// finished. Read through the parameter they would be loaded at the start and
// held in scalar registers over the main loop, which has none to spare: the
// tile pointers then move to vector registers and every k-step copies them back.
template <typename T, size_t OFFSET>
__device__ __forceinline__ T late_args() {
  constexpr size_t kWords = sizeof(T) / 8;
  static_assert(sizeof(T) % 8 == 0 && alignof(T) == 8 && OFFSET % 8 == 0, "read as 64-bit words");
  typedef const __attribute__((address_space(4))) uint64_t *words;
  words p = (words)__builtin_amdgcn_kernarg_segment_ptr() + OFFSET / 8;
  asm volatile("" : "+s"(p));
  uint64_t w[kWords];
#pragma unroll
  for (size_t i = 0; i < kWords; ++i) w[i] = p[i];
  T e;
  __builtin_memcpy(&e, w, sizeof(e));
  return e;
}
__device__ __forceinline__ EpilogueArgs epilogue_args() {
  return late_args<EpilogueArgs, offsetof(ProductKernelArgs, op) + offsetof(ProductOpArgs, ep)>();
}

// What the epilogue needs of one row's eight columns, as loaded: the residual's 16
// or 32 bytes and the row's scale.
struct RowTerms { i32x4 lo, hi; float scale; };
template <int SCALES>
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
  if (SCALES == kScalesRowCol && e.row_scale) t.scale = e.row_scale[m];
  return t;
}

// Of eight columns, the same for every row.
struct ColumnTerms { f32x8 bias, scale; };
template <int SCALES>
__device__ __forceinline__ ColumnTerms column_terms(const EpilogueArgs &e, int32_t n) {
  ColumnTerms t = {{}, {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}};
  if (e.bias) t.bias = load8_as(e.bias, e.bias_type, n);
  if (SCALES == kScalesRowCol && e.col_scale) t.scale = load8(e.col_scale + n);
  if (SCALES == kScalesOne && e.row_scale) {
    const float s = *e.row_scale;
    t.scale = f32x8{s, s, s, s, s, s, s, s};
  }
  return t;
}

// A tile's sums as fp32: int8 operands leave 32-bit integers, exact, and this is their
// one rounding.
typedef __attribute__((ext_vector_type(8))) int i32x8;
template <bool I8>
__device__ __forceinline__ f32x8 sums_of(const f32x8 &staged) {
  if constexpr (I8) return __builtin_convertvector(__builtin_bit_cast(i32x8, staged), f32x8);
  else return staged;
}

// z of rows m and (where `both`) m + step, columns n .. n + 7, to out (and pre).
// TERMS: there is a residual or a row scale.
template <int SCALES, bool TERMS>
__device__ __forceinline__ void finish_rows(const EpilogueArgs &e, int64_t m, int32_t step, bool both, int32_t n, f32x8 z0, f32x8 z1,
                                            const ColumnTerms &col, const RowTerms &t0, const RowTerms &t1) {
  if constexpr (SCALES != kScalesNone) {
    if constexpr (TERMS && SCALES == kScalesRowCol) {
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

template <int FORM, int STAGES = FORM == kFormTN || FORM == kFormTNScaled ? 4 : 8>
struct ProductOp {
  using Args = ProductOpArgs;
  static constexpr bool AT = FORM == kFormTN || FORM == kFormTNScaled, E8 = FORM == kFormNTE4m3, I8 = FORM == kFormNTI8;
  static constexpr bool BT = FORM == kFormNT || E8 || I8, kPlain = false, kWide = !AT;
  static constexpr int kScales = product_scales(FORM);
  static constexpr bool kDirect = false, kSuper = form_is_super(FORM);
  // 16 x 16 blocks for both tile edges: a k-step's fragments are read a whole step
  // ahead of their MFMAs (the 128 x 128 tile's other form, 32 x 32 blocks read half
  // a step ahead, measured 160 us against 152 on 1024 x 8192 x 8192). k-contiguous
  // operands come two k-steps at a time (8192^3 NT 759 -> 742 us, and 785 -> 730 with
  // their loads spread over the step; NN 734 -> 700; 1000 x 4104 x 2056 61 -> 47); a
  // pair's loads then have one to two steps to land in a ring of four stages, enough
  // for the 256 x 256 tile's steps but not for the shorter ones of 128 x 128, which
  // get eight (and one workgroup a CU). The forms of super-tiles take eight where every
  // unit has a CU to itself, and otherwise four and two workgroups a CU, each of which
  // fills and finishes its tile under the other's MFMAs (int8 2048 x 4096 x 2048, 512 tiles: 22.3
  // us against 35.7; 1000 x 4104 x 2064, 264 tiles: 22.7 and 31.1 with the last eight split;
  // 1024 x 4096 x 4096, 256 tiles: 29.3 with four stages, 26.5 with eight).
  template <int EDGE> using Tile = Cfg<EDGE, EDGE, 2, 2, 16, EDGE == 128 ? STAGES : 4>;
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
    const ColumnTerms col = column_terms<kScales>(e, n);
    const int64_t m0 = (int64_t)m_base + r0;
    auto finish = [&](auto terms) {
      constexpr bool kTerms = decltype(terms)::value;
      const RowTerms none = {{0, 0, 0, 0}, {0, 0, 0, 0}, 1.0f};
      auto ask = [&](int i) -> RowTerms { return i < rows ? row_terms<kScales>(e, m0 + i * RPI, n) : none; };
      RowTerms t[4] = {none, none, none, none};
      if constexpr (kTerms) {
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] = ask(u);
      }
      f32x8 z0 = staged(0), z1 = staged(1);
#pragma unroll 1
      for (int i = 0; i < rows; i += 2) {
        const f32x8 a0 = sums_of<I8>(z0), a1 = sums_of<I8>(z1);
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
        finish_rows<kScales, kTerms>(e, m0 + i * RPI, RPI, i + 1 < rows, n, a0, a1, col, t0, t1);
      }
    };
    if (e.residual || (kScales == kScalesRowCol && e.row_scale)) finish(std::true_type{});
    else finish(std::false_type{});
  }
};

// The tiles that were split along k: their chunks' sums, added in chunk order,
// through the epilogue. A second launch, so that the whole machine reads the
// sums: the workgroup that completes a tile, left to finish it alone (as the
// plain GEMM's split tail is), reads its S x 64 or 256 KiB at the 55 GB/s or so
// that one CU gets past its L2 (100 x 1024 x 8192, 8 tiles in 8 chunks: 24.8 us).
struct ReduceArgs {
  EpilogueArgs ep;
  const float *ws;
  int32_t m, n, tiles_n, first, chunks;  // first: the first split tile
  int32_t tiles_m, super_rows;
};
// Its grid: EDGE rows a tile, 256 / (EDGE / 8) a workgroup.
template <int EDGE>
constexpr uint32_t reduce_grid(int tiles) { return (uint32_t)tiles * (EDGE / (256 / (EDGE / 8))); }

// Eight columns (the q-th eight) of row r of split tile `tile`: its chunks' sums, added in chunk order.
template <int EDGE, bool I8>
__device__ __forceinline__ f32x8 chunk_sum(const float *ws, uint32_t tile, uint32_t r, uint32_t q, int32_t chunks) {
  const float *p = ws + (size_t)tile * chunks * (EDGE * EDGE) + r * EDGE + 8u * q;
  f32x8 z = load8(p);
  for (int32_t c = 1; c < chunks; ++c) {
    const f32x8 v = load8(p + (size_t)c * (EDGE * EDGE));
    if constexpr (I8) z = __builtin_bit_cast(f32x8, __builtin_bit_cast(i32x8, z) + __builtin_bit_cast(i32x8, v));
    else z += v;
  }
  return sums_of<I8>(z);
}

template <int EDGE, int SCALES, bool I8, bool SUPER>
__device__ __forceinline__ void reduce_tiles(const ReduceArgs &a) {
  constexpr int LPR = EDGE / 8, kRows = 256 / LPR, kParts = EDGE / kRows;  // a workgroup: kRows rows of a tile
  const uint32_t q = threadIdx.x % LPR, r = blockIdx.x % kParts * kRows + threadIdx.x / LPR, tile = blockIdx.x / kParts;
  const int32_t t = a.first + (int32_t)tile;
  int32_t m_t = t / a.tiles_n, n_t = t % a.tiles_n;
  if constexpr (SUPER) decode_super_tile(t, a.tiles_m, a.tiles_n, a.super_rows, m_t, n_t);
  const int32_t m = m_t * EDGE + (int32_t)r, n = n_t * EDGE + (int32_t)(8u * q);
  if (m >= a.m || n >= a.n) return;
  const RowTerms row = row_terms<SCALES>(a.ep, m, n);
  const ColumnTerms col = column_terms<SCALES>(a.ep, n);
  const f32x8 z = chunk_sum<EDGE, I8>(a.ws, tile, r, q, a.chunks);
  finish_rows<SCALES, true>(a.ep, m, 0, false, n, z, z, col, row, row);
}

}  // namespace ptg
