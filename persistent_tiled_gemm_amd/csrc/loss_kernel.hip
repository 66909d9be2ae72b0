// Softmax cross entropy of an output head, z = x w^T with a column for each of the
// vocabulary's entries, without the logits z reaching memory.
//
// Loss: the product's tiles (gemm_body.hpp, both operands k-contiguous) end in each
// row's maximum and sum of exp(z - maximum) over the wave's columns, taken from the
// accumulators as they lie in registers: a lane holds a quarter of a row's columns,
// two exchanges between lanes join the quarters. 8 bytes a row and block of 128 columns
// go to memory in place of 256 or 512; a second launch joins the blocks,
//   lse = M + log sum_b s_b exp(m_b - M),  loss = lse - z_label,
// in block order, so nothing depends on the order of workgroups. The wave that holds a
// label's column writes its logit.
//
// Gradient: the same tiles, computed again, end in dz = weight (exp(z - lse) - [label]),
// rounded to bf16, for the two products that follow. Half a step of bf16 is 2^-9 to 2^-8
// of each dz; the loss's own factor (a mean's 1 / count) is left to those products'
// epilogues, so that it is not rounded with dz, and the label's entry of an
// unpredicted token, -1 + p, is exact to p.
//
// Bound by power and MFMA issue, as the product is, where there are tiles enough: 4096 x
// 131072 x 4096, loss 2.97 ms (1481 TFLOP/s; the vendor library's logits alone 3.06), the
// gradient's logits 399 us of 1162 for each 16384 entries. Few tiles fill and drain: 1000 x
// 50264 x 2056, 788 tiles of 33 two-step loads, 201 us with w in the last-level cache and 236
// from memory; 777 x 10240 x 1032's dz, 160 tiles, 41 us.
#include "loss_device.hpp"
#include "product_op.hpp"

namespace ptg {

struct LossKernelArgs {
  KernelArgs gemm;
  ProductOpArgs op;
  LossTerms loss;
};

__device__ __forceinline__ LossTerms loss_terms() { return late_args<LossTerms, offsetof(LossKernelArgs, loss)>(); }

// A row's label as a column of the product, -1 where it has none there.
__device__ __forceinline__ int32_t label_column(int64_t label, int64_t first) {
  const int64_t at = label - first;
  return label < 0 || at < 0 || at >= (int64_t)1 << 30 ? -1 : (int32_t)at;
}

// What the gradient takes of a row: exp(z - lse) = 2^(z log2 e - offset), dz = factor (that
// - [column == at]). A row that is not counted has factor 0, and its dz are zeros whatever
// its logits are, NaN included. A label past the vocabulary is a mistake, shown as NaN.
struct RowGrad { float offset, factor; int32_t at, pad; };
__device__ __forceinline__ RowGrad row_grad(int64_t label, float lse, float weight, int64_t first, int64_t entries) {
  const float factor = label < 0 ? 0.0f : label >= entries ? __uint_as_float(0x7fc00000u) : weight;
  return {lse * kLog2E, factor, label_column(label, first), 0};
}
__device__ __forceinline__ float probability(float z, const RowGrad &r) { return __builtin_amdgcn_exp2f(fmaf(z, kLog2E, -r.offset)); }
__device__ __forceinline__ float times_factor(float factor, float v) { return factor == 0.0f ? 0.0f : factor * v; }

template <int FORM, int STAGES>
struct LossOp {
  using Args = ProductOpArgs;
  static constexpr bool AT = false, BT = true, E8 = false, I8 = false, kPlain = false, kWide = true, kDirect = true, kSuper = true;
  static constexpr bool kGrad = FORM == kFormLogitGrad;
  template <int EDGE> using Tile = typename ProductOp<kFormNT, STAGES>::template Tile<EDGE>;
  static __device__ __forceinline__ int32_t lda(const KernelProblem &, const Args &op) { return op.lda; }
  static __device__ __forceinline__ int32_t ldb(const KernelProblem &, const Args &op) { return op.ldb; }

  // A row's terms as asked for, and as finish reads them.
  struct Ask { int64_t label; float lse, weight; };
  using Row = typename std::conditional<kGrad, RowGrad, int32_t>::type;
  static __device__ __forceinline__ Ask ask(int32_t m, int32_t M) {
    const LossTerms l = loss_terms();
    Ask a = {-1, 0.0f, 1.0f};
    if (m >= M) return a;
    a.label = l.label[m];
    if constexpr (kGrad) {
      a.lse = l.lse[m];
      if (l.weight) a.weight = l.weight[m];
    }
    return a;
  }
  static __device__ __forceinline__ Row row(const Ask &a) {
    const LossTerms l = loss_terms();
    if constexpr (kGrad) return row_grad(a.label, a.lse, a.weight, l.first, l.entries);
    else return label_column(a.label, l.first);
  }

  // The wave's WM x WN accumulators: lane l holds, of row l mod 16 of its MI blocks of
  // rows, the columns 16 ni + 4 (l / 16) + 0..3. They leave the accumulator registers a few
  // blocks at a time (the statements that name them: otherwise all 256 would at once, for
  // memory).
  template <class CF, class Acc>
  static __device__ __forceinline__ void finish(Acc &acc, const Row *rows, uint32_t lane, int32_t m_base, int32_t n_base, int32_t M, int32_t N) {
    static_assert(CF::MB == 16 && CF::WN == loss_block(CF::BN_) && CF::NI % 2 == 0, "blocks");
    if (n_base >= N) return;  // a block past the vocabulary
    asm volatile("" : "+v"(lane));
    if (n_base + CF::WN > N) {  // columns past the vocabulary: exp(-infinity) has no part, and dz is 0 there
      int32_t left = N - n_base - (int32_t)(4u * (lane >> 4));
#pragma unroll
      for (int mi = 0; mi < CF::MI; ++mi) {
#pragma unroll
        for (int ni = 0; ni < CF::NI; ++ni) {
          asm volatile("" : "+a"(acc[mi][ni]), "+v"(left));  // (no masks kept from block to block)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mi][ni][e] = 16 * ni + e < left ? acc[mi][ni][e] : -INFINITY;
          asm volatile("" : "+a"(acc[mi][ni]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (kGrad) grad<CF>(acc, rows, lane, m_base, n_base, M, N);
    else stats<CF>(acc, rows, lane, m_base, n_base, M);
  }

  // Two blocks of rows at a time (their exchanges between lanes overlap).
  template <class CF, class Acc>
  static __device__ __forceinline__ void stats(Acc &acc, const Row *rows, uint32_t lane, int32_t m_base, int32_t n_base, int32_t M) {
    constexpr int MI = CF::MI, NI = CF::NI, G = 2;
    const LossTerms l = loss_terms();
    const uint32_t quarter = lane >> 4;
    const int32_t row = m_base + (int32_t)(lane & 15u), first = n_base + (int32_t)(4u * quarter);
    float2 *out = l.partial + (size_t)(n_base / CF::WN) * (size_t)M;
#pragma unroll
    for (int g = 0; g < MI; g += G) {
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) asm volatile("" : "+a"(acc[g + u][ni]));
      int32_t at[G];  // the label, from the lane's first column on
      float top[G], sum[G];
#pragma unroll
      for (int u = 0; u < G; ++u) {
        at[u] = rows[16 * (g + u) + (int)(lane & 15u)] - first;
        top[u] = -INFINITY;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const auto &z = acc[g + u][ni];
          top[u] = fmaxf(top[u], fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
        }
      }
#pragma unroll
      for (int o = 16; o < 64; o <<= 1)
#pragma unroll
        for (int u = 0; u < G; ++u) top[u] = fmaxf(top[u], __shfl_xor(top[u], o, 64));
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const float offset = offset_of(top[u]);
        float s = 0.0f;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
          for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(fmaf(acc[g + u][ni][e], kLog2E, -offset));
        sum[u] = put_right(s, top[u], offset);
        if (__ballot(at[u] >= 0 && at[u] < CF::WN)) {  // few tiles hold a label of theirs
          float picked = 0.0f;
          bool mine = false;
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool here = at[u] == 16 * ni + e;
              picked = here ? acc[g + u][ni][e] : picked;
              mine = mine || here;
            }
          if (mine) l.picked[row + 16 * (g + u)] = picked;
        }
      }
#pragma unroll
      for (int o = 16; o < 64; o <<= 1)
#pragma unroll
        for (int u = 0; u < G; ++u) sum[u] += __shfl_xor(sum[u], o, 64);
      // each quarter of the lanes writes a quarter of the rows
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const int32_t m = row + 16 * (g + u);
        if ((uint32_t)((g + u) & 3) == quarter && m < M) out[m] = make_float2(top[u], sum[u]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // dz of two blocks of columns at a time: four bf16 a lane and block, which two exchanges of
  // lane quarters turn into eight consecutive ones, so that a store writes 64 bytes of
  // sixteen rows. (Through LDS, in whole rows, a tile took some 12 us longer.)
  template <class CF, class Acc>
  static __device__ __forceinline__ void grad(Acc &acc, const Row *rows, uint32_t lane, int32_t m_base, int32_t n_base, int32_t M, int32_t N) {
    constexpr int MI = CF::MI, NI = CF::NI;
    const LossTerms l = loss_terms();
    const uint32_t quarter = lane >> 4;
    const int32_t row = m_base + (int32_t)(lane & 15u), first = n_base + (int32_t)(4u * quarter);
    const int32_t n = n_base + (int32_t)(16u * (quarter >> 1) + 8u * (quarter & 1u));  // the lane's columns of a store
    __bf16 *out = (__bf16 *)l.dz + (int64_t)row * l.lddz + n;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      RowGrad r = rows[16 * mi + (int)(lane & 15u)];
      r.at -= first;
      const bool none = r.factor == 0.0f, in = row + 16 * mi < M;
      auto pair = [&](int ni, bool labelled) {
        typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
        u32x2 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          asm volatile("" : "+a"(acc[mi][ni + h]));
          f32x4 d;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float p = probability(acc[mi][ni + h][e], r);
            if (labelled) p -= r.at == 16 * (ni + h) + e ? 1.0f : 0.0f;
            d[e] = p * r.factor;
          }
          v[h] = __builtin_bit_cast(u32x2, __builtin_convertvector(d, bf16x4));
          if (none) v[h] = u32x2{0u, 0u};
        }
        // quarters (a0 a1 a2 a3), (b0 b1 b2 b3) -> (a0 a2 b0 b2), (a1 a3 b1 b3)
        i32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const auto x = __builtin_amdgcn_permlane32_swap(v[0][j], v[1][j], false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
          w[j] = (int)y[0];
          w[2 + j] = (int)y[1];
        }
        if (in && n + 16 * ni < N) *(i32x4 *)(out + 16 * ni) = w;
      };
      if (__ballot(r.at >= 0 && r.at < CF::WN)) {  // few tiles hold a label of theirs
#pragma unroll
        for (int ni = 0; ni < NI; ni += 2) pair(ni, true);
      } else {
#pragma unroll
        for (int ni = 0; ni < NI; ni += 2) pair(ni, false);
      }
      out += 16 * l.lddz;
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Staged rows (see ProductOp) of a K-chunk's sums, to their slot.
  template <int RP, int ROW_B, int STRIDE>
  static __device__ __forceinline__ void flush(const Args &, const unsigned char *wl, uint32_t lane, int32_t m_base, int32_t n_base,
                                               int32_t M, int32_t N, float *slot) {
    constexpr int LPR = ROW_B / 32, RPI = 64 / LPR;
    asm volatile("" : "+v"(lane));
    const uint32_t q = lane % LPR, r0 = lane / LPR;
    const int32_t left = M - m_base - (int32_t)r0;
    if (n_base + (int32_t)(8u * q) >= N || left <= 0) return;
    const int rows = left >= RP ? RP / RPI : (left + RPI - 1) / RPI;
#pragma unroll 4
    for (int i = 0; i < rows; ++i) {
      const uint32_t row = (uint32_t)(i * RPI) + r0;
      const f32x4 lo = *(const f32x4 *)(wl + row * ROW_B + (((2u * q) ^ (row & 15u)) << 4));
      const f32x4 hi = *(const f32x4 *)(wl + row * ROW_B + (((2u * q + 1u) ^ (row & 15u)) << 4));
      store8(slot + row * STRIDE + 8u * q, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

template <int EDGE, int FORM, int STAGES, int MODE>
__global__ __launch_bounds__(256, stages_workgroups(EDGE, STAGES)) void ptg_loss_kernel(const LossKernelArgs a) {
  gemm_body<EDGE, EDGE, MODE, false, LossOp<FORM, STAGES>>(a.gemm, a.op);
}

// The tiles that were split along k: their chunks' sums, added in chunk order, then what
// a whole tile's wave does with them. A row's lanes follow each other, so a block's
// EDGE / 2 columns lie in EDGE / 16 of them.
struct LossChunksArgs {
  LossTerms loss;
  const float *ws;
  int32_t m, n, tiles_m, tiles_n, super_rows, first, chunks;
};
template <int EDGE, int FORM>
__global__ __launch_bounds__(256) void ptg_loss_chunks_kernel(const LossChunksArgs a) {
  constexpr int LPR = EDGE / 8, kRows = 256 / LPR, kParts = EDGE / kRows, kLanes = LPR / 2;
  const uint32_t q = threadIdx.x % LPR, r = blockIdx.x % kParts * kRows + threadIdx.x / LPR, tile = blockIdx.x / kParts;
  int32_t m_t, n_t;
  decode_super_tile(a.first + (int32_t)tile, a.tiles_m, a.tiles_n, a.super_rows, m_t, n_t);
  const int32_t m = m_t * EDGE + (int32_t)r, n = n_t * EDGE + (int32_t)(8u * q);
  const bool in = m < a.m && n < a.n;
  f32x8 z = {};
  if (in) z = chunk_sum<EDGE, false>(a.ws, tile, r, q, a.chunks);
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = n + e < a.n ? z[e] : -INFINITY;  // (see finish)
  if constexpr (FORM == kFormLogitGrad) {
    if (!in) return;
    const RowGrad g = row_grad(a.loss.label[m], a.loss.lse[m], a.loss.weight ? a.loss.weight[m] : 1.0f, a.loss.first, a.loss.entries);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = times_factor(g.factor, probability(z[e], g) - (g.at == n + e ? 1.0f : 0.0f));
    store8((__bf16 *)a.loss.dz + (int64_t)m * a.loss.lddz + n, z);
  } else {
    float top = -INFINITY, sum = 0.0f;
    if (in) {
      const int64_t at = a.loss.label[m] - a.loss.first - n;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        top = fmaxf(top, z[e]);
        if (at == e && a.loss.label[m] >= 0) a.loss.picked[m] = z[e];
      }
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float offset = offset_of(top);
    if (in) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += __builtin_amdgcn_exp2f(fmaf(z[e], kLog2E, -offset));
    }
    sum = put_right(sum, top, offset);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor(sum, o, 64);
    if (in && q % kLanes == 0) a.loss.partial[(size_t)(n / loss_block(EDGE)) * (size_t)a.m + m] = make_float2(top, sum);
  }
}

// The blocks of a row joined: R rows a workgroup, whose threads take a slice of the blocks
// each, eight at a time with all their loads under way, and meet in a tree of lanes, then of
// waves; the order is fixed. Sixteen rows fill a 128-byte line. Bound by latency: 4 rows of 2048
// blocks 3.6 us, 4096 rows of 1024 blocks 8.2 (one block after the other, each waiting for
// the one before, took 12.6 and 57).
struct LossJoinArgs {
  const float2 *partial;
  const int64_t *label;
  float *lse, *loss;
  int64_t entries;
  int32_t blocks, m;
};
template <int R>
__global__ __launch_bounds__(512) void ptg_loss_join_kernel(const LossJoinArgs a) {
  constexpr int S = 512 / R, U = 8, kWaves = 8;
  __shared__ float2 lds[kWaves][R];
  const int32_t r = (int32_t)threadIdx.x % R, slice = (int32_t)threadIdx.x / R;
  const int32_t m = (int32_t)blockIdx.x * R + r;
  const bool ends = slice == 0 && m < a.m;  // writes the row's results
  const int64_t label = ends ? a.label[m] : -1;
  const float picked = ends ? a.lse[m] : 0.0f;
  float top = -INFINITY, sum = 0.0f;
  if (m < a.m) {
    for (int32_t b0 = slice; b0 < a.blocks; b0 += U * S) {
      float2 p[U];
      float t = top;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t b = b0 + u * S;
        p[u] = b < a.blocks ? a.partial[(size_t)b * (size_t)a.m + m] : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) t = fmaxf(t, p[u].x);
      sum = rescaled(sum, top, t);
#pragma unroll
      for (int u = 0; u < U; ++u) sum += rescaled(p[u].y, p[u].x, t);
      top = t;
    }
  }
#pragma unroll
  for (int o = R; o < 64; o <<= 1) {
    const float from = __shfl_xor(top, o, 64), other = __shfl_xor(sum, o, 64), t = fmaxf(top, from);
    sum = rescaled(sum, top, t) + rescaled(other, from, t);
    top = t;
  }
  if ((threadIdx.x & 63u) < (uint32_t)R) lds[threadIdx.x >> 6][r] = make_float2(top, sum);
  __syncthreads();
  if (!ends) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds[w][r].x);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += rescaled(lds[w][r].y, lds[w][r].x, top);
  const float lse = top + logf(sum);
  a.lse[m] = lse;
  if (a.loss) a.loss[m] = label < 0 ? 0.0f : label >= a.entries ? __uint_as_float(0x7fc00000u) : lse - picked;
}

hipError_t launch_loss_join(const float2 *partial, int32_t blocks, const int64_t *label, int64_t entries, float *lse, float *loss, int32_t m,
                            hipStream_t s) {
  const LossJoinArgs a = {partial, label, lse, loss, entries, blocks, m};
  if (m >= 16) hipLaunchKernelGGL(ptg_loss_join_kernel<16>, dim3((uint32_t)(m + 15) / 16u), dim3(512), 0, s, a);
  else if (m > 1) hipLaunchKernelGGL(ptg_loss_join_kernel<2>, dim3((uint32_t)(m + 1) / 2u), dim3(512), 0, s, a);
  else hipLaunchKernelGGL(ptg_loss_join_kernel<1>, dim3(1), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int EDGE>
static hipError_t reduce_edge(int form, const LossChunksArgs &a, int tiles, hipStream_t s) {
  const dim3 grid(reduce_grid<EDGE>(tiles));
  if (form == kFormLoss) hipLaunchKernelGGL((ptg_loss_chunks_kernel<EDGE, kFormLoss>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((ptg_loss_chunks_kernel<EDGE, kFormLogitGrad>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_reduce_loss(int tile_edge, int form, const LossTerms &loss, const float *ws, int32_t m, int32_t n, int32_t super_rows,
                              int32_t first, int32_t tiles, int32_t chunks, hipStream_t s) {
  const LossChunksArgs a = {loss, ws, m, n, (m + tile_edge - 1) / tile_edge, (n + tile_edge - 1) / tile_edge, super_rows, first, chunks};
  return tile_edge == 256 ? reduce_edge<256>(form, a, tiles, s) : reduce_edge<128>(form, a, tiles, s);
}

template <int EDGE, int FORM, int STAGES, int MODE>
static hipError_t launch_one(const LossKernelArgs &a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((ptg_loss_kernel<EDGE, FORM, STAGES, MODE>), dim3((uint32_t)grid), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int FORM>
static hipError_t launch_form(int tile_edge, int mode, bool alone, const LossKernelArgs &a, int grid, hipStream_t s) {
  if (tile_edge == 256)
    return mode == kDynamic ? launch_one<256, FORM, 4, kDynamic>(a, grid, s) : launch_one<256, FORM, 4, kNonPersistent>(a, grid, s);
  if (alone) return launch_one<128, FORM, 8, kNonPersistent>(a, grid, s);
  return mode == kDynamic ? launch_one<128, FORM, 4, kDynamic>(a, grid, s) : launch_one<128, FORM, 4, kNonPersistent>(a, grid, s);
}

hipError_t launch_product_loss(int tile_edge, int form, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op,
                               const LossTerms &loss, int grid, hipStream_t s) {
  const LossKernelArgs a = {args, op, loss};
  return form == kFormLoss ? launch_form<kFormLoss>(tile_edge, mode, alone, a, grid, s)
                           : launch_form<kFormLogitGrad>(tile_edge, mode, alone, a, grid, s);
}

}  // namespace ptg
