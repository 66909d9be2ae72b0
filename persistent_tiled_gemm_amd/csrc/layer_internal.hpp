// Types shared by the layer operators' host code and kernels (not part of the
// C ABI; the numbers equal the ABI's LAYER_* constants).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ptg_gemm.h"
#include "ptg_internal.hpp"

namespace ptg {

enum LayerType { kTypeF32 = 0, kTypeBf16 = 1, kTypeE4m3 = 2, kTypeI8 = 3 };
enum LayerAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct NormArgs {
  const void *x, *residual, *weight;
  void *sum_out, *out;
  float *scale;
  int64_t ldx, ldr, lds, ldo;
  int32_t m, n;
  int32_t type, weight_type, out_type;
  float eps;
};

struct QuantiseArgs {
  const void *x;
  void *out;
  float *scale;
  int64_t ldx, ldo;
  int32_t m, n;
  int32_t type, out_type;
};

struct NormGradArgs {
  const void *dy, *s, *weight, *dsum;
  void *dx;
  float *partial;  // [partial rows][n] sums of dweight, or NULL
  int64_t lddy, lds, lddsum, lddx;
  int32_t m, n;
  int32_t type, dy_type, weight_type;
  float eps;
};

struct ActGradArgs {
  const void *dout, *pre;
  void *dpre;
  float *partial;  // [row groups][n] sums of dbias, or NULL
  int64_t lddo, ldp, lddp;
  int32_t m, n;
  int32_t act;
  int32_t rows_per_group;
};

// What a product's epilogue does with z = sum_k a b: out = act(z scales + bias) + residual.
struct EpilogueArgs {
  const float *row_scale, *col_scale;
  const void *bias, *residual;
  void *pre, *out;
  int64_t ldr, ldp, ldo;
  int32_t bias_type, residual_type, out_type;
  int32_t act;
};

// What the products of a cross entropy make of their logits z (m rows, a column for each of the vocabulary's entries).
struct LossTerms {
  const int64_t *label;  // m; negative: the row is not counted
  const float *lse;      // gradient: m
  const float *weight;   // gradient: m, or NULL
  float *picked;         // loss: m, the label's logit
  float2 *partial;       // loss: [column block][m], each block's largest logit and the sum of exp(z - it)
  void *dz;              // gradient: m x n, bf16
  int64_t lddz;
  int64_t first;         // the vocabulary's entry of column 0
  int64_t entries;       // of the whole vocabulary
};

// The operands of a product out[m][n] = sum_k A(m, k) B(n, k), each with the
// contracted index along its rows ("k-contiguous") or down its columns.
struct ProductArgs {
  const void *a, *b;
  int64_t lda, ldb;
  int32_t m, n, k;
  EpilogueArgs ep;
  LossTerms loss;        // the loss forms', in the epilogue's place
  int32_t super_rows;    // of forms in super-tiles
};

// Forms of a product, by operand layout and type.
enum ProductForm {
  kFormNT = 0,     // A m x k, B n x k, bf16: a linear layer
  kFormNN = 1,     // A m x k, B k x n, bf16: the gradient of x
  kFormTN = 2,     // A k x m, B k x n, bf16: the gradient of w
  kFormNTE4m3 = 3, // A m x k, B n x k, e4m3
  kFormNTI8 = 4,   // A m x k, B n x k, int8
  kFormNNScaled = 5,  // kFormNN and kFormTN with one factor, read from the device, for all sums
  kFormTNScaled = 6,
  kFormLoss = 7,      // kFormNT's sums as logits: each row's maximum and sum of exponentials by column blocks
  kFormLogitGrad = 8  // kFormNT's sums as logits: their gradient
};
constexpr bool form_is_super(int form) { return form >= kFormNTI8; }  // tiles in the order of decode_super_tile
constexpr bool form_is_loss(int form) { return form == kFormLoss || form == kFormLogitGrad; }
constexpr int64_t form_units(int form) { return form == kFormNTE4m3 || form == kFormNTI8 ? 2 : 1; }  // values per 16 bits along k
// The factors that a form's epilogue takes: of each row and column, or one (at row_scale).
enum ProductScales { kScalesNone = 0, kScalesRowCol = 1, kScalesOne = 2 };
constexpr int product_scales(int form) {
  return form == kFormNTE4m3 || form == kFormNTI8 ? kScalesRowCol : form == kFormNNScaled || form == kFormTNScaled ? kScalesOne : kScalesNone;
}

hipError_t launch_rmsnorm(const NormArgs &a, int cu_count, hipStream_t s);
hipError_t launch_quantise(const QuantiseArgs &a, int cu_count, hipStream_t s);
// Rows of the partial sums that launch_rmsnorm_backward writes for m x n.
int rmsnorm_partial_rows(int32_t m, int32_t n, int cu_count);
hipError_t launch_rmsnorm_backward(const NormGradArgs &a, int cu_count, hipStream_t s);
// out[j] = sum over `rows` of partial[row][j] (+ out[j] with accumulate), in row order.
hipError_t launch_column_sum(const float *partial, int rows, int32_t n, float *out, int accumulate, hipStream_t s);
hipError_t launch_activation_backward(const ActGradArgs &a, int row_groups, hipStream_t s);

// The product for few rows (m <= kRowsMost, the most that the kernel takes).
constexpr int32_t kRowsMost = 64;
struct RowsArgs {
  const void *x, *w;
  float *partial;      // the parts of tiles whose k several workgroups share
  uint32_t *arrivals;  // one count a tile, zero between calls
  EpilogueArgs ep;
  int32_t ldx, ldw, m, n, k;
};
// Whether a product (k-contiguous operands) runs there rather than as tiles.
// (type: of both operands)
bool rows_preferred(const ProductArgs &p, int type);
// Workspace of a call, floats; *tiles: the arrival counts it uses.
int64_t rows_partial_floats(const ProductArgs &p, int type, int cu_count, int64_t *tiles);
hipError_t launch_rows(const ProductArgs &p, int type, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s);
// The same with x in LDS: int8 operands, and bf16 with a cross entropy's end.
bool rows_shared_preferred(const ProductArgs &p, int type, int cu_count);
int64_t rows_shared_floats(const ProductArgs &p, int type, int cu_count, int64_t *tiles);
hipError_t launch_rows_shared(const ProductArgs &p, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s);
int32_t rows_shared_loss_block(const ProductArgs &p, int cu_count);
hipError_t launch_rows_shared_loss(const ProductArgs &p, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s);
// A cross entropy's end of the same product (bf16): p.loss, in column blocks of rows_loss_block.
int32_t rows_loss_block(const ProductArgs &p, int cu_count);
hipError_t launch_rows_loss(const ProductArgs &p, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s);

// What a tiled product takes beside the GEMM's own arguments. Row strides in
// 16-bit units (two e4m3 values), as the GEMM's body counts them.
struct ProductOpArgs {
  EpilogueArgs ep;
  int32_t lda, ldb;
};
// Workgroups of the tiled product that a CU holds at once: by its LDS stages, and by form (at most).
constexpr int stages_workgroups(int tile_edge, int stages) { return tile_edge == 128 && stages == 4 ? 2 : 1; }
constexpr int product_workgroups(int tile_edge, int form) { return tile_edge == 128 && (form == kFormTN || form_is_super(form)) ? 2 : 1; }
// mode: kDynamic or kNonPersistent
hipError_t launch_product(int tile_edge, int form, int mode, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s);
// The same for the int8 form, the scaled forms and the loss forms. alone: no more units than CUs.
hipError_t launch_product_i8(int tile_edge, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op, int grid, hipStream_t s);
hipError_t launch_product_scaled(int tile_edge, int form, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op, int grid,
                                 hipStream_t s);
hipError_t launch_product_loss(int tile_edge, int form, int mode, bool alone, const KernelArgs &args, const ProductOpArgs &op, const LossTerms &loss,
                               int grid, hipStream_t s);
// Adds the chunks of the tiles [first, first + tiles) and finishes them.
hipError_t launch_product_reduce(int tile_edge, int form, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t first,
                                 int32_t tiles, int32_t chunks, hipStream_t s);
hipError_t launch_reduce_i8(int tile_edge, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t super_rows, int32_t first,
                            int32_t tiles, int32_t chunks, hipStream_t s);
hipError_t launch_reduce_scaled(int tile_edge, const ProductOpArgs &op, const float *ws, int32_t m, int32_t n, int32_t super_rows,
                                int32_t first, int32_t tiles, int32_t chunks, hipStream_t s);
hipError_t launch_reduce_loss(int tile_edge, int form, const LossTerms &loss, const float *ws, int32_t m, int32_t n, int32_t super_rows,
                              int32_t first, int32_t tiles, int32_t chunks, hipStream_t s);
// Columns of a block of the tiles that leaves one partial maximum and sum (the few-row kernels': rows_loss_block, rows_shared_loss_block).
constexpr int32_t loss_block(int tile_edge) { return tile_edge / 2; }
// lse and loss of m rows from `blocks` partial maxima and sums each; lse holds the labels' logits before.
hipError_t launch_loss_join(const float2 *partial, int32_t blocks, const int64_t *label, int64_t entries, float *lse, float *loss, int32_t m,
                            hipStream_t s);
// A plan's split-tail workspace, for other partial sums between its runs.
float *plan_workspace(gemm_tile_cfg plan, int64_t *floats);
// The product as a run of a GEMM plan: its tiles and dynamic scheduler; the tiles
// from split_base on are split into `split` K-chunks each (1: none), which a
// second kernel joins. The caller orders runs on different streams and waits for
// them: the plan keeps no stream of theirs, so that they may end once they are over.
gemm_status plan_run_product(gemm_tile_cfg plan, const ProductArgs &a, int form, int32_t split, int64_t split_base, hipStream_t s);
// The device status of a plan's runs, which are over; it is cleared.
gemm_status plan_status(gemm_tile_cfg plan);

}  // namespace ptg
