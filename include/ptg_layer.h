/*
 * ptg_layer.h - C ABI of the layer operators around the persistent tiled GEMM
 * (MI355X, gfx950): the RMS norm with the residual's addition, the matrix
 * product with bias, activation and residual in its epilogue, and the
 * gradients of both. Together they are a pre-norm feed-forward layer:
 *
 *   layer_rmsnorm              s = x + residual, y = s / rms(s) * weight, bf16, fp32, or e4m3
 *                              or int8 with one scale a row (the next product's operand)
 *   layer_linear               out = act(x . w^T + bias) + residual
 *   layer_activation_backward  dpre = dout * act'(pre), dbias
 *   layer_linear_backward      dx = dpre . w, dw = dpre^T . x
 *   layer_rmsnorm_backward     dx (of x and of residual alike), dweight
 *
 * and, at the ends of a stack of such layers, what serves it in 8 bits and what trains it:
 *
 *   layer_quantize                rows to int8 or e4m3 codes with one scale each
 *   layer_cross_entropy           log sum exp and loss of an output head, without its logits
 *   layer_cross_entropy_backward  dx and dw of that loss
 *
 * Layouts. Matrices are row-major with a row stride in elements (ld*), rows
 * dense; a weight is n x k as a linear layer keeps it. Device pointers only,
 * 16-byte aligned. Row lengths and strides are multiples of 8 elements (16 for
 * e4m3 and int8 operands of a product); the number of rows m is arbitrary, 0 included.
 * Outputs and scratch share no memory with inputs or each other but where a function
 * says so.
 * A stride is at least the row's length; with m <= 1, or rows of no elements, it is
 * not looked at.
 *
 * Types. Stream and operand types are named per argument. Sums, norms,
 * products and activations are held in fp32; each output is rounded once, to
 * the nearest value of its type, from the fp32 result. (Relative error of an
 * activation at its argument, in units of 2^-24, far tails included: silu 9, gelu
 * 31, tanh-gelu 9 and 6.25 for each unit of the logistic function's argument.) e4m3 operands are
 * widened to bf16 (exactly) before they are multiplied: the e4m3 matrix
 * instructions would be faster, but they add eight products at a time and drop
 * what lies 2^-13 below the largest of the eight. int8 operands are multiplied as
 * they are, twice as many in the same time, and their sums are 32-bit integers, exact.
 *
 * Speed. k-contiguous operands (x, w, dpre in layer_linear_backward's dx) are
 * read 128 bytes of a row at a time: rows that start on 128-byte lines (strides
 * that are multiples of 64 bf16 or 128 e4m3 or int8 elements) run fastest, rows off the
 * 64-byte lines up to a third slower.
 *
 * Ownership, streams, errors. As in ptg_gemm.h: the caller owns every tensor
 * and keeps it alive until the stream has passed the call; calls are
 * asynchronous and stream-ordered and allocate nothing; arguments are checked
 * before anything is enqueued. The plan (layer_cfg) owns the scratch: the tile
 * schedulers' state, the split products' partial sums and the partial column
 * sums. Calls of one plan on different streams are ordered on the device (a
 * call waits for the plan's previous stream), so that stream must stay valid
 * until the plan's next call, layer_sync or layer_destroy (layer_sync does not
 * let go of it once a call was captured: replays may follow). A plan is not
 * thread-safe. layer_rmsnorm and layer_quantize need no plan.
 *
 * Graph capture. Every call may be captured once the plan's last call was made
 * on the capture stream (a call on a new stream waits with an event for the
 * previous one, which a capture refuses). A replay uses the plan's scratch like
 * a call: order replays and other calls of the same plan on one stream.
 *
 * No result depends on the order in which workgroups run: sums that several
 * workgroups share are written as partial sums and added in a fixed order.
 */
#ifndef PTG_LAYER_H
#define PTG_LAYER_H

#include "ptg_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define LAYER_F32 0
#define LAYER_BF16 1
#define LAYER_E4M3 2 /* 8 bits, 4 exponent and 3 mantissa bits, largest value 448, no infinities */
#define LAYER_I8 3   /* 8-bit integers, two's complement */

/*
 * Activations of a pre-activation z:
 *   NONE z;  RELU max(z, 0) (gradient 0 at z = 0; NaN stays NaN);
 *   GELU z (1 + erf(z / sqrt 2)) / 2;
 *   GELU_TANH z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2;
 *   SILU z / (1 + exp(-z)).
 */
#define LAYER_ACT_NONE 0
#define LAYER_ACT_RELU 1
#define LAYER_ACT_GELU 2
#define LAYER_ACT_GELU_TANH 3
#define LAYER_ACT_SILU 4

/* Size limits (GEMM_E_SHAPE beyond them). */
#define LAYER_MAX_ROWS (1 << 30)
#define LAYER_MAX_COLS (1 << 20)     /* n, k and row strides */
#define LAYER_MAX_NORM_COLS (1 << 15) /* n of the norm: a row is held in one workgroup's registers */
#define LAYER_MAX_I8_K 131056        /* k of an int8 product: 2^14 k stays under 2^31 */

/* Opaque plan: owns all scratch. */
typedef struct layer_plan *layer_cfg;

/*
 * Build a plan on `device`, which must be the current device and gfx950. All
 * allocation happens here (about 96 MiB: the split products' partial sums for
 * both tile sizes, which the column sums share). Errors: GEMM_E_INVALID_ARG
 * (out NULL, no such device), GEMM_E_UNSUPPORTED, GEMM_E_DEVICE, GEMM_E_NOMEM,
 * GEMM_E_HIP.
 */
gemm_status layer_create(layer_cfg *out, int32_t device);

/* Release the plan (synchronises its last stream first). NULL is a no-op. */
gemm_status layer_destroy(layer_cfg cfg);

/*
 * Synchronise the plan's last stream and return (then clear) the device-side
 * status of its products, as gemm_sync does. GEMM_OK before the first call.
 */
gemm_status layer_sync(layer_cfg cfg);

/* Text of the last HIP error seen by this plan ("" if none). */
const char *layer_last_hip_error(layer_cfg cfg);

/*
 * s = x + residual (residual NULL: s = x); r = 1 / sqrt(mean_j s_j^2 + eps);
 * y_j = s_j r weight_j. The sum enters the norm unrounded; sum_out (NULL: not
 * kept) receives it rounded to `type`, and may be x or residual itself (same
 * pointer and stride: the residual stream updated in place).
 *
 * out_type LAYER_E4M3 or LAYER_I8: `scale` receives one fp32 value a row,
 * max_j |y_j| / 448 or / 127 (at least 2^-126; 1 where the row's y is all
 * zeros), and out the codes y_j / scale (the fp32 quotient, rounded to nearest).
 * The scale's reader multiplies: y is about code * scale. A row whose y holds a
 * NaN or an infinity gets a NaN scale and NaN codes (int8: zeros). scale must
 * be NULL for the other types.
 *
 * Squares are summed in fp32: a row whose sum of squares passes 3.4e38
 * (values of about 1e18 and more) has r = 0.
 * weight may be NULL (all ones). weight_type: LAYER_F32 or LAYER_BF16.
 * One launch. m == 0 or n == 0 enqueues nothing.
 * Errors: GEMM_E_INVALID_ARG (a NULL or misaligned pointer, an unknown type, a
 * scale where there is none to write or none where there is, eps negative or
 * NaN), GEMM_E_SHAPE (negative, not a multiple of 8, over a limit, a stride
 * shorter than the row), GEMM_E_UNSUPPORTED (current device not gfx950), GEMM_E_HIP.
 */
typedef struct layer_rmsnorm_args {
  const void *x;        /* m x n, type */
  const void *residual; /* m x n, type, or NULL */
  const void *weight;   /* n, weight_type, or NULL */
  void *sum_out;        /* m x n, type, or NULL */
  void *out;            /* m x n, out_type */
  float *scale;         /* m, e4m3 and int8 outputs only */
  int64_t m, n;
  int64_t ldx, ldr, lds, ldo;
  int32_t type;         /* LAYER_F32 or LAYER_BF16: x, residual, sum_out */
  int32_t weight_type;
  int32_t out_type;     /* LAYER_F32, LAYER_BF16, LAYER_E4M3 or LAYER_I8 */
  float eps;
} layer_rmsnorm_args;

gemm_status layer_rmsnorm(const layer_rmsnorm_args *args, void *stream);

/*
 * The gradient at a given s (the forward pass's sum_out, or x without a
 * residual): with r as above (computed again from s), h = s r and
 * g = dy weight,
 *   dx_j = r (g_j - h_j mean_i(g_i h_i)) + dsum_j     (the gradient of x and of residual)
 *   dweight_j = sum_m dy_mj h_mj                       (+ dweight_j with `accumulate`)
 * dsum: the gradient that reaches sum_out from the rest of the network (NULL:
 * none). dx (NULL: not wanted) may be dsum itself (same pointer and stride).
 * dweight (fp32, NULL: not wanted; a second launch). With m == 0 dweight is
 * zeroed (unless accumulate is set). Errors as layer_rmsnorm, and GEMM_E_DEVICE.
 */
typedef struct layer_rmsnorm_grad_args {
  const void *dy;     /* m x n, dy_type */
  const void *s;      /* m x n, type */
  const void *weight; /* n, weight_type, or NULL (all ones) */
  const void *dsum;   /* m x n, type, or NULL */
  void *dx;           /* m x n, type, or NULL */
  float *dweight;     /* n, or NULL */
  int64_t m, n;
  int64_t lddy, lds, lddsum, lddx;
  int32_t type;       /* LAYER_F32 or LAYER_BF16: s, dsum, dx */
  int32_t dy_type;    /* LAYER_F32 or LAYER_BF16 */
  int32_t weight_type;
  int32_t accumulate; /* 1: add to dweight instead of overwriting it */
  float eps;
} layer_rmsnorm_grad_args;

gemm_status layer_rmsnorm_backward(const layer_rmsnorm_grad_args *args, layer_cfg cfg, void *stream);

/*
 * z_mn = x_scale_m w_scale_n sum_k x_mk w_nk + bias_n;  pre = z;
 * out = act(z) + residual.
 * in_type LAYER_BF16: x and w are bf16, x_scale and w_scale NULL.
 * in_type LAYER_E4M3 or LAYER_I8: x and w are e4m3 or int8; x_scale (m, fp32; NULL: 1)
 * and w_scale (n, fp32; NULL: 1) are their row scales (each token's and each output
 * channel's). k is then a multiple of 16, in int8 at most LAYER_MAX_I8_K; the sum of
 * int8 products is exact and rounded to fp32 before it meets the scales.
 * pre (bf16, NULL: not kept) receives z for layer_activation_backward. The
 * activation is taken of the unrounded z. residual may be out itself (same
 * pointer, stride and type). k == 0 gives z = bias. m == 0 or n == 0 enqueues
 * nothing.
 * Few rows (a decode step) read every weight once and split k over the machine
 * when n alone does not fill it; many rows run as tiles under the dynamic tile
 * scheduler, with k split as well where there are too few of them (then a second
 * launch adds the parts).
 * Errors: GEMM_E_INVALID_ARG (a NULL or misaligned pointer, an unknown type or
 * activation, a scale with bf16 operands), GEMM_E_SHAPE, GEMM_E_DEVICE,
 * GEMM_E_HIP.
 */
typedef struct layer_linear_args {
  const void *x;         /* m x k, in_type */
  const void *w;         /* n x k, in_type */
  const float *x_scale;  /* m, or NULL */
  const float *w_scale;  /* n, or NULL */
  const void *bias;      /* n, bias_type, or NULL */
  const void *residual;  /* m x n, residual_type, or NULL */
  void *pre;             /* m x n, bf16, or NULL */
  void *out;             /* m x n, out_type */
  int64_t m, n, k;
  int64_t ldx, ldw, ldr, ldp, ldo;
  int32_t in_type;       /* LAYER_BF16, LAYER_E4M3 or LAYER_I8 */
  int32_t bias_type;     /* LAYER_F32 or LAYER_BF16 */
  int32_t residual_type; /* LAYER_F32 or LAYER_BF16 */
  int32_t out_type;      /* LAYER_F32 or LAYER_BF16 */
  int32_t activation;
  int32_t pad;
} layer_linear_args;

gemm_status layer_linear(const layer_linear_args *args, layer_cfg cfg, void *stream);

/*
 * dpre_mn = dout_mn act'(pre_mn), rounded to bf16, and dbias_n = sum_m of it
 * before that rounding (fp32; + dbias_n with `accumulate`). dpre or dbias may be
 * NULL (not wanted; dbias is a second launch); dpre may be dout or pre itself
 * (same stride). pre is not read with LAYER_ACT_NONE and may be NULL then. With
 * m == 0 dbias is zeroed (unless accumulate is set). Errors as layer_linear.
 */
typedef struct layer_activation_grad_args {
  const void *dout; /* m x n, bf16 */
  const void *pre;  /* m x n, bf16 */
  void *dpre;       /* m x n, bf16, or NULL */
  float *dbias;     /* n, or NULL */
  int64_t m, n;
  int64_t lddo, ldp, lddp;
  int32_t activation;
  int32_t accumulate;
} layer_activation_grad_args;

gemm_status layer_activation_backward(const layer_activation_grad_args *args, layer_cfg cfg, void *stream);

/*
 * dx_mk = sum_n dpre_mn w_nk and dw_nk = sum_m dpre_mn x_mk (+ dw_nk with
 * `accumulate`, read in dw's type). dpre, x and w are bf16; dx and dw (NULL: not wanted)
 * fp32 or bf16. x is only read for dw, w only for dx. One launch each, or
 * two where k is split. With m == 0 dw is zeroed (unless accumulate is set).
 * Errors as layer_linear.
 */
typedef struct layer_linear_grad_args {
  const void *dpre; /* m x n */
  const void *x;    /* m x k */
  const void *w;    /* n x k */
  void *dx;         /* m x k, dx_type, or NULL */
  void *dw;         /* n x k, dw_type, or NULL */
  int64_t m, n, k;
  int64_t lddp, ldx, ldw, lddx, lddw;
  int32_t dx_type;  /* LAYER_F32 or LAYER_BF16 */
  int32_t dw_type;  /* LAYER_F32 or LAYER_BF16 */
  int32_t accumulate;
  int32_t pad;
} layer_linear_grad_args;

gemm_status layer_linear_backward(const layer_linear_grad_args *args, layer_cfg cfg, void *stream);

/*
 * Rows to 8-bit codes with one scale each: scale_m = max_j |x_mj| / top (the fp32
 * quotient, at least 2^-126; 1 where the row is all zeros), out = x / scale (the
 * fp32 quotient, rounded to nearest, ties to even); top is 127 for LAYER_I8 (codes
 * -127 .. 127) and 448 for LAYER_E4M3. The scale's reader multiplies: x is about
 * code * scale. A row that holds a NaN or an infinity gets a NaN scale (and NaN
 * codes, or zeros in int8). These are the operands and scales of layer_linear: of x a
 * scale for each token, of w one for each of its n rows.
 * One launch, no plan. m == 0 or n == 0 enqueues nothing (and writes no scale).
 * Errors: GEMM_E_INVALID_ARG (a NULL or misaligned pointer, an unknown type),
 * GEMM_E_SHAPE, GEMM_E_UNSUPPORTED (current device not gfx950), GEMM_E_HIP.
 */
typedef struct layer_quantize_args {
  const void *x; /* m x n, type */
  void *out;     /* m x n, out_type */
  float *scale;  /* m */
  int64_t m, n;
  int64_t ldx, ldo;
  int32_t type;     /* LAYER_F32 or LAYER_BF16 */
  int32_t out_type; /* LAYER_I8 or LAYER_E4M3 */
} layer_quantize_args;

gemm_status layer_quantize(const layer_quantize_args *args, void *stream);

/*
 * Softmax cross entropy of an output head, without its logits: with z = x . w^T
 * (m tokens, n entries of the vocabulary, any number of them),
 *   lse_m = log sum_v exp z_mv,  loss_m = lse_m - z_m,label.
 * A negative label: the row is not counted, its loss is 0 (its lse is written all
 * the same). A label of n or more is a mistake that no call can see in time: its
 * loss is NaN, and so are its gradients. Logits, maxima and sums are fp32; they
 * are taken tile by tile, 8 bytes a row and block of the vocabulary reach memory.
 * loss may be NULL. lse holds other values while the call runs and shares no
 * memory with loss. A logit of NaN gives the row NaN; w rows of -infinity work
 * where the logit is -infinity.
 * Two launches, three where products are split along k (and in parts of the rows
 * where the workspace does not hold 8 bytes a row and 128 entries for all of
 * them). m == 0 enqueues nothing.
 * Errors: GEMM_E_INVALID_ARG (a NULL or misaligned pointer, loss and lse the same),
 * GEMM_E_SHAPE (also n == 0 with rows), GEMM_E_DEVICE, GEMM_E_HIP.
 */
typedef struct layer_cross_entropy_args {
  const void *x;        /* m x k, bf16 */
  const void *w;        /* n x k, bf16 */
  const int64_t *label; /* m */
  float *lse;           /* m */
  float *loss;          /* m, or NULL */
  int64_t m, n, k;
  int64_t ldx, ldw;
} layer_cross_entropy_args;

gemm_status layer_cross_entropy(const layer_cross_entropy_args *args, layer_cfg cfg, void *stream);

/*
 * The gradient of dloss sum_m weight_m loss_m, from the forward pass's lse: with
 *   dz_mv = weight_m (exp(z_mv - lse_m) - [v = label_m])   (0 in rows not counted)
 * rounded to bf16 (the logits are computed again),
 *   dx = dloss dz . w,  dw = dloss dz^T . x (+ dw with `accumulate`, in dw's type).
 * weight (fp32, NULL: ones): one factor a token, e.g. an incoming gradient. dloss:
 * one fp32 value on the device (NULL: 1), e.g. the 1 / count of a mean; it is applied
 * in fp32 after the products. dx and dw: fp32 or bf16, NULL: not wanted. Rows that
 * are not counted, or weigh 0, have dz = 0 whatever their logits are; x must hold
 * finite values there all the same (0 times NaN is NaN in dw). In the same way an
 * entry that a row of -infinity in w masks has dz = 0, and dw takes such a w, but
 * dx needs a finite one: 0 times -infinity is NaN, in the infinite columns of every
 * row of dx.
 *
 * scratch: dz is made and used in pieces of the vocabulary, whole 256s of its
 * entries, as large as scratch_bytes allow: 2 m bytes an entry (of whole 8s) and, with more
 * than one piece and a bf16 dx, 4 m k bytes before them for dx's sum.
 * layer_cross_entropy_scratch gives the bytes for (at most) `pieces` pieces; the
 * fewer, the faster: each costs dx's sum once through memory. It is at the call's
 * disposal while the call runs, and any two calls may share it in turn.
 * Three launches a piece, six where products are split along k. With m == 0 dw is
 * zeroed (unless accumulate is set). No result depends on the order in which
 * workgroups run. The pieces' size may change the order of the sums over k, over the
 * tokens and over the vocabulary, and with it the last bits of dz, dw and dx; the room
 * for a bf16 dx's sum is not the pieces', so dw alone and dw beside such a dx may
 * differ in them.
 * Errors: as layer_cross_entropy; GEMM_E_SHAPE where scratch_bytes hold no piece.
 */
typedef struct layer_cross_entropy_grad_args {
  const void *x;        /* m x k, bf16 */
  const void *w;        /* n x k, bf16 */
  const int64_t *label; /* m */
  const float *lse;     /* m */
  const float *weight;  /* m, or NULL */
  const float *dloss;   /* 1, or NULL */
  void *dx;             /* m x k, dx_type, or NULL */
  void *dw;             /* n x k, dw_type, or NULL */
  void *scratch;        /* 16-byte aligned */
  int64_t scratch_bytes;
  int64_t m, n, k;
  int64_t ldx, ldw, lddx, lddw;
  int32_t dx_type;      /* LAYER_F32 or LAYER_BF16 */
  int32_t dw_type;      /* LAYER_F32 or LAYER_BF16 */
  int32_t accumulate;
  int32_t pad;
} layer_cross_entropy_grad_args;

/* Bytes of scratch for at most `pieces` pieces (-1: a size or `pieces` out of range). */
int64_t layer_cross_entropy_scratch(int64_t m, int64_t n, int64_t k, int32_t pieces);

gemm_status layer_cross_entropy_backward(const layer_cross_entropy_grad_args *args, layer_cfg cfg, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PTG_LAYER_H */
