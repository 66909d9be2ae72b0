// Host side of the layer operators' C ABI (include/ptg_layer.h): argument
// checks, the plan and its scratch, and the choice of kernel per call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <new>

#include "layer_internal.hpp"
#include "ptg_layer.h"

static_assert(LAYER_F32 == ptg::kTypeF32 && LAYER_BF16 == ptg::kTypeBf16 && LAYER_E4M3 == ptg::kTypeE4m3, "types");
static_assert(LAYER_ACT_NONE == ptg::kActNone && LAYER_ACT_RELU == ptg::kActRelu && LAYER_ACT_GELU == ptg::kActGelu &&
                  LAYER_ACT_GELU_TANH == ptg::kActGeluTanh && LAYER_ACT_SILU == ptg::kActSilu, "activations");

struct layer_plan {
  int device = 0;
  int cu_count = 0;
  gemm_tile_cfg tiles256 = nullptr, tiles128 = nullptr;  // the tiled products' plans
  float *ws = nullptr;             // partial sums: the 256 x 256 plan's workspace
  int64_t ws_floats = 0;
  uint32_t *d_arrivals = nullptr;  // arrival counts of the few-row product's shared tiles, zero between calls
  hipEvent_t stream_switch = nullptr;
  hipStream_t last_stream = nullptr;
  bool has_run = false;   // last_stream may hold work of the plan
  bool captured = false;  // a call was captured: replays may follow on its stream at any time
  char last_error[256] = "";  // of a fixed size: no call of the C ABI may throw
};

namespace {

constexpr int64_t kArrivals = 4096;  // tiles whose k is shared: CUs / 2 at most (rows_shape), checked at each call

gemm_status hip_fail(layer_plan *p, hipError_t e, const char *what) {
  if (p) std::snprintf(p->last_error, sizeof(p->last_error), "%s: %s", what, hipGetErrorString(e));
  return GEMM_E_HIP;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One device property read per device and process: the layer_rmsnorm call has
// no plan to keep it in.
gemm_status current_gfx950(int *cu_count) {
  constexpr int kMost = 64;
  static int cus[kMost];  // 0: not read yet; -1: another part. Every writer writes the same value.
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return GEMM_E_HIP;
  if (dev < 0 || dev >= kMost) return GEMM_E_DEVICE;
  int c = __atomic_load_n(&cus[dev], __ATOMIC_RELAXED);
  if (c == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_E_HIP;
    c = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? prop.multiProcessorCount : -1;
    __atomic_store_n(&cus[dev], c, __ATOMIC_RELAXED);
  }
  if (c < 0) return GEMM_E_UNSUPPORTED;
  *cu_count = c;
  return GEMM_OK;
}

gemm_status check_device(layer_plan *p) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(p, e, "hipGetDevice");
  return dev == p->device ? GEMM_OK : GEMM_E_DEVICE;
}

// The plan's scratch serves one call at a time: a call on another stream than
// the last one first waits, on the device, for what that stream holds so far.
gemm_status order_after_last_stream(layer_plan *p, hipStream_t s) {
  if (p->has_run && s != p->last_stream) {
    hipError_t e = hipEventRecord(p->stream_switch, p->last_stream);
    if (e != hipSuccess) return hip_fail(p, e, "hipEventRecord(stream switch)");
    e = hipStreamWaitEvent(s, p->stream_switch, 0);
    if (e != hipSuccess) return hip_fail(p, e, "hipStreamWaitEvent(stream switch)");
  }
  hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(s, &capture);
  if (e != hipSuccess) return hip_fail(p, e, "hipStreamIsCapturing");
  p->captured = p->captured || capture != hipStreamCaptureStatusNone;
  p->last_stream = s;
  p->has_run = true;
  return GEMM_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stream_type(int32_t t) { return t == LAYER_F32 || t == LAYER_BF16; }

// Sizes of an m x n matrix whose rows are multiples of `step` elements.
bool bad_size(int64_t m, int64_t n, int64_t step) {
  return m < 0 || n < 0 || m > LAYER_MAX_ROWS || n > LAYER_MAX_COLS || n % step != 0;
}
// A row stride of a matrix with m rows of n elements (not looked at with one row, or rows of no elements).
bool bad_stride(int64_t ld, int64_t m, int64_t n, int64_t step) {
  return m > 1 && n > 0 && (ld < n || ld > LAYER_MAX_COLS || ld % step != 0);
}

// The GEMM plan of a layer plan: the library's defaults with a split tail.
gemm_status make_tiles(gemm_tile_cfg *out, int32_t edge, int32_t device) {
  gemm_tile_desc d;
  gemm_status st = gemm_default_desc(&d, edge, device);
  if (st != GEMM_OK) return st;
  d.tail_split = GEMM_TAIL_SPLIT_AUTO;
  d.max_groups = 1;
  return gemm_create(out, &d);
}

// How a product of T output tiles and nk k-steps (32 deep) runs: tile edge, and
// the K-chunks S that the tiles from `base` on are split into.
struct TileChoice { int edge; int32_t split; int64_t base; double us; };

// The choice is the least of the times that these fits give, in microseconds (256
// CUs; fitted over m = 100 .. 4096, n = 1024 .. 16384, k = 768 .. 8192 in each
// form). They compare choices and do not foretell a call: of 86 products over twice
// that range (bf16, e4m3, dx and dw; no epilogue terms) the measured time was 1.11
// times the fit at the median, 0.95 and 2.0 at the first and last tenth, and within
// 15% for 56% of them. What they leave out: a unit's fill, drain and writes are
// counted once a launch and not again for the further units of a CU, nor are the
// bytes of a large output, so that few k-steps a tile take up to 2.5 times the fit
// (8418 x 8912 x 136: 37 and 87) and dw over few rows, which writes fp32, up to 6.5;
// nor are the terms of the epilogue. 8192^3: 694 and 728, in e4m3 591 and 636.
//   - a k-step of a 128 x 128 tile: NT and NN 0.28 with one tile a CU at a time
//     (their stages fill its LDS), e4m3 0.41; TN 0.23, and with two tiles a CU
//     together 0.44; 8 to fill and drain, 2 less where one wave takes every unit;
//   - a k-step of a 256 x 256 tile: from the first to the second figure as more
//     CUs work (power and memory shared): 0.48 to 0.66, e4m3 0.9 to 1.12; 18 to
//     fill and drain;
//   - rows of a k-contiguous operand that do not start on 64-byte lines: 128 x 128
//     steps 1.33 times as long, 256 x 256 ones 1.13 (NN, with one such operand, 1.05;
//     e4m3, which takes half the bytes a product, 1.1 in both);
//   - splitting: 4 for the second launch, and each chunk's sums written and read,
//     0.02 a chunk of 128 x 128, 0.06 of 256 x 256.
// Both sides where it matters (NT): 512 x 8192 x 8192, 256 tiles of 128: 79 us, 64
// of 256 in 4 chunks: 76; 1024 x 8192 x 8192, 512 of 128: 155, 128 of 256: 154, in
// 2 chunks: 118; 1024 x 4096 x 4096, 256 of 128: 44, 64 of 256 in 4 chunks: 54;
// 256 x 4096 x 4096, 64 of 128: 43, in 4 chunks: 24; 100 x 1024 x 8192, 8 of 128:
// 62, in 8 chunks: 20; 1000 x 4104 x 2056 (rows off the lines), 264 of 128: 58, the
// last eight in 6 chunks: 47, 68 of 256 in 3 chunks: 55 (chosen: the last eight in 13
// chunks, whose fit is 40 and whose time 49).
TileChoice choose_tiles(const ptg::ProductArgs &a, int form, int64_t cus) {
  const bool e8 = form == ptg::kFormNTE4m3, tn = form == ptg::kFormTN;
  const int64_t nk = ceil_div(e8 ? a.k / 2 : a.k, 32), line = e8 ? 64 : 32;
  const bool off_line = !tn && ((a.m > 1 && a.lda % line != 0) || (form != ptg::kFormNN && a.ldb % line != 0));
  const double slow128 = off_line ? (e8 ? 1.1 : 1.33) : 1.0, slow256 = off_line ? (e8 ? 1.1 : form == ptg::kFormNT ? 1.13 : 1.05) : 1.0;
  TileChoice best = {256, 1, 0, 1e300};
  for (const int edge : {128, 256}) {
    const int64_t T = ceil_div(a.m, edge) * ceil_div(a.n, edge);
    const int64_t slots = edge == 256 ? cus : 2 * cus;  // chunks the workspace holds
    // the time of `units` tiles or chunks of `steps` k-steps
    auto run = [&](int64_t units, int64_t steps) {
      const double load = (double)units / (double)cus, rounds = (double)ceil_div(units, cus);
      double step;
      if (edge == 256) step = slow256 * (load <= 1.0 ? (e8 ? 0.9 + 0.22 * load * load : 0.48 + 0.18 * load * load) : (e8 ? 1.12 : 0.66) * rounds);
      else if (tn) step = load <= 1.0 ? 0.23 : std::max(0.44, 0.23 * load);
      else step = slow128 * (e8 ? 0.41 : 0.28) * rounds;
      return (double)steps * step;
    };
    const int64_t resident = cus * ptg::product_workgroups(edge, form);
    auto fixed = [&](int64_t units) { return (edge == 256 ? 18.0 : 8.0) - (units <= resident ? 2.0 : 0.0); };
    const double join = edge == 256 ? 0.06 : 0.02;
    const double whole = fixed(T) + run(T, nk);
    if (whole < best.us) best = {edge, 1, 0, whole};
    // all tiles, or those of the partial last wave
    const int64_t waves = T / cus * cus;
    for (const int64_t base : {(int64_t)0, waves}) {
      const int64_t r = T - base;
      if (r == 0 || (base != 0 && edge == 128 && tn)) continue;  // (TN: small tiles' last wave shares the CUs of the wave before)
      const double before = base ? run(base, nk) : 0.0;
      for (int32_t S = 2; S <= 32 && r * S <= slots && nk / S >= 4; ++S) {
        const double us = fixed(base + r * S) + before + run(r * S, ceil_div(nk, S)) + 4.0 + join * (double)(r * S);
        if (us < best.us) best = {edge, S, base, us};
      }
      if (base == waves) break;  // fewer tiles than CUs: both are the same
    }
  }
  return best;
}

gemm_status run_tiles(layer_plan *p, const ptg::ProductArgs &a, int form, hipStream_t s) {
  const TileChoice c = choose_tiles(a, form, p->cu_count);
  gemm_tile_cfg t = c.edge == 256 ? p->tiles256 : p->tiles128;
  gemm_status st = ptg::plan_run_product(t, a, form, c.split, c.base, s);
  if (st == GEMM_E_HIP) std::snprintf(p->last_error, sizeof(p->last_error), "%s", gemm_last_hip_error(t));
  return st;
}

// The stride the kernels get: a matrix of one row has its row's length, whatever the caller said.
int64_t stride_of(int64_t ld, int64_t m, int64_t n) { return m > 1 && n > 0 ? ld : std::max<int64_t>(n, 8); }

// Partial sums of n columns over at most `wanted` rows: as many rows as the
// workspace holds (a chunk of 256 x 256 a CU: 16 rows of the widest matrix).
int64_t partial_rows(const layer_plan *p, int64_t wanted, int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>(wanted, p->ws_floats / std::max<int64_t>(n, 1)));
}

}  // namespace

extern "C" {

gemm_status layer_create(layer_cfg *out, int32_t device) {
  if (!out) return GEMM_E_INVALID_ARG;
  *out = nullptr;
  int ndev = 0, cur = -1;
  if (hipGetDeviceCount(&ndev) != hipSuccess) return GEMM_E_HIP;
  if (device < 0 || device >= ndev) return GEMM_E_INVALID_ARG;
  if (hipGetDevice(&cur) != hipSuccess) return GEMM_E_HIP;
  if (cur != device) return GEMM_E_DEVICE;
  int cus = 0;
  gemm_status st = current_gfx950(&cus);
  if (st != GEMM_OK) return st;
  layer_plan *p = new (std::nothrow) layer_plan();
  if (!p) return GEMM_E_NOMEM;
  p->device = device;
  p->cu_count = cus;
  if (hipMalloc(&p->d_arrivals, sizeof(uint32_t) * (size_t)kArrivals) != hipSuccess) {
    p->d_arrivals = nullptr;
    layer_destroy(p);
    return GEMM_E_NOMEM;
  }
  // waited for: a first call's stream need not wait for the null stream
  if (hipMemset(p->d_arrivals, 0, sizeof(uint32_t) * (size_t)kArrivals) != hipSuccess || hipStreamSynchronize(nullptr) != hipSuccess) {
    layer_destroy(p);
    return GEMM_E_HIP;
  }
  if (hipEventCreateWithFlags(&p->stream_switch, hipEventDisableTiming) != hipSuccess) {
    p->stream_switch = nullptr;
    layer_destroy(p);
    return GEMM_E_HIP;
  }
  if ((st = make_tiles(&p->tiles256, 256, device)) != GEMM_OK || (st = make_tiles(&p->tiles128, 128, device)) != GEMM_OK) {
    layer_destroy(p);
    return st;
  }
  p->ws = ptg::plan_workspace(p->tiles256, &p->ws_floats);
  *out = p;
  return GEMM_OK;
}

gemm_status layer_destroy(layer_cfg p) {
  if (!p) return GEMM_OK;
  if (p->has_run) (void)hipStreamSynchronize(p->last_stream);
  (void)gemm_destroy(p->tiles256);
  (void)gemm_destroy(p->tiles128);
  if (p->stream_switch) (void)hipEventDestroy(p->stream_switch);
  if (p->d_arrivals) (void)hipFree(p->d_arrivals);
  delete p;
  return GEMM_OK;
}

gemm_status layer_sync(layer_cfg p) {
  if (!p) return GEMM_E_INVALID_ARG;
  if (!p->has_run) return GEMM_OK;
  hipError_t e = hipStreamSynchronize(p->last_stream);
  if (e != hipSuccess) return hip_fail(p, e, "hipStreamSynchronize");
  p->has_run = p->captured;  // nothing left to wait for: the stream may end
  gemm_status st = GEMM_OK;
  for (gemm_tile_cfg t : {p->tiles256, p->tiles128}) {
    const gemm_status one = ptg::plan_status(t);
    if (one == GEMM_OK) continue;
    std::snprintf(p->last_error, sizeof(p->last_error), "%s", gemm_last_hip_error(t));
    st = one;
  }
  return st;
}

const char *layer_last_hip_error(layer_cfg p) { return p ? p->last_error : ""; }

gemm_status layer_rmsnorm(const layer_rmsnorm_args *a, void *stream) {
  if (!a) return GEMM_E_INVALID_ARG;
  if (!stream_type(a->type) || (a->out_type != LAYER_E4M3 && !stream_type(a->out_type)) ||
      (a->weight && !stream_type(a->weight_type)) || !(a->eps >= 0.0f))
    return GEMM_E_INVALID_ARG;
  if (bad_size(a->m, a->n, 8) || a->n > LAYER_MAX_NORM_COLS || bad_stride(a->ldx, a->m, a->n, 8) ||
      (a->residual && bad_stride(a->ldr, a->m, a->n, 8)) || (a->sum_out && bad_stride(a->lds, a->m, a->n, 8)) ||
      bad_stride(a->ldo, a->m, a->n, 8))
    return GEMM_E_SHAPE;
  if ((a->out_type == LAYER_E4M3) != (a->scale != nullptr) && (a->m > 0 || a->scale)) return GEMM_E_INVALID_ARG;
  if (a->m == 0 || a->n == 0) return GEMM_OK;
  if (!a->x || !a->out || !aligned16(a->x) || !aligned16(a->residual) || !aligned16(a->weight) || !aligned16(a->sum_out) ||
      !aligned16(a->out) || (reinterpret_cast<uintptr_t>(a->scale) & 3u))
    return GEMM_E_INVALID_ARG;
  int cus = 0;
  gemm_status st = current_gfx950(&cus);
  if (st != GEMM_OK) return st;
  ptg::NormArgs k;
  std::memset(&k, 0, sizeof(k));
  k.x = a->x;
  k.residual = a->residual;
  k.weight = a->weight;
  k.sum_out = a->sum_out;
  k.out = a->out;
  k.scale = a->scale;
  k.ldx = stride_of(a->ldx, a->m, a->n);
  k.ldr = stride_of(a->ldr, a->m, a->n);
  k.lds = stride_of(a->lds, a->m, a->n);
  k.ldo = stride_of(a->ldo, a->m, a->n);
  k.m = (int32_t)a->m;
  k.n = (int32_t)a->n;
  k.type = a->type;
  k.weight_type = a->weight_type;
  k.out_type = a->out_type;
  k.eps = a->eps;
  return ptg::launch_rmsnorm(k, cus, static_cast<hipStream_t>(stream)) == hipSuccess ? GEMM_OK : GEMM_E_HIP;
}

gemm_status layer_rmsnorm_backward(const layer_rmsnorm_grad_args *a, layer_cfg p, void *stream) {
  if (!a || !p) return GEMM_E_INVALID_ARG;
  if (!stream_type(a->type) || !stream_type(a->dy_type) || (a->weight && !stream_type(a->weight_type)) || !(a->eps >= 0.0f) ||
      a->accumulate < 0 || a->accumulate > 1)
    return GEMM_E_INVALID_ARG;
  if (bad_size(a->m, a->n, 8) || a->n > LAYER_MAX_NORM_COLS || bad_stride(a->lddy, a->m, a->n, 8) ||
      bad_stride(a->lds, a->m, a->n, 8) || (a->dsum && bad_stride(a->lddsum, a->m, a->n, 8)) ||
      (a->dx && bad_stride(a->lddx, a->m, a->n, 8)))
    return GEMM_E_SHAPE;
  if (!aligned16(a->dy) || !aligned16(a->s) || !aligned16(a->weight) || !aligned16(a->dsum) || !aligned16(a->dx) ||
      !aligned16(a->dweight) || (a->m > 0 && a->n > 0 && (!a->dy || !a->s)))
    return GEMM_E_INVALID_ARG;
  gemm_status st = check_device(p);
  if (st != GEMM_OK) return st;
  if (a->n == 0 || (!a->dx && !a->dweight) || (a->m == 0 && (!a->dweight || a->accumulate))) return GEMM_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = order_after_last_stream(p, s);
  if (st != GEMM_OK) return st;
  int rows = 0;
  hipError_t e;
  if (a->m > 0) {
    ptg::NormGradArgs k;
    std::memset(&k, 0, sizeof(k));
    k.dy = a->dy;
    k.s = a->s;
    k.weight = a->weight;
    k.dsum = a->dsum;
    k.dx = a->dx;
    k.partial = a->dweight ? p->ws : nullptr;
    k.lddy = stride_of(a->lddy, a->m, a->n);
    k.lds = stride_of(a->lds, a->m, a->n);
    k.lddsum = stride_of(a->lddsum, a->m, a->n);
    k.lddx = stride_of(a->lddx, a->m, a->n);
    k.m = (int32_t)a->m;
    k.n = (int32_t)a->n;
    k.type = a->type;
    k.dy_type = a->dy_type;
    k.weight_type = a->weight_type;
    k.eps = a->eps;
    // at most 8 x CUs groups of rows of at most 1024, or 2 x CUs of 4096, or CUs
    // of 32768 elements: within the workspace
    rows = ptg::rmsnorm_partial_rows(k.m, k.n, p->cu_count);
    if ((int64_t)rows * a->n > p->ws_floats) return GEMM_E_SHAPE;
    e = ptg::launch_rmsnorm_backward(k, p->cu_count, s);
    if (e != hipSuccess) return hip_fail(p, e, "rmsnorm backward");
  }
  if (a->dweight) {
    e = ptg::launch_column_sum(p->ws, rows, (int32_t)a->n, a->dweight, a->accumulate, s);
    if (e != hipSuccess) return hip_fail(p, e, "column sum");
  }
  return GEMM_OK;
}

gemm_status layer_linear(const layer_linear_args *a, layer_cfg p, void *stream) {
  if (!a || !p) return GEMM_E_INVALID_ARG;
  const bool e8 = a->in_type == LAYER_E4M3;
  if ((!e8 && a->in_type != LAYER_BF16) || (a->bias && !stream_type(a->bias_type)) ||
      (a->residual && !stream_type(a->residual_type)) || !stream_type(a->out_type) || a->activation < LAYER_ACT_NONE ||
      a->activation > LAYER_ACT_SILU || (!e8 && (a->x_scale || a->w_scale)))
    return GEMM_E_INVALID_ARG;
  const int64_t step = e8 ? 16 : 8;
  if (bad_size(a->m, a->n, 8) || bad_size(a->n, a->k, step) || a->n > LAYER_MAX_COLS || bad_stride(a->ldx, a->m, a->k, step) ||
      bad_stride(a->ldw, a->n, a->k, step) || bad_stride(a->ldo, a->m, a->n, 8) ||
      (a->residual && bad_stride(a->ldr, a->m, a->n, 8)) || (a->pre && bad_stride(a->ldp, a->m, a->n, 8)))
    return GEMM_E_SHAPE;
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->x_scale) || !aligned16(a->w_scale) || !aligned16(a->bias) ||
      !aligned16(a->residual) || !aligned16(a->pre) || !aligned16(a->out))
    return GEMM_E_INVALID_ARG;
  const bool empty = a->m == 0 || a->n == 0;
  if (!empty && (!a->out || (a->k > 0 && (!a->x || !a->w)))) return GEMM_E_INVALID_ARG;
  gemm_status st = check_device(p);
  if (st != GEMM_OK || empty) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = order_after_last_stream(p, s);
  if (st != GEMM_OK) return st;
  ptg::ProductArgs k;
  std::memset(&k, 0, sizeof(k));
  k.a = a->x;
  k.b = a->w;
  k.lda = stride_of(a->ldx, a->m, a->k);
  k.ldb = stride_of(a->ldw, a->n, a->k);
  k.m = (int32_t)a->m;
  k.n = (int32_t)a->n;
  k.k = (int32_t)a->k;
  k.ep.row_scale = a->x_scale;
  k.ep.col_scale = a->w_scale;
  k.ep.bias = a->bias;
  k.ep.residual = a->residual;
  k.ep.pre = a->pre;
  k.ep.out = a->out;
  k.ep.ldr = stride_of(a->ldr, a->m, a->n);
  k.ep.ldp = stride_of(a->ldp, a->m, a->n);
  k.ep.ldo = stride_of(a->ldo, a->m, a->n);
  k.ep.bias_type = a->bias_type;
  k.ep.residual_type = a->residual_type;
  k.ep.out_type = a->out_type;
  k.ep.act = a->activation;
  if (ptg::rows_preferred(k, e8)) {
    int64_t tiles = 0;
    if (ptg::rows_partial_floats(k, e8, p->cu_count, &tiles) > p->ws_floats || tiles > kArrivals) return GEMM_E_SHAPE;
    hipError_t e = ptg::launch_rows(k, e8, p->ws, p->d_arrivals, p->cu_count, s);
    return e == hipSuccess ? GEMM_OK : hip_fail(p, e, "linear");
  }
  return run_tiles(p, k, e8 ? ptg::kFormNTE4m3 : ptg::kFormNT, s);
}

gemm_status layer_activation_backward(const layer_activation_grad_args *a, layer_cfg p, void *stream) {
  if (!a || !p) return GEMM_E_INVALID_ARG;
  if (a->activation < LAYER_ACT_NONE || a->activation > LAYER_ACT_SILU || a->accumulate < 0 || a->accumulate > 1)
    return GEMM_E_INVALID_ARG;
  const bool none = a->activation == LAYER_ACT_NONE;
  if (bad_size(a->m, a->n, 8) || bad_stride(a->lddo, a->m, a->n, 8) || (!none && a->pre && bad_stride(a->ldp, a->m, a->n, 8)) ||
      (a->dpre && bad_stride(a->lddp, a->m, a->n, 8)))
    return GEMM_E_SHAPE;
  if (!aligned16(a->dout) || (!none && !aligned16(a->pre)) || !aligned16(a->dpre) || !aligned16(a->dbias) ||
      (a->m > 0 && a->n > 0 && (!a->dout || (!none && !a->pre))))
    return GEMM_E_INVALID_ARG;
  gemm_status st = check_device(p);
  if (st != GEMM_OK) return st;
  if (a->n == 0 || (!a->dpre && !a->dbias) || (a->m == 0 && (!a->dbias || a->accumulate))) return GEMM_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = order_after_last_stream(p, s);
  if (st != GEMM_OK) return st;
  int64_t groups = 0;
  hipError_t e;
  if (a->m > 0) {
    ptg::ActGradArgs k;
    std::memset(&k, 0, sizeof(k));
    k.dout = a->dout;
    k.pre = a->pre;
    k.dpre = a->dpre;
    k.partial = a->dbias ? p->ws : nullptr;
    k.lddo = stride_of(a->lddo, a->m, a->n);
    k.ldp = stride_of(a->ldp, a->m, a->n);
    k.lddp = stride_of(a->lddp, a->m, a->n);
    k.m = (int32_t)a->m;
    k.n = (int32_t)a->n;
    k.act = a->activation;
    // eight workgroups a CU, each with 16 rows at least (four a wave)
    const int64_t strips = ceil_div(a->n, 512);
    groups = partial_rows(p, std::min<int64_t>(ceil_div((int64_t)p->cu_count * 8, strips), ceil_div(a->m, 16)), a->n);
    k.rows_per_group = (int32_t)ceil_div(a->m, groups);
    groups = ceil_div(a->m, k.rows_per_group);
    e = ptg::launch_activation_backward(k, (int)groups, s);
    if (e != hipSuccess) return hip_fail(p, e, "activation backward");
  }
  if (a->dbias) {
    e = ptg::launch_column_sum(p->ws, (int)groups, (int32_t)a->n, a->dbias, a->accumulate, s);
    if (e != hipSuccess) return hip_fail(p, e, "column sum");
  }
  return GEMM_OK;
}

gemm_status layer_linear_backward(const layer_linear_grad_args *a, layer_cfg p, void *stream) {
  if (!a || !p) return GEMM_E_INVALID_ARG;
  if ((a->dx && !stream_type(a->dx_type)) || (a->dw && !stream_type(a->dw_type)) || a->accumulate < 0 || a->accumulate > 1)
    return GEMM_E_INVALID_ARG;
  if (bad_size(a->m, a->n, 8) || bad_size(a->m, a->k, 8) || bad_stride(a->lddp, a->m, a->n, 8) ||
      (a->dw && bad_stride(a->ldx, a->m, a->k, 8)) || (a->dx && bad_stride(a->ldw, a->n, a->k, 8)) ||
      (a->dx && bad_stride(a->lddx, a->m, a->k, 8)) || (a->dw && bad_stride(a->lddw, a->n, a->k, 8)))
    return GEMM_E_SHAPE;
  if (!aligned16(a->dpre) || (a->dw && !aligned16(a->x)) || (a->dx && !aligned16(a->w)) || !aligned16(a->dx) || !aligned16(a->dw))
    return GEMM_E_INVALID_ARG;
  const bool any_dx = a->dx && a->m > 0 && a->k > 0;
  const bool any_dw = a->dw && a->n > 0 && a->k > 0 && !(a->m == 0 && a->accumulate);
  if ((any_dx && a->n > 0 && (!a->dpre || !a->w)) || (any_dw && a->m > 0 && (!a->dpre || !a->x))) return GEMM_E_INVALID_ARG;
  gemm_status st = check_device(p);
  if (st != GEMM_OK || (!any_dx && !any_dw)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = order_after_last_stream(p, s);
  if (st != GEMM_OK) return st;
  ptg::ProductArgs k;
  if (any_dx) {
    std::memset(&k, 0, sizeof(k));
    k.a = a->dpre;
    k.b = a->w;
    k.lda = stride_of(a->lddp, a->m, a->n);
    k.ldb = stride_of(a->ldw, a->n, a->k);
    k.m = (int32_t)a->m;
    k.n = (int32_t)a->k;
    k.k = (int32_t)a->n;
    k.ep.out = a->dx;
    k.ep.ldo = stride_of(a->lddx, a->m, a->k);
    k.ep.out_type = a->dx_type;
    st = run_tiles(p, k, ptg::kFormNN, s);
    if (st != GEMM_OK) return st;
  }
  if (any_dw) {
    std::memset(&k, 0, sizeof(k));
    k.a = a->dpre;
    k.b = a->x;
    k.lda = stride_of(a->lddp, a->m, a->n);
    k.ldb = stride_of(a->ldx, a->m, a->k);
    k.m = (int32_t)a->n;
    k.n = (int32_t)a->k;
    k.k = (int32_t)a->m;
    k.ep.out = a->dw;
    k.ep.ldo = stride_of(a->lddw, a->n, a->k);
    k.ep.out_type = a->dw_type;
    k.ep.residual = a->accumulate ? a->dw : nullptr;
    k.ep.ldr = stride_of(a->lddw, a->n, a->k);
    k.ep.residual_type = a->dw_type;
    st = run_tiles(p, k, ptg::kFormTN, s);
    if (st != GEMM_OK) return st;
  }
  return GEMM_OK;
}

}  // extern "C"
