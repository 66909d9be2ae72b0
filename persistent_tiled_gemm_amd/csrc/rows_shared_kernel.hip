// The product for some rows (up to 64) with x in LDS: int8 operands with the layer
// operators' epilogue, and bf16 operands with a cross entropy's end (see loss_kernel.hip).
//
// rows_kernel.hip reads w and x alike from memory into MFMA operands. x comes from the
// caches, but returns in turn with w, and so takes its share of the loads that a CU can
// have under way: 8192^2 in int8 took 15.4 us for one row of x and 21 for 24, what w and
// all the copies of x take at 5.8 TB/s. Here a workgroup owns 16 rows of w a wave and
// one share of k (of S): it brings x's share to LDS once for all its waves, and each
// wave then streams its own rows of w over the whole share, with nothing else in its
// queue. (8192^2: 24 rows 22.0 -> 17.9 us, 64 rows 27.2 -> 20.9; 16384 x 4096: 31.7 -> 20.2.)
// No wave's sums meet another's; the shares of k meet in the plan's workspace, as in
// rows_kernel.hip. Bound by latency at few rows (24 rows: 67 MB of w, 11.6 us at the rate of a
// plain read): x's way to LDS comes before the first product, the meeting after the last.
//
// LDS: 256-byte segments, segment by segment, x's rows one after the other in each; 16-byte
// chunk c of row r sits in slot c ^ (r mod 16), so that 16 rows' reads of one chunk are
// free of bank conflicts.
#include <algorithm>

#include "layer_device.hpp"
#include "loss_device.hpp"

namespace ptg {

static constexpr int kSharedBytes = 128 * 1024;
static constexpr int kPolicyStream = 2;  // nt: w is read once

template <bool I8>
__device__ __forceinline__ f32x4 mfma_step(const i32x4 &w, const i32x4 &x, const f32x4 &acc) {
  if constexpr (I8) return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, __builtin_bit_cast(i32x4, acc), 0, 0, 0));
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}
template <bool I8>
__device__ __forceinline__ f32x4 add_parts(const f32x4 &a, const f32x4 &b) {
  if constexpr (I8) return __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, a) + __builtin_bit_cast(i32x4, b));
  else return a + b;
}

// I8: int8 operands and the layer operators' epilogue; otherwise bf16 and a cross entropy's.
// Lengths and strides in bytes from here on.
template <bool I8, int MT, int WAVES, int DEPTH>
__device__ __forceinline__ void rows_shared(const RowsArgs &a, const LossTerms &loss) {
  constexpr int kRows = 16 * MT;
  constexpr uint32_t kSize = I8 ? 1u : 2u;
  const uint32_t bytes = (uint32_t)a.k * kSize, ldx = (uint32_t)a.ldx * kSize, ldw = (uint32_t)a.ldw * kSize;
  __shared__ __attribute__((aligned(1024))) unsigned char xs[kSharedBytes];
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = wave_uniform(tid >> 6);
  const uint32_t tile = blockIdx.x, part = blockIdx.y;
  const int32_t n0 = (int32_t)(tile * WAVES + wave) * 16;
  const uint32_t row = lane & 15u, group = lane >> 4;

  // the workgroup's share of k, in segments of 256 bytes (four steps of 64)
  const uint32_t segs = (bytes + 255u) / 256u;
  const uint32_t g0 = segs * part / gridDim.y, count = segs * (part + 1u) / gridDim.y - g0;
  // each wave starts part-way into the share and wraps around, so that the waves spread
  // over the memory channels
  const uint32_t rot = count > 1u ? (((tile * (uint32_t)WAVES + wave) * 2654435761u) >> 16) % count : 0u;

  // ---- x to LDS: a load moves four rows' segment
  {
    const i32x4 xr = make_rsrc_words(a.x);
    const uint32_t base = lds_addr(xs);
    const uint32_t loads = count * (uint32_t)(kRows / 4);
    for (uint32_t i = wave; i < loads; i += WAVES) {
      const uint32_t seg = i / (uint32_t)(kRows / 4), r = (i % (uint32_t)(kRows / 4)) * 4u + group;
      const uint32_t at = (g0 + seg) * 256u + (row ^ (r & 15u)) * 16u;
      load16_to_lds(xr, base + i * 1024u, (int32_t)r < a.m && at < bytes ? r * ldx + at : kBufOob);
    }
  }

  // ---- w: DEPTH segments of the wave's rows under way. Segments past the share are asked
  // for out of range (zeros, no traffic), so that every turn of the loop is alike and waits for
  // the oldest segment alone. They are not multiplied: LDS holds no zeros of x for them, and 0
  // times an infinity is NaN.
  const __amdgpu_buffer_rsrc_t wr = make_rsrc((const unsigned char *)a.w + (size_t)n0 * (size_t)ldw);
  const bool w_in = n0 + (int32_t)row < a.n;
  const uint32_t w_row = row * ldw;  // byte offset of the lane's row
  // bf16: a sum for every second or fourth step, so that a chain of fp32 additions is no longer than
  // in rows_kernel.hip, where the waves split k (one sum: a fifth more error at k = 4096)
  constexpr int kSums = I8 ? 1 : MT == 4 ? 2 : 4;
  f32x4 sums[MT][kSums] = {};  // (int8: the bits of integers)
  i32x4 w[DEPTH][4];
  auto seg_of = [&](uint32_t g) -> uint32_t { return g + rot < count ? g + rot : g + rot - count; };
  auto load = [&](int d, uint32_t g) {
    const uint32_t first = (g0 + seg_of(g)) * 256u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t at = first + 64u * (uint32_t)u + 16u * group;
      const bool in = w_in && g < count && at < bytes;
      w[d][u] = __builtin_amdgcn_raw_buffer_load_b128(wr, in ? (int)(w_row + at) : (int)kBufOob, 0, kPolicyStream);
    }
  };
  const uint32_t off = row * 256u + ((group ^ row) << 4);  // of the lane's chunk in a segment, first step
  auto multiply = [&](int d, uint32_t g) {
    const unsigned char *seg = xs + seg_of(g) * (uint32_t)(kRows * 256);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const i32x4 x = *(const i32x4 *)(seg + (off ^ (uint32_t)(64 * u)) + t * 16 * 256);
        sums[t][u % kSums] = mfma_step<I8>(w[d][u], x, sums[t][u % kSums]);
      }
  };
  if (count > 0) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, (uint32_t)d);
    // x has landed once no more loads are under way than those
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(DEPTH * 4) : "memory");
    wg_barrier();
    uint32_t g = 0;
    for (; g + DEPTH <= count; g += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        multiply(d, g + (uint32_t)d);
        load(d, g + (uint32_t)(d + DEPTH));
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
      if (g + (uint32_t)d < count) multiply(d, g + (uint32_t)d);
  }

  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int h = kSums / 2; h > 0; h /= 2)
#pragma unroll
      for (int q = 0; q < h; ++q) sums[t][q] = add_parts<I8>(sums[t][q], sums[t][q + h]);
    acc[t] = sums[t][0];
  }

  // ---- the shares of k meet: each part through to memory, a relaxed count, and the last
  // workgroup of the tile adds the parts, in order (integers give the same in any)
  const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.partial);
  constexpr uint32_t kSlots = (uint32_t)(WAVES * MT * 64);
  const uint32_t mine = wave * (uint32_t)(MT * 64) + lane;
  if (gridDim.y > 1) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
      store16_agent(pr, ((tile * gridDim.y + part) * kSlots + mine + (uint32_t)t * 64u) * 16u, acc[t]);
    wait_vmem_all();
    __syncthreads();
    if (tid == 0) {
      const uint32_t before = __hip_atomic_fetch_add(&a.arrivals[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = before + 1u == gridDim.y ? 1u : 0u;
      if (last) __hip_atomic_store(&a.arrivals[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (wave_uniform(last) == 0) return;
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t p = 0; p < gridDim.y; ++p) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = add_parts<I8>(acc[t], load16_agent(pr, ((tile * gridDim.y + p) * kSlots + mine + (uint32_t)t * 64u) * 16u));
    }
  }
  if constexpr (!I8) {
    // a lane holds four columns of row 16 t + row: the wave's 16 of a row are in four lanes.
    // The waves' maxima and sums meet in LDS (x is done with), one block a workgroup.
    float2 *meet = (float2 *)xs;  // [row][wave]
    __syncthreads();
    const int32_t first = n0 + 4 * (int32_t)group;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int32_t m = 16 * t + (int32_t)row;
      const int64_t label = m < a.m ? loss.label[m] : -1;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (first + q < a.n && label == first + q) loss.picked[m] = acc[t][q];
        top = first + q < a.n ? fmaxf(top, acc[t][q]) : top;
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float offset = offset_of(top);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += first + q < a.n ? __builtin_amdgcn_exp2f(fmaf(acc[t][q], kLog2E, -offset)) : 0.0f;
      sum = put_right(sum, top, offset);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (group == 0) meet[(uint32_t)m * WAVES + wave] = make_float2(top, sum);
    }
    __syncthreads();
    const int32_t m = (int32_t)tid;
    if (m >= a.m || m >= kRows) return;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) top = fmaxf(top, meet[m * WAVES + v].x);
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += rescaled(meet[m * WAVES + v].y, meet[m * WAVES + v].x, top);
    loss.partial[(size_t)tile * (size_t)a.m + m] = make_float2(top, sum);
    return;
  }
  // ---- epilogue: four columns of one row at a time
  const EpilogueArgs &e = a.ep;
  const int32_t n = n0 + 4 * (int32_t)group;
  if (n >= a.n) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = 16 * t + (int32_t)row;
    if (m >= a.m) continue;
    f32x4 z = __builtin_convertvector(__builtin_bit_cast(i32x4, acc[t]), f32x4);
    if (e.row_scale) z *= e.row_scale[m];
    if (e.col_scale) z *= *(const f32x4 *)(e.col_scale + n);
    if (e.bias) z += load4_as(e.bias, e.bias_type, n);
    if (e.pre) store4((__bf16 *)e.pre + m * e.ldp + n, z);
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] = act_f32(e.act, z[q]);
    if (e.residual) z += load4_as(e.residual, e.residual_type, m * e.ldr + n);
    if (e.out_type == kTypeF32) *(f32x4 *)((float *)e.out + m * e.ldo + n) = z;
    else store4((__bf16 *)e.out + m * e.ldo + n, z);
  }
}

template <int MT, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void ptg_rows_shared_i8_kernel(const RowsArgs a) {
  rows_shared<true, MT, WAVES, DEPTH>(a, LossTerms{});
}
template <int MT, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void ptg_rows_shared_loss_kernel(const RowsArgs a, const LossTerms loss) {
  rows_shared<false, MT, WAVES, DEPTH>(a, loss);
}

// The shape of a call: 16-row blocks of x, the waves of a workgroup (16 rows of w each) and
// the shares of k: as many as bring the workgroups to the CUs' number, and as x needs to
// fit. Up to 32 rows and 128 MiB of w four waves with four segments under way; more of
// either take eight with two, so that fewer workgroups hold copies of x (int8 8192^2, 64 rows:
// four 24.2 us, eight 20.9; 32768 x 8192, 24 rows: 63.9 and 54.5; 16384 x 4096, 32 rows: 16.2 and
// 17.3; the loss of 16384 x 8192, 24 rows: 66.8 and 58.6, of 16384 x 1024, 20 rows: 13.0 and 14.0).
struct SharedShape { int mt, waves; int64_t tiles, split; };
static SharedShape shared_shape(const ProductArgs &p, int type, int cu_count) {
  SharedShape f;
  f.mt = p.m <= 16 ? 1 : p.m <= 32 ? 2 : 4;
  f.waves = f.mt == 4 || (int64_t)p.n * p.k * (type == kTypeI8 ? 1 : 2) >= (int64_t)128 << 20 ? 8 : 4;
  f.tiles = (p.n + 16 * f.waves - 1) / (16 * f.waves);
  const int64_t segs = ((int64_t)p.k * (type == kTypeI8 ? 1 : 2) + 255) / 256, fits = kSharedBytes / (f.mt * 16 * 256);
  f.split = std::max<int64_t>({1, std::min<int64_t>({cu_count / f.tiles, segs, 16}), (segs + fits - 1) / fits});
  return f;
}

int64_t rows_shared_floats(const ProductArgs &p, int type, int cu_count, int64_t *tiles) {
  const SharedShape f = shared_shape(p, type, cu_count);
  *tiles = f.split > 1 ? f.tiles : 0;
  return *tiles * f.split * f.waves * f.mt * 256;
}

// Where w is large enough to be worth x's way through LDS. int8: from 8 rows on with 32 Mi
// elements of w (8192^2: 4 rows 16.5 us here and 16.1 there, 8 rows 16.4 and 16.6, 24 rows
// 17.9 and 22.0), from 32 rows on with 16 Mi (4096^2: 24 rows 9.4 and 8.8, 48 rows 10.9 and
// 11.4). Smaller w runs in the few-row kernel at every m (2048^2, 64 rows: 9.6 and 7.5).
// The cross entropy's bf16, with rows of 1024 (100000 x 512, 8 rows: 37 and 30): from 2 rows on
// with 64 Mi elements (131072 x 2048: 1 row 100 and 99, 3 rows 101 and 105; 32768 x 4096, 4 rows:
// 52.3 and 57.3), from 8 on with 32 Mi; from 17 on with 16 Mi (4096^2, 24 rows: 16.0 and 18.1)
// up to where the tiles are as fast, whose x is read less often (24 rows: 8192 x 4096 20.8 here
// and 28.8 as tiles, 16384 x 8192 58.6 and 73, 32768 x 4096 57 and 52, 50264 x 2056, 32 rows: 79
// and 42).
bool rows_shared_preferred(const ProductArgs &p, int type, int cu_count) {
  const int64_t size = (int64_t)p.n * p.k, mi = (int64_t)1 << 20;
  if (p.m > kRowsMost || size < 16 * mi || shared_shape(p, type, cu_count).split > 16) return false;
  if (type == kTypeI8) return p.m >= (size < 32 * mi ? 32 : 8);
  if (p.k < 1024) return false;
  if (p.m <= 16) return size >= 64 * mi ? p.m >= 2 : p.m >= 8 && size >= 32 * mi;
  return p.n <= 32768 && (size < 128 * mi || p.n <= 16384);
}

static RowsArgs rows_args(const ProductArgs &p, float *partial, uint32_t *arrivals) {
  RowsArgs a;
  a.x = p.a;
  a.w = p.b;
  a.ldx = (int32_t)p.lda;
  a.ldw = (int32_t)p.ldb;
  a.m = p.m;
  a.n = p.n;
  a.k = p.k;
  a.partial = partial;
  a.arrivals = arrivals;
  a.ep = p.ep;
  return a;
}

hipError_t launch_rows_shared(const ProductArgs &p, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s) {
  const SharedShape f = shared_shape(p, kTypeI8, cu_count);
  const RowsArgs a = rows_args(p, partial, arrivals);
  const dim3 grid((uint32_t)f.tiles, (uint32_t)f.split), block(64 * f.waves);
  if (f.mt == 1 && f.waves == 4) hipLaunchKernelGGL((ptg_rows_shared_i8_kernel<1, 4, 4>), grid, block, 0, s, a);
  else if (f.mt == 1) hipLaunchKernelGGL((ptg_rows_shared_i8_kernel<1, 8, 2>), grid, block, 0, s, a);
  else if (f.mt == 2 && f.waves == 4) hipLaunchKernelGGL((ptg_rows_shared_i8_kernel<2, 4, 4>), grid, block, 0, s, a);
  else if (f.mt == 2) hipLaunchKernelGGL((ptg_rows_shared_i8_kernel<2, 8, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((ptg_rows_shared_i8_kernel<4, 8, 2>), grid, block, 0, s, a);
  return hipGetLastError();
}

int32_t rows_shared_loss_block(const ProductArgs &p, int cu_count) { return 16 * shared_shape(p, kTypeBf16, cu_count).waves; }

hipError_t launch_rows_shared_loss(const ProductArgs &p, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s) {
  const SharedShape f = shared_shape(p, kTypeBf16, cu_count);
  const RowsArgs a = rows_args(p, partial, arrivals);
  const dim3 grid((uint32_t)f.tiles, (uint32_t)f.split), block(64 * f.waves);
  if (f.mt == 1 && f.waves == 4) hipLaunchKernelGGL((ptg_rows_shared_loss_kernel<1, 4, 4>), grid, block, 0, s, a, p.loss);
  else if (f.mt == 1) hipLaunchKernelGGL((ptg_rows_shared_loss_kernel<1, 8, 2>), grid, block, 0, s, a, p.loss);
  else if (f.mt == 2 && f.waves == 4) hipLaunchKernelGGL((ptg_rows_shared_loss_kernel<2, 4, 4>), grid, block, 0, s, a, p.loss);
  else if (f.mt == 2) hipLaunchKernelGGL((ptg_rows_shared_loss_kernel<2, 8, 2>), grid, block, 0, s, a, p.loss);
  else hipLaunchKernelGGL((ptg_rows_shared_loss_kernel<4, 8, 2>), grid, block, 0, s, a, p.loss);
  return hipGetLastError();
}

}  // namespace ptg
