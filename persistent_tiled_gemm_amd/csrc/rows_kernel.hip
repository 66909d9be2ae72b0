// The product of the layer operators for few rows (a decode step): out = act(x .
// w^T scales + bias) + residual with m up to 64.
//
// Every weight is used for at most 64 rows, so the kernel is bound by reading w
// once; everything is laid out for bytes in flight. A workgroup owns 16 NBLK rows
// of w and, of k, the share S-th of the grid gives it; its waves split that share
// again, so a wave streams 16 NBLK x (k / S / waves) of w straight from memory
// into MFMA operands (v_mfma_f32_16x16x32_bf16: 16 rows of w against 16 rows of
// x), with no LDS on the way. Batches of U steps are double-buffered in
// registers: the next batch's loads are under way while one is multiplied. x
// (whose rows the caches hold) is read beside w the same way. The waves' sums
// meet in LDS, the workgroups' (S > 1) in the plan's workspace: the last one to
// arrive adds the S parts in order and finishes the tile. 8192^2: one row in bf16
// 26.8 us (5.0 TB/s of w, and some 4 us of launch, first loads and join in it), 24
// rows in e4m3 21.6 (3.1 TB/s).
#include <algorithm>

#include "layer_device.hpp"

namespace ptg {

// Two bf16 from two of four e4m3 values (exact).
__device__ __forceinline__ uint32_t widen_pair(uint32_t four, bool high) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const bf16x2 v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)four, 1.0f, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)four, 1.0f, false);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const i32x4 v = {(int)widen_pair(lo, false), (int)widen_pair(lo, true), (int)widen_pair(hi, false), (int)widen_pair(hi, true)};
  return __builtin_bit_cast(bf16x8, v);
}

static constexpr int kPolicyStream = 2;  // nt: w is read once

template <bool E8, int MT, int NBLK, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void ptg_rows_kernel(const RowsArgs a) {
  constexpr int kItems = MT * NBLK;  // 16 x 16 blocks of the workgroup's tile
  constexpr int kStep = E8 ? 64 : 32;
  constexpr uint32_t kSize = E8 ? 1u : 2u;
  __shared__ f32x4 sums[WAVES][kItems][64];
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = wave_uniform(tid >> 6);
  const uint32_t tile = blockIdx.x, part = blockIdx.y;
  const int32_t n0 = (int32_t)tile * (16 * NBLK);
  const int32_t row = (int32_t)(lane & 15u), group = (int32_t)(lane >> 4);

  // this wave's steps [s0, s1), from an even one on: a batch's steps come in pairs
  // that share the rows' 128-byte lines (split between two batches, a line's halves
  // were fetched from memory twice at times: 151 MB instead of 139 for 8192^2, one
  // row, 27.9 -> 26.8 us)
  const uint32_t parts = gridDim.y * (uint32_t)WAVES, mine = part * (uint32_t)WAVES + wave;
  const uint32_t steps = ((uint32_t)a.k + kStep - 1) / kStep;
  const uint32_t lines = (steps + 1) / 2;
  const int32_t s0 = 2 * (int32_t)((uint64_t)lines * mine / parts);
  const int32_t s1 = min((int32_t)steps, 2 * (int32_t)((uint64_t)lines * (mine + 1) / parts));

  // Each wave starts part-way into its range and wraps around (a phase from its
  // place in the grid; the order of a sum depends on that alone). Started at
  // their first steps, waves whose ranges lie a multiple of 4 KiB apart read the
  // same few memory channels at a time: 4096 x 16384, one row, 39.7 us
  // against 27.4.
  const int32_t count = s1 - s0;
  const int32_t rot = count > 1 ? (int32_t)((((tile * 8u + wave) * 2654435761u) >> 16) % (uint32_t)count & ~1u) : 0;

  const __amdgpu_buffer_rsrc_t wr = make_rsrc((const unsigned char *)a.w + (size_t)n0 * (size_t)a.ldw * kSize);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x);
  uint32_t w_row[NBLK], x_row[MT];  // byte offsets of the lane's rows; past the matrix: out of range, read as zeros
#pragma unroll
  for (int b = 0; b < NBLK; ++b) w_row[b] = n0 + 16 * b + row < a.n ? (uint32_t)(16 * b + row) * (uint32_t)a.ldw * kSize : kBufOob;
#pragma unroll
  for (int t = 0; t < MT; ++t) x_row[t] = 16 * t + row < a.m ? (uint32_t)(16 * t + row) * (uint32_t)a.ldx * kSize : kBufOob;

  f32x4 acc[MT][NBLK] = {};
  struct Batch { i32x4 w[U][NBLK], x[U][MT]; };
  auto load = [&](Batch &f, int32_t s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // 16 bytes a lane: chunk `group` of the step's 64
      const int32_t i = s + u + rot;
      const uint32_t at = (uint32_t)(i < s1 ? i : i - count) * 64u + 16u * (uint32_t)group;
      const bool in = s + u < s1 && at < (uint32_t)a.k * kSize;
#pragma unroll
      for (int b = 0; b < NBLK; ++b)
        f.w[u][b] = __builtin_amdgcn_raw_buffer_load_b128(wr, in && w_row[b] != kBufOob ? (int)(w_row[b] + at) : (int)kBufOob, 0, kPolicyStream);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        f.x[u][t] = __builtin_amdgcn_raw_buffer_load_b128(xr, in && x_row[t] != kBufOob ? (int)(x_row[t] + at) : (int)kBufOob, 0, 0);
    }
  };
  auto multiply = [&](const Batch &f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < (E8 ? 2 : 1); ++h) {
        bf16x8 wf[NBLK], xf[MT];
#pragma unroll
        for (int b = 0; b < NBLK; ++b)
          wf[b] = E8 ? widen8((uint32_t)f.w[u][b][2 * h], (uint32_t)f.w[u][b][2 * h + 1]) : __builtin_bit_cast(bf16x8, f.w[u][b]);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          xf[t] = E8 ? widen8((uint32_t)f.x[u][t][2 * h], (uint32_t)f.x[u][t][2 * h + 1]) : __builtin_bit_cast(bf16x8, f.x[u][t]);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int b = 0; b < NBLK; ++b) acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[b], xf[t], acc[t][b], 0, 0, 0);
      }
    }
  };
  if (s0 < s1) {
    Batch f0, f1;
    load(f0, s0);
    for (int32_t s = s0; s < s1; s += 2 * U) {
      if (s + U < s1) load(f1, s + U);
      multiply(f0);
      if (s + U >= s1) break;
      if (s + 2 * U < s1) load(f0, s + 2 * U);
      multiply(f1);
    }
  }

  // ---- the waves' sums, in wave order. Lane l of a block holds columns n = 4 (l / 16) + 0..3 of row m = l mod 16.
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int b = 0; b < NBLK; ++b) sums[wave][t * NBLK + b][lane] = acc[t][b];
  __syncthreads();
  const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.partial);
  const uint32_t slots = (uint32_t)(kItems * 64);
  for (uint32_t i = tid; i < slots; i += 64 * WAVES) {
    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) z += sums[w][i >> 6][i & 63u];
    if (gridDim.y > 1) store16_agent(pr, ((tile * gridDim.y + part) * slots + i) * 16u, z);
    else sums[0][i >> 6][i & 63u] = z;
  }
  if (gridDim.y > 1) {
    // as the GEMM's split tail: parts written through the XCD's cache, a relaxed
    // count, and the last workgroup of the tile adds the parts in order
    wait_vmem_all();
    __syncthreads();
    if (tid == 0) {
      const uint32_t before = __hip_atomic_fetch_add(&a.arrivals[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = before + 1u == gridDim.y ? 1u : 0u;
      if (last) __hip_atomic_store(&a.arrivals[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (wave_uniform(last) == 0) return;
  }
  // ---- epilogue: four columns of one row at a time
  const EpilogueArgs &e = a.ep;
  for (uint32_t i = tid; i < slots; i += 64 * WAVES) {
    const uint32_t item = i >> 6, l = i & 63u;
    const int64_t m = (int64_t)(16u * (item / NBLK) + (l & 15u));
    const int32_t n = n0 + (int32_t)(16u * (item % NBLK) + 4u * (l >> 4));
    if (m >= a.m || n >= a.n) continue;
    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    if (gridDim.y > 1) {
      for (uint32_t p = 0; p < gridDim.y; ++p) z += load16_agent(pr, ((tile * gridDim.y + p) * slots + i) * 16u);
    } else {
      z = sums[0][item][l];
    }
    if constexpr (E8) {
      if (e.row_scale) z *= e.row_scale[m];
      if (e.col_scale) z *= *(const f32x4 *)(e.col_scale + n);
    }
    if (e.bias) z += load4_as(e.bias, e.bias_type, n);
    if (e.pre) store4((__bf16 *)e.pre + m * e.ldp + n, z);
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] = act_f32(e.act, z[q]);
    if (e.residual) z += load4_as(e.residual, e.residual_type, m * e.ldr + n);
    if (e.out_type == kTypeF32) *(f32x4 *)((float *)e.out + m * e.ldo + n) = z;
    else store4((__bf16 *)e.out + m * e.ldo + n, z);
  }
}

// The shape of a call: 16-row blocks of x and w a workgroup takes, its waves, and
// the workgroups that share a tile's k. Measured over n, k = 512 .. 16384 and 1,
// 8, 16, 32 and 64 rows in both types:
//   - a workgroup a CU (two with one block of w), of four waves (eight while
//     there are fewer than 1024): more waves only shorten each one's run through
//     memory (16384 x 4096 e4m3, one row: eight 18.6 us, four 15.9);
//   - x is read again for every 16 NBLK rows of w, from L2, which shows from some
//     ten rows on (from the first in e4m3, where it is widened again too): two
//     blocks of w up to 16 rows, four for more, where w is large enough that the
//     tiles still fill the machine (8192^2 bf16, 16 rows: one block 36 us, two 33 to
//     35; e4m3, 8 rows: one 18.7, two 16.9). More than 16 rows of so large a w come
//     here in e4m3 alone, and 32 at most (rows_preferred). Smaller w: one block up
//     to 16 rows, two for more (4096^2, 32 rows: two 14.9, four 14.8; 2048^2: two
//     9.0, one 8.7);
//   - k is shared until there are as many workgroups as CUs, while a wave keeps
//     four steps (1024 x 8192, one row: 12.6 us unshared, 9.1 with four).
struct RowsShape { int mt, nblk, waves, split; };
static RowsShape rows_shape(int32_t m, int32_t n, int32_t k, bool e8, int cu_count) {
  RowsShape f;
  const bool large = (int64_t)n * k >= (int64_t)32 << 20;
  f.mt = m <= 16 ? 1 : m <= 32 ? 2 : 4;
  f.nblk = m <= 16 ? (large && (e8 || m > 8) ? 2 : 1) : (large && e8 ? 4 : 2);
  const int64_t tiles = (n + 16 * f.nblk - 1) / (16 * f.nblk);
  f.waves = f.nblk == 1 && tiles < 4 * cu_count ? 8 : 4;
  const int64_t steps = (k + (e8 ? 63 : 31)) / (e8 ? 64 : 32);
  f.split = (int)std::max<int64_t>(1, std::min<int64_t>({cu_count / tiles, steps / (4 * f.waves), 16}));
  return f;
}

// Few rows run here, except where the tiles are as fast: they read x once for 128
// rows of w, and reach 3.5 TB/s whatever m. From 17 rows on for w of 32 Mi
// elements (bf16, 8192^2: 16 rows 33 to 35 us here, 37 as tiles; 32 rows 40 and
// 38; 64 rows 51 and 40; 4096^2: 64 rows 20 and 22), from 33 in e4m3 (8192^2: 32
// rows 24 and 29, 64 rows 31 and 31), and from 5 where bf16 rows do not start on
// 64-byte lines (5000^2: one row 21.8 and 23.0, 8 rows 25.5 and 23.8, 64 44 and 29).
bool rows_preferred(const ProductArgs &p, bool e8) {
  if (p.m > kRowsMost) return false;
  const int64_t size = (int64_t)p.n * p.k;
  if (e8) return p.m <= 32 || size < (int64_t)32 << 20;
  if (p.m > 4 && p.ldb % 32 != 0 && size >= (int64_t)16 << 20) return false;
  return p.m <= 16 || size < (int64_t)32 << 20;
}

int64_t rows_partial_floats(const ProductArgs &p, bool e8, int cu_count, int64_t *tiles) {
  const RowsShape f = rows_shape(p.m, p.n, p.k, e8, cu_count);
  *tiles = f.split > 1 ? (p.n + 16 * f.nblk - 1) / (16 * f.nblk) : 0;
  return *tiles * f.split * f.mt * f.nblk * 256;
}

template <bool E8>
static hipError_t rows_blocks(const RowsShape &f, const RowsArgs &a, dim3 grid, hipStream_t s) {
  const dim3 block(64 * f.waves);
  if constexpr (E8) {
    if (f.mt == 2 && f.nblk == 4) {
      hipLaunchKernelGGL((ptg_rows_kernel<E8, 2, 4, 4, 2>), grid, block, 0, s, a);
      return hipGetLastError();
    }
  }
  if (f.mt == 1 && f.nblk == 1 && f.waves == 4) hipLaunchKernelGGL((ptg_rows_kernel<E8, 1, 1, 4, 4>), grid, block, 0, s, a);
  else if (f.mt == 1 && f.nblk == 1) hipLaunchKernelGGL((ptg_rows_kernel<E8, 1, 1, 8, 4>), grid, block, 0, s, a);
  else if (f.mt == 1) hipLaunchKernelGGL((ptg_rows_kernel<E8, 1, 2, 4, 4>), grid, block, 0, s, a);
  else if (f.mt == 2 && f.nblk == 2) hipLaunchKernelGGL((ptg_rows_kernel<E8, 2, 2, 4, 2>), grid, block, 0, s, a);
  else if (f.mt == 4 && f.nblk == 2) hipLaunchKernelGGL((ptg_rows_kernel<E8, 4, 2, 4, 2>), grid, block, 0, s, a);
  else return hipErrorInvalidValue;  // rows_preferred sends no such call here
  return hipGetLastError();
}

hipError_t launch_rows(const ProductArgs &p, bool e8, float *partial, uint32_t *arrivals, int cu_count, hipStream_t s) {
  const RowsShape f = rows_shape(p.m, p.n, p.k, e8, cu_count);
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
  const dim3 grid((uint32_t)((p.n + 16 * f.nblk - 1) / (16 * f.nblk)), (uint32_t)f.split);
  return e8 ? rows_blocks<true>(f, a, grid, s) : rows_blocks<false>(f, a, grid, s);
}

}  // namespace ptg
