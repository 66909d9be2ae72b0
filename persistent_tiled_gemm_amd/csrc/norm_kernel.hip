// RMS norm with the residual's addition, its gradient, and the column sums that
// finish a gradient's partial sums.
//
// A row lives in the registers of one row group: T threads (a wave for n up to
// 2048, 256 threads up to 8192, 1024 beyond) hold NCH chunks of eight
// consecutive elements each, so x and residual are read once and everything
// after the row's sums works on registers.
#include "layer_device.hpp"

namespace ptg {

// Row-group size and chunks per thread for rows of n elements.
struct NormShape { int threads, chunks; };
static NormShape norm_shape(int32_t n) {
  const int c = (n + 7) / 8;
  const int t = c <= 4 * 64 ? 64 : c <= 4 * 256 ? 256 : 1024;
  const int per = (c + t - 1) / t;
  return {t, per <= 1 ? 1 : per <= 2 ? 2 : 4};
}

// Sum and maximum of a pair over the row group, in every thread.
template <int T>
__device__ __forceinline__ void group_reduce(float &sum, uint32_t &top, float *lds_sum, uint32_t *lds_top) {
  sum = wave_sum(sum);
  top = wave_umax(top);
  if constexpr (T > 64) {
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63u) == 0) {
      lds_sum[wave] = sum;
      lds_top[wave] = top;
    }
    __syncthreads();
    sum = 0.0f;
    top = 0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) {
      sum += lds_sum[w];
      top = max(top, lds_top[w]);
    }
  }
}

// Forward. The largest |y| of an e4m3 row is r max |s weight|, so the sum of
// squares and that maximum come from one reduction. |s weight| is compared as
// bit patterns: they order like the values, and a NaN's are the largest, so a
// NaN reaches the scale instead of being skipped.
template <int T, int NCH, typename TS, typename TO>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_rmsnorm_kernel(const NormArgs a) {
  constexpr int kGroups = T < 256 ? 256 / T : 1;
  __shared__ float lds_sum[16];
  __shared__ uint32_t lds_top[16];
  const int32_t t = (int32_t)threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * kGroups + (int32_t)threadIdx.x / T;
  if (T < 256 && row >= a.m) return;  // whole waves leave; larger groups have one row a workgroup
  const TS *x = (const TS *)a.x + row * a.ldx;
  const TS *res = a.residual ? (const TS *)a.residual + row * a.ldr : nullptr;
  f32x8 v[NCH], w[NCH];
  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int32_t j = (c * T + t) * 8;
    v[c] = f32x8{};
    w[c] = f32x8{1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (j < a.n) {
      v[c] = load8(x + j);
      if (res) v[c] += load8(res + j);
      if (a.weight) w[c] = load8_as(a.weight, a.weight_type, j);
    }
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum += v[c][e] * v[c][e];
      const float p = v[c][e] * w[c][e];
      top = max(top, __float_as_uint(p) & 0x7fffffffu);
      w[c][e] = p;
    }
  if (a.sum_out) {
    TS *so = (TS *)a.sum_out + row * a.lds;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      if (j < a.n) store8(so + j, v[c]);
    }
  }
  group_reduce<T>(sum, top, lds_sum, lds_top);
  const float r = 1.0f / sqrtf(sum / (float)a.n + a.eps);
  float inv_scale = 1.0f;
  if constexpr (std::is_same<TO, e4m3_t>::value) {
    // the floor keeps 1 / scale finite (r / scale need not be: y is formed first)
    const float amax = __uint_as_float(top) * r;
    float scale = amax == 0.0f ? 1.0f : fmaxf(amax / kE4m3Max, 0x1p-126f);
    if (!(amax < INFINITY)) scale = __uint_as_float(0x7fc00000u);  // NaN or infinity in y
    if (t == 0) a.scale[row] = scale;
    inv_scale = 1.0f / scale;
  }
  TO *out = (TO *)a.out + row * a.ldo;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int32_t j = (c * T + t) * 8;
    if (j < a.n) {
      f32x8 y = w[c] * r;
      if constexpr (std::is_same<TO, e4m3_t>::value) y *= inv_scale;
      store8(out + j, y);
    }
  }
}

// Gradient. Row groups stride over the rows; a thread's columns are the same
// for every row, so its share of dweight stays in registers and leaves once,
// as one partial row per group.
template <int T, int NCH, typename TS, typename TD>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_rmsnorm_backward_kernel(const NormGradArgs a, int32_t groups) {
  constexpr int kGroups = T < 256 ? 256 / T : 1;
  __shared__ float lds[2][2][16];
  const int32_t t = (int32_t)threadIdx.x % T;
  const int32_t group = (int32_t)blockIdx.x * kGroups + (int32_t)threadIdx.x / T;
  f32x8 w[NCH], dw[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int32_t j = (c * T + t) * 8;
    dw[c] = f32x8{};
    w[c] = f32x8{1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (j < a.n && a.weight) w[c] = load8_as(a.weight, a.weight_type, j);
  }
  const float inv_n = 1.0f / (float)a.n;
  int buf = 0;
  for (int64_t row = group; row < a.m; row += groups, buf ^= 1) {
    const TS *sp = (const TS *)a.s + row * a.lds;
    const TD *dp = (const TD *)a.dy + row * a.lddy;
    f32x8 s[NCH], d[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      s[c] = f32x8{};
      d[c] = f32x8{};
      if (j < a.n) {
        s[c] = load8(sp + j);
        d[c] = load8(dp + j);
      }
    }
    float ss = 0.0f, gs = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += s[c][e] * s[c][e];
        gs += d[c][e] * w[c][e] * s[c][e];
      }
    ss = wave_sum(ss);
    gs = wave_sum(gs);
    if constexpr (T > 64) {
      const uint32_t wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63u) == 0) {
        lds[buf][0][wave] = ss;
        lds[buf][1][wave] = gs;
      }
      __syncthreads();  // two buffers: a row's reads are over before the row after next writes
      ss = 0.0f;
      gs = 0.0f;
#pragma unroll
      for (int q = 0; q < T / 64; ++q) {
        ss += lds[buf][0][q];
        gs += lds[buf][1][q];
      }
    }
    const float r = 1.0f / sqrtf(ss * inv_n + a.eps);
    const float k = r * r * (gs * inv_n) * r;  // r h_j mean(g h) = s_j k
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      if (j < a.n) {
        if (a.dx) {
          f32x8 dx = d[c] * w[c] * r - s[c] * k;
          if (a.dsum) dx += load8((const TS *)a.dsum + row * a.lddsum + j);
          store8((TS *)a.dx + row * a.lddx + j, dx);
        }
        dw[c] += d[c] * (s[c] * r);
      }
    }
  }
  if (a.partial) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      if (j < a.n && group < groups) store8(a.partial + (int64_t)group * a.n + j, dw[c]);
    }
  }
}

// 64 columns a workgroup: 16 threads of four columns, 16 interleaved sets of rows.
__global__ __launch_bounds__(256) void ptg_column_sum_kernel(const float *partial, int32_t rows, int32_t n, float *out,
                                                             int32_t accumulate) {
  __shared__ f32x4 lds[16][16];
  const int32_t cx = (int32_t)threadIdx.x & 15, ry = (int32_t)threadIdx.x >> 4;
  const int32_t j = ((int32_t)blockIdx.x * 16 + cx) * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j < n)
    for (int32_t r = ry; r < rows; r += 16) v += *(const f32x4 *)(partial + (int64_t)r * n + j);
  lds[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && j < n) {
    v = accumulate ? *(const f32x4 *)(out + j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 16; ++q) v += lds[q][cx];
    *(f32x4 *)(out + j) = v;
  }
}

template <int T, int NCH, typename TS>
static void rmsnorm_out(const NormArgs &a, hipStream_t s) {
  const int per = T < 256 ? 256 / T : 1;
  const dim3 grid((uint32_t)(((int64_t)a.m + per - 1) / per)), block(T < 256 ? 256 : T);
  if (a.out_type == kTypeF32) hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, float>), grid, block, 0, s, a);
  else if (a.out_type == kTypeBf16) hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, __bf16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, e4m3_t>), grid, block, 0, s, a);
}

template <int T, typename TS>
static void rmsnorm_chunks(const NormArgs &a, int chunks, hipStream_t s) {
  if (chunks == 1) rmsnorm_out<T, 1, TS>(a, s);
  else if (chunks == 2) rmsnorm_out<T, 2, TS>(a, s);
  else rmsnorm_out<T, 4, TS>(a, s);
}

template <typename TS>
static void rmsnorm_type(const NormArgs &a, hipStream_t s) {
  const NormShape f = norm_shape(a.n);
  if (f.threads == 64) rmsnorm_chunks<64, TS>(a, f.chunks, s);
  else if (f.threads == 256) rmsnorm_chunks<256, TS>(a, f.chunks, s);
  else rmsnorm_chunks<1024, TS>(a, f.chunks, s);
}

hipError_t launch_rmsnorm(const NormArgs &a, int, hipStream_t s) {
  if (a.type == kTypeF32) rmsnorm_type<float>(a, s);
  else rmsnorm_type<__bf16>(a, s);
  return hipGetLastError();
}

int rmsnorm_partial_rows(int32_t m, int32_t n, int cu_count) {
  const NormShape f = norm_shape(n);
  const int64_t most = (int64_t)cu_count * (f.threads == 1024 ? 1 : 2) * (f.threads < 256 ? 256 / f.threads : 1);
  return (int)(m < most ? m : most);
}

template <int T, int NCH, typename TS>
static void backward_dy(const NormGradArgs &a, int groups, hipStream_t s) {
  const int per = T < 256 ? 256 / T : 1;
  const dim3 grid((uint32_t)((groups + per - 1) / per)), block(T < 256 ? 256 : T);
  if (a.dy_type == kTypeF32) hipLaunchKernelGGL((ptg_rmsnorm_backward_kernel<T, NCH, TS, float>), grid, block, 0, s, a, groups);
  else hipLaunchKernelGGL((ptg_rmsnorm_backward_kernel<T, NCH, TS, __bf16>), grid, block, 0, s, a, groups);
}

template <int T, typename TS>
static void backward_chunks(const NormGradArgs &a, int chunks, int groups, hipStream_t s) {
  if (chunks == 1) backward_dy<T, 1, TS>(a, groups, s);
  else if (chunks == 2) backward_dy<T, 2, TS>(a, groups, s);
  else backward_dy<T, 4, TS>(a, groups, s);
}

template <typename TS>
static void backward_type(const NormGradArgs &a, int groups, hipStream_t s) {
  const NormShape f = norm_shape(a.n);
  if (f.threads == 64) backward_chunks<64, TS>(a, f.chunks, groups, s);
  else if (f.threads == 256) backward_chunks<256, TS>(a, f.chunks, groups, s);
  else backward_chunks<1024, TS>(a, f.chunks, groups, s);
}

hipError_t launch_rmsnorm_backward(const NormGradArgs &a, int cu_count, hipStream_t s) {
  const int groups = rmsnorm_partial_rows(a.m, a.n, cu_count);
  if (a.type == kTypeF32) backward_type<float>(a, groups, s);
  else backward_type<__bf16>(a, groups, s);
  return hipGetLastError();
}

hipError_t launch_column_sum(const float *partial, int rows, int32_t n, float *out, int accumulate, hipStream_t s) {
  hipLaunchKernelGGL(ptg_column_sum_kernel, dim3((uint32_t)((n + 63) / 64)), dim3(256), 0, s, partial, rows, n, out, accumulate);
  return hipGetLastError();
}

}  // namespace ptg
