// RMS norm with the residual's addition, its gradient, and the column sums that
// finish a gradient's partial sums.
//
// A row lives in the registers of one row group: T threads (a wave for n up to
// 1024, 256 threads up to 4096, 1024 beyond) hold NCH chunks of eight
// consecutive elements each, so x and residual are read once and everything
// after the row's sums works on registers. Groups stride over the rows and ask for
// the next row before the present one's sums are known. Two chunks a thread
// rather than four: 16384 x 8192 to e4m3, 174 us with 256 threads and four
// chunks, 163 with 1024 and one (164.5 with the codes' exact quotient: 5.7 TB/s; a
// large copy reaches 4.7, a read 5.8).
#include "layer_device.hpp"

namespace ptg {

// Row-group size and chunks per thread for rows of n elements.
struct NormShape { int threads, chunks; };
static NormShape norm_shape(int32_t n) {
  const int c = (n + 7) / 8;
  const int t = c <= 2 * 64 ? 64 : c <= 2 * 256 ? 256 : 1024;
  const int per = (c + t - 1) / t;
  return {t, per <= 1 ? 1 : per <= 2 ? 2 : 4};
}

// Forward. The largest |y| of an e4m3 or int8 row is r max |s weight|, so the sum of
// squares and that maximum come from one reduction. |s weight| is compared as
// bit patterns: they order like the values, and a NaN's are the largest, so a
// NaN reaches the scale instead of being skipped.
template <int T, int NCH, typename TS, typename TO>
__device__ __forceinline__ void rmsnorm_rows(const NormArgs &a, int32_t groups) {
  constexpr int kGroups = T < 256 ? 256 / T : 1;
  constexpr bool E8 = std::is_same<TO, e4m3_t>::value || std::is_same<TO, i8_t>::value;  // codes with a scale a row
  __shared__ float lds_sum[2][16];
  __shared__ uint32_t lds_top[2][16];
  const int32_t t = (int32_t)threadIdx.x % T;
  const int32_t group = (int32_t)blockIdx.x * kGroups + (int32_t)threadIdx.x / T;
  typedef typename Raw8<TS>::type raw;
  struct Row { raw x[NCH], r[NCH]; };
  auto ask = [&](Row &f, int64_t row) {
    const TS *x = (const TS *)a.x + row * a.ldx, *res = (const TS *)a.residual + row * a.ldr;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      f.x[c] = {};
      f.r[c] = {};
      if (j < a.n) {
        f.x[c] = *(const raw *)(x + j);
        if (a.residual) f.r[c] = *(const raw *)(res + j);
      }
    }
  };
  // a workgroup of 1024 threads has 128 registers a thread: with four chunks the next row does not fit
  constexpr bool kAhead = T < 1024 || NCH * (16 + (int)sizeof(TS) * 4) <= 72;
  Row next;
  if (kAhead && group < a.m) ask(next, group);
  f32x8 w[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int32_t j = (c * T + t) * 8;
    w[c] = f32x8{1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (j < a.n && a.weight) w[c] = load8_as(a.weight, a.weight_type, j);
  }
  int buf = 0;
  for (int64_t row = group; row < a.m; row += groups, buf ^= 1) {
    f32x8 v[NCH];
    float sum = 0.0f;
    uint32_t top = 0;
    if constexpr (!kAhead) ask(next, row);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      v[c] = widen(next.x[c]) + widen(next.r[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += v[c][e] * v[c][e];
        if (E8) top = max(top, __float_as_uint(v[c][e] * w[c][e]) & 0x7fffffffu);
      }
    }
    if (kAhead && row + groups < a.m) ask(next, row + groups);
    if (a.sum_out) {
      TS *so = (TS *)a.sum_out + row * a.lds;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int32_t j = (c * T + t) * 8;
        if (j < a.n) store8_nt(so + j, v[c]);
      }
    }
    sum = wave_sum(sum);
    if (E8) top = wave_umax(top);
    if constexpr (T > 64) {
      const uint32_t wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63u) == 0) {
        lds_sum[buf][wave] = sum;
        lds_top[buf][wave] = top;
      }
      // two buffers: a row's reads are over before the row after next writes. (The
      // barrier alone: the next row's loads stay under way.)
      wait_lds_all();
      wg_barrier();
      sum = 0.0f;
      top = 0;
#pragma unroll
      for (int q = 0; q < T / 64; ++q) {
        sum += lds_sum[buf][q];
        top = max(top, lds_top[buf][q]);
      }
    }
    const float r = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    float lift = 1.0f, lifted = 1.0f, inv_lifted = 1.0f;
    bool bad = false;
    if constexpr (E8) {
      // the floor keeps 1 / scale finite (r / scale need not be: y is formed first)
      const float amax = __uint_as_float(top) * r;
      float scale = amax == 0.0f ? 1.0f : fmaxf(amax / kTop<TO>, 0x1p-126f);
      bad = !(amax < INFINITY);
      if (bad) scale = __uint_as_float(0x7fc00000u);  // NaN or infinity in y
      if (t == 0) a.scale[row] = scale;
      if (scale < 0x1p-60f) lift = 0x1p64f;  // the quotient's remainder stays above the subnormal numbers
      lifted = scale * lift;
      inv_lifted = 1.0f / lifted;
    }
    TO *out = (TO *)a.out + row * a.ldo;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      if (j < a.n) {
        f32x8 y = v[c] * w[c] * r;
        if constexpr (E8) {
          // y / scale: the product with the reciprocal, put right by its remainder (the
          // product alone is off by a step of fp32 now and then, and a code next to a
          // tie then by a step of e4m3: 1 in 10^6. 16384 x 8192: 163.3 -> 164.5 us).
          y *= lift;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float q = y[e] * inv_lifted;
            y[e] = fmaf(fmaf(-q, lifted, y[e]), inv_lifted, q);
          }
        }
        if constexpr (E8) store_codes(out + j, y, bad);
        else store8_nt(out + j, y);
      }
    }
  }
}
template <int T, int NCH, typename TS, typename TO>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_rmsnorm_kernel(const NormArgs a, int32_t groups) {
  rmsnorm_rows<T, NCH, TS, TO>(a, groups);
}
template <int T, int NCH, typename TS>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_norm_i8_kernel(const NormArgs a, int32_t groups) {
  rmsnorm_rows<T, NCH, TS, i8_t>(a, groups);
}

// Gradient. Row groups stride over the rows; a thread's columns are the same
// for every row, so its share of dweight stays in registers and leaves once,
// as one partial row per group (8192 x 8192 with dsum: 97 us, 5.5 TB/s, and 5 of
// column sums). The next row's three operands are asked for
// before a row's sums are known, as loaded (bf16 rows hold half the registers).
template <int T, int NCH, typename TS, typename TD>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_rmsnorm_backward_kernel(const NormGradArgs a, int32_t groups) {
  constexpr int kGroups = T < 256 ? 256 / T : 1;
  __shared__ float lds[2][2][16];
  const int32_t t = (int32_t)threadIdx.x % T;
  const int32_t group = (int32_t)blockIdx.x * kGroups + (int32_t)threadIdx.x / T;
  // First column of the thread's chunk c. With four chunks it is worked out where it
  // is used: kept, with the addresses that follow from it, it would not fit.
  auto at = [&](int c) -> int32_t {
    int32_t mine = t;
    if constexpr (T == 1024 && NCH == 4) asm volatile("" : "+v"(mine)::"memory");
    return (c * T + mine) * 8;
  };
  f32x8 kept[NCH], dw[NCH];  // the thread's columns of weight and its share of dweight
  auto weight = [&](int c) -> f32x8 {
    const int32_t j = at(c);
    if (j < a.n && a.weight) return load8_as(a.weight, a.weight_type, j);
    return f32x8{1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
  };
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    dw[c] = f32x8{};
    kept[c] = weight(c);
  }
  struct Row { typename Raw8<TS>::type s[NCH], u[NCH]; typename Raw8<TD>::type d[NCH]; };
  const bool has_u = a.dx && a.dsum;
  auto ask = [&](Row &f, int64_t row) {
    const TS *sp = (const TS *)a.s + row * a.lds, *up = (const TS *)a.dsum + row * a.lddsum;
    const TD *dp = (const TD *)a.dy + row * a.lddy;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      f.s[c] = {};
      f.d[c] = {};
      f.u[c] = {};
      if (j < a.n) {
        f.s[c] = *(const typename Raw8<TS>::type *)(sp + j);
        f.d[c] = *(const typename Raw8<TD>::type *)(dp + j);
        if (has_u) f.u[c] = *(const typename Raw8<TS>::type *)(up + j);
      }
    }
  };
  const float inv_n = 1.0f / (float)a.n;
  // registers: 16 a chunk for weight and dweight, kRaw for a row as loaded. A
  // workgroup of 1024 threads has 128 a thread: long rows are held without the
  // next one, or not at all, nor the weight (the second look comes from the caches:
  // 1000 x 32768, 95 us, 2.7 TB/s of what has to be moved).
  constexpr int kRaw = NCH * (4 * (int)sizeof(TS) + 2 * (int)sizeof(TD));
  constexpr bool kAhead = T < 1024 || NCH * 16 + 2 * kRaw <= 72, kHold = T < 1024 || NCH * 16 + kRaw <= 64;
  int buf = 0;
  Row next;
  if (kAhead && group < a.m) ask(next, group);
  for (int64_t row = group; row < a.m; row += groups, buf ^= 1) {
    if constexpr (kHold && !kAhead) ask(next, row);
    const Row f = next;
    const TS *sp = (const TS *)a.s + row * a.lds, *up = (const TS *)a.dsum + row * a.lddsum;
    const TD *dp = (const TD *)a.dy + row * a.lddy;
    float ss = 0.0f, gs = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      f32x8 s = {}, d = {};
      if constexpr (kHold) {
        s = widen(f.s[c]);
        d = widen(f.d[c]);
      } else {
        const int32_t j = at(c);
        if (j < a.n) {
          s = load8(sp + j);
          d = load8(dp + j);
        }
      }
      const f32x8 w = kHold ? kept[c] : weight(c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += s[e] * s[e];
        gs += d[e] * w[e] * s[e];
      }
      if constexpr (!kHold) asm volatile("" : "+v"(ss), "+v"(gs));  // before the next chunk is asked for
    }
    if (kAhead && row + groups < a.m) ask(next, row + groups);
    ss = wave_sum(ss);
    gs = wave_sum(gs);
    if constexpr (T > 64) {
      const uint32_t wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63u) == 0) {
        lds[buf][0][wave] = ss;
        lds[buf][1][wave] = gs;
      }
      // two buffers: a row's reads are over before the row after next writes. (The barrier alone: the next row's
      // loads stay under way.)
      wait_lds_all();
      wg_barrier();
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
      const int32_t j = at(c);
      f32x8 s = {}, d = {};
      const f32x8 w = kHold ? kept[c] : weight(c);
      if constexpr (kHold) {
        s = widen(f.s[c]);
        d = widen(f.d[c]);
      } else if (j < a.n) {
        s = load8(sp + j);
        d = load8(dp + j);
      }
      if (a.dx && j < a.n) {
        f32x8 dx = d * w * r - s * k;
        if (has_u) dx += kHold ? widen(f.u[c]) : load8(up + j);
        store8((TS *)a.dx + row * a.lddx + j, dx);
      }
      dw[c] += d * (s * r);
      if constexpr (!kHold) asm volatile("" : "+v"(dw[c]));
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

// 32 columns a workgroup: 8 threads of four columns, 64 interleaved sets of rows
// whose loads are independent (at the few hundred rows there are, latency counts:
// 512 x 2056 took 11.8 us with 16 sets in a dependent loop). Sets are added in order.
__global__ __launch_bounds__(512) void ptg_column_sum_kernel(const float *partial, int32_t rows, int32_t n, float *out,
                                                             int32_t accumulate) {
  __shared__ f32x4 lds[64][8];
  const int32_t cx = (int32_t)threadIdx.x & 7, ry = (int32_t)threadIdx.x >> 3;
  const int32_t j = ((int32_t)blockIdx.x * 8 + cx) * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j < n) {
    for (int32_t r = ry; r < rows; r += 64 * 8) {
      f32x4 p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        p[u] = r + 64 * u < rows ? *(const f32x4 *)(partial + (int64_t)(r + 64 * u) * n + j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 8; ++u) v += p[u];
    }
  }
  lds[ry][cx] = v;
  __syncthreads();
  if (ry < 8) {  // eight sets each, then those eight sums
    v = lds[ry * 8][cx];
#pragma unroll
    for (int q = 1; q < 8; ++q) v += lds[ry * 8 + q][cx];
  }
  __syncthreads();
  if (ry < 8) lds[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && j < n) {
    v = accumulate ? *(const f32x4 *)(out + j) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 8; ++q) v += lds[q][cx];
    *(f32x4 *)(out + j) = v;
  }
}

template <int T, int NCH, typename TS>
static void rmsnorm_out(const NormArgs &a, int groups, hipStream_t s) {
  const int per = T < 256 ? 256 / T : 1;
  const dim3 grid((uint32_t)((groups + per - 1) / per)), block(T < 256 ? 256 : T);
  if (a.out_type == kTypeF32) hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, float>), grid, block, 0, s, a, groups);
  else if (a.out_type == kTypeBf16) hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, __bf16>), grid, block, 0, s, a, groups);
  else if (a.out_type == kTypeI8) hipLaunchKernelGGL((ptg_norm_i8_kernel<T, NCH, TS>), grid, block, 0, s, a, groups);
  else hipLaunchKernelGGL((ptg_rmsnorm_kernel<T, NCH, TS, e4m3_t>), grid, block, 0, s, a, groups);
}

template <int T, typename TS>
static void rmsnorm_chunks(const NormArgs &a, int chunks, int groups, hipStream_t s) {
  if (chunks == 1) rmsnorm_out<T, 1, TS>(a, groups, s);
  else if (chunks == 2) rmsnorm_out<T, 2, TS>(a, groups, s);
  else if constexpr (T == 1024) rmsnorm_out<T, 4, TS>(a, groups, s);  // the others change to more threads first
}

template <typename TS>
static void rmsnorm_type(const NormArgs &a, int groups, hipStream_t s) {
  const NormShape f = norm_shape(a.n);
  if (f.threads == 64) rmsnorm_chunks<64, TS>(a, f.chunks, groups, s);
  else if (f.threads == 256) rmsnorm_chunks<256, TS>(a, f.chunks, groups, s);
  else rmsnorm_chunks<1024, TS>(a, f.chunks, groups, s);
}

hipError_t launch_rmsnorm(const NormArgs &a, int cu_count, hipStream_t s) {
  const NormShape f = norm_shape(a.n);
  const int64_t most = (int64_t)cu_count * 1024 / f.threads;  // 1024 threads a CU (twice or four times as many: the same time)
  const int groups = (int)(a.m < most ? a.m : most);
  if (a.type == kTypeF32) rmsnorm_type<float>(a, groups, s);
  else rmsnorm_type<__bf16>(a, groups, s);
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
  else if constexpr (T == 1024) backward_dy<T, 4, TS>(a, groups, s);  // the others change to more threads first
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
  hipLaunchKernelGGL(ptg_column_sum_kernel, dim3((uint32_t)((n + 31) / 32)), dim3(512), 0, s, partial, rows, n, out, accumulate);
  return hipGetLastError();
}

}  // namespace ptg
