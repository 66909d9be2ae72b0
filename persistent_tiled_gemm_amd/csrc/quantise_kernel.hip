// Rows to 8-bit codes with one scale each: scale = max |x| / top, code = x / scale rounded
// to nearest, ties to even (top 127 for int8, 448 for e4m3).
//
// Bound by memory: each element is read once and leaves as one byte (16384 x 8192 bf16: 77 us,
// 5.2 TB/s, as fast as a copy; 1111 x 10248 fp32: 11.7, 4.9 TB/s). A row lives in the
// registers of one row group, as in the norm: T threads hold NCH chunks of eight
// consecutive elements each; groups stride over the rows and ask for the next row
// before the present one's maximum is known. Rows over 32768 elements are read twice,
// the second time from the caches.
#include "layer_device.hpp"

namespace ptg {

// A row's scale and what its quotients are formed with. |x| is compared as bit patterns,
// which order like the values, a NaN's above all: a NaN or infinity gives the scale NaN.
// The quotient x / scale is the product with the reciprocal, put right by its remainder:
// correctly rounded, as a division is (the reciprocal is). Where the scale is small,
// both are lifted first, so that the remainder stays above the subnormal numbers.
struct RowScale {
  float scale, lift, lifted, inv;
  bool bad;
};
template <typename TO>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale r;
  const float amax = __uint_as_float(top);
  r.bad = !(amax < INFINITY);
  r.scale = amax == 0.0f ? 1.0f : fmaxf(amax / kTop<TO>, 0x1p-126f);
  if (r.bad) r.scale = __uint_as_float(0x7fc00000u);
  r.lift = r.scale < 0x1p-60f ? 0x1p64f : 1.0f;
  r.lifted = r.scale * r.lift;
  r.inv = 1.0f / r.lifted;
  return r;
}
__device__ __forceinline__ f32x8 quotients(f32x8 v, const RowScale &r) {
  v *= r.lift;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = v[e] * r.inv;
    v[e] = fmaf(-fmaf(q, r.lifted, -v[e]), r.inv, q);  // (this way round, -0 keeps its sign)
  }
  return v;
}

// The largest |v| of the row group's threads (T a wave, or all of a workgroup).
template <int T>
__device__ __forceinline__ uint32_t group_top(uint32_t top, uint32_t *lds) {
  top = wave_umax(top);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63u) == 0) lds[threadIdx.x >> 6] = top;
    wait_lds_all();
    wg_barrier();
    top = 0;
#pragma unroll
    for (int q = 0; q < T / 64; ++q) top = max(top, lds[q]);
  }
  return top;
}
__device__ __forceinline__ uint32_t top8(const f32x8 &v, uint32_t top) {
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  return top;
}

template <int T, int NCH, typename TS, typename TO>
__global__ __launch_bounds__(T < 256 ? 256 : T) void ptg_quantise_kernel(const QuantiseArgs a, int32_t groups) {
  constexpr int kGroups = T < 256 ? 256 / T : 1;
  __shared__ uint32_t lds[2][16];
  const int32_t t = (int32_t)threadIdx.x % T;
  const int32_t group = (int32_t)blockIdx.x * kGroups + (int32_t)threadIdx.x / T;
  typedef typename Raw8<TS>::type raw;
  struct Row { raw x[NCH]; };
  auto ask = [&](Row &f, int64_t row) {
    const TS *x = (const TS *)a.x + row * a.ldx;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      f.x[c] = {};
      if (j < a.n) f.x[c] = *(const raw *)(x + j);
    }
  };
  Row next;
  if (group < a.m) ask(next, group);
  int buf = 0;
  for (int64_t row = group; row < a.m; row += groups, buf ^= 1) {
    const Row mine = next;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) top = top8(widen(mine.x[c]), top);
    if (row + groups < a.m) ask(next, row + groups);
    // (two buffers: a row's reads are over before the row after next writes)
    const RowScale r = row_scale<TO>(group_top<T>(top, lds[buf]));
    if (t == 0) a.scale[row] = r.scale;
    TO *out = (TO *)a.out + row * a.ldo;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int32_t j = (c * T + t) * 8;
      if (j < a.n) store_codes(out + j, quotients(widen(mine.x[c]), r), r.bad);
    }
  }
}

template <typename TS, typename TO>
__global__ __launch_bounds__(1024) void ptg_quantise_long_kernel(const QuantiseArgs a) {
  __shared__ uint32_t lds[2][16];
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, buf ^= 1) {
    const TS *x = (const TS *)a.x + row * a.ldx;
    TO *out = (TO *)a.out + row * a.ldo;
    uint32_t top = 0;
#pragma unroll 4
    for (int32_t j = (int32_t)threadIdx.x * 8; j < a.n; j += 8192) top = top8(load8(x + j), top);
    const RowScale r = row_scale<TO>(group_top<1024>(top, lds[buf]));
    if (threadIdx.x == 0) a.scale[row] = r.scale;
#pragma unroll 4
    for (int32_t j = (int32_t)threadIdx.x * 8; j < a.n; j += 8192) store_codes(out + j, quotients(load8(x + j), r), r.bad);
  }
}

template <int T, int NCH, typename TS, typename TO>
static hipError_t launch_shape(const QuantiseArgs &a, int cu_count, hipStream_t s) {
  constexpr int kBlock = T < 256 ? 256 : T, kGroups = kBlock / T;
  // every group a CU's 2048 threads hold
  const int64_t resident = (int64_t)cu_count * (2048 / kBlock);
  const int64_t grid = std::min<int64_t>((a.m + kGroups - 1) / kGroups, resident);
  hipLaunchKernelGGL((ptg_quantise_kernel<T, NCH, TS, TO>), dim3((uint32_t)grid), dim3(kBlock), 0, s, a, (int32_t)(grid * kGroups));
  return hipGetLastError();
}

template <typename TS, typename TO>
static hipError_t launch_types(const QuantiseArgs &a, int cu_count, hipStream_t s) {
  const int32_t chunks = (a.n + 7) / 8;
  if (chunks <= 64) return launch_shape<64, 1, TS, TO>(a, cu_count, s);
  if (chunks <= 128) return launch_shape<64, 2, TS, TO>(a, cu_count, s);
  if (chunks <= 256) return launch_shape<256, 1, TS, TO>(a, cu_count, s);
  if (chunks <= 512) return launch_shape<256, 2, TS, TO>(a, cu_count, s);
  if (chunks <= 1024) return launch_shape<1024, 1, TS, TO>(a, cu_count, s);
  if (chunks <= 2048) return launch_shape<1024, 2, TS, TO>(a, cu_count, s);
  if (chunks <= 4096) return launch_shape<1024, 4, TS, TO>(a, cu_count, s);
  const int64_t grid = std::min<int64_t>(a.m, (int64_t)cu_count * 2);
  hipLaunchKernelGGL((ptg_quantise_long_kernel<TS, TO>), dim3((uint32_t)grid), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_quantise(const QuantiseArgs &a, int cu_count, hipStream_t s) {
  if (a.type == kTypeF32)
    return a.out_type == kTypeI8 ? launch_types<float, i8_t>(a, cu_count, s) : launch_types<float, e4m3_t>(a, cu_count, s);
  return a.out_type == kTypeI8 ? launch_types<__bf16, i8_t>(a, cu_count, s) : launch_types<__bf16, e4m3_t>(a, cu_count, s);
}

}  // namespace ptg
