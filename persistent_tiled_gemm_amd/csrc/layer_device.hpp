// Device-side pieces shared by the layer operators' kernels: 8-element loads
// and stores of the stream types, activations and their derivatives, and the
// shapes the host and the kernels agree on.
#pragma once

#include "ptg_device.hpp"
#include "layer_internal.hpp"

namespace ptg {

typedef __attribute__((ext_vector_type(8))) float f32x8;

// Eight consecutive elements as fp32. Rows are 16-byte aligned (8-byte for e4m3).
template <typename T> __device__ __forceinline__ f32x8 load8(const T *p);
template <> __device__ __forceinline__ f32x8 load8<float>(const float *p) {
  const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <> __device__ __forceinline__ f32x8 load8<__bf16>(const __bf16 *p) {
  return __builtin_convertvector(*(const bf16x8 *)p, f32x8);
}
// The same eight elements as they lie in memory, and widened.
template <typename T> struct Raw8;
typedef f32x8 f32x8_a16 __attribute__((aligned(16)));  // rows of fp32 are 16-byte aligned
template <> struct Raw8<float> { typedef f32x8_a16 type; };
template <> struct Raw8<__bf16> { typedef bf16x8 type; };
__device__ __forceinline__ f32x8 widen(const f32x8_a16 &v) { return v; }
__device__ __forceinline__ f32x8 widen(const bf16x8 &v) { return __builtin_convertvector(v, f32x8); }
// The element type named at run time (the weight's or a bias's: read once a row or column).
__device__ __forceinline__ f32x8 load8_as(const void *p, int32_t type, int64_t i) {
  return type == kTypeF32 ? load8((const float *)p + i) : load8((const __bf16 *)p + i);
}

// Rounded to nearest even, once, from the fp32 result.
template <typename T> __device__ __forceinline__ void store8(T *p, const f32x8 &v);
template <> __device__ __forceinline__ void store8<float>(float *p, const f32x8 &v) {
  *(f32x4 *)p = __builtin_shufflevector(v, v, 0, 1, 2, 3);
  *(f32x4 *)(p + 4) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
}
template <> __device__ __forceinline__ void store8<__bf16>(__bf16 *p, const f32x8 &v) {
  *(bf16x8 *)p = __builtin_convertvector(v, bf16x8);
}
static constexpr float kE4m3Max = 448.0f;  // the largest e4m3 value
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
// Four at a time (rows are 8-byte aligned there).
__device__ __forceinline__ f32x4 load4_as(const void *p, int32_t type, int64_t i) {
  return type == kTypeF32 ? *(const f32x4 *)((const float *)p + i) : __builtin_convertvector(*(const bf16x4 *)((const __bf16 *)p + i), f32x4);
}
__device__ __forceinline__ void store4(__bf16 *p, const f32x4 &v) { *(bf16x4 *)p = __builtin_convertvector(v, bf16x4); }
struct e4m3_t { uint8_t bits; };
template <> __device__ __forceinline__ void store8<e4m3_t>(e4m3_t *p, const f32x8 &v) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  *(int2 *)p = make_int2(lo, hi);
}

// z p for p in [0, 1] that vanishes as z goes to -infinity: the most negative
// value stands in for -infinity, whose product with p = 0 would be NaN. (A NaN z
// has a NaN p.)
__device__ __forceinline__ float times_p(float z, float p) { return fmaxf(z, -3.402823466e38f) * p; }

// e^t as 2^h (1 + l ln 2): h is the fp32 product of t with log2 e, l what its rounding
// left out (|t| 2^-24, which 2^h would turn into as much of the result: 2^-18 at t =
// -60). Relative error: 2^-23 from the instruction and two roundings. l is NaN or
// large only where 2^h is 0, infinite or NaN itself: kept within 1, it does no harm.
static constexpr float kLog2e = 1.4426950216293335f, kLog2eLow = 1.925962991e-8f;  // their sum is log2 e
static constexpr float kLn2 = 0.69314718055994531f;
__device__ __forceinline__ float exp2_parts(float h, float l) {
  return __builtin_amdgcn_exp2f(h) * fmaf(__builtin_amdgcn_fmed3f(l, -1.0f, 1.0f), kLn2, 1.0f);
}
__device__ __forceinline__ float exp_f32(float t) {
  const float h = t * kLog2e;
  return exp2_parts(h, fmaf(t, kLog2eLow, fmaf(t, kLog2e, -h)));
}
// The same without the second part, off by 1.25 |t| 2^-24 more: for a t that is a
// rounded formula itself and brings several |t| 2^-24 along.
__device__ __forceinline__ float exp_of_rounded(float t) { return __builtin_amdgcn_exp2f(t * kLog2e); }

// The same past the caches: written once, not read by the kernel that writes it.
template <typename T> __device__ __forceinline__ void store8_nt(T *p, const f32x8 &v);
template <> __device__ __forceinline__ void store8_nt<float>(float *p, const f32x8 &v) {
  __builtin_nontemporal_store(__builtin_shufflevector(v, v, 0, 1, 2, 3), (f32x4 *)p);
  __builtin_nontemporal_store(__builtin_shufflevector(v, v, 4, 5, 6, 7), (f32x4 *)(p + 4));
}
template <> __device__ __forceinline__ void store8_nt<__bf16>(__bf16 *p, const f32x8 &v) {
  __builtin_nontemporal_store(__builtin_convertvector(v, bf16x8), (bf16x8 *)p);
}

// Activations in fp32. The logistic function is 1 / (1 + e), e = e^-t: an e that
// overflows to infinity gives 0.
__device__ __forceinline__ float logistic(float e) { return __builtin_amdgcn_rcpf(1.0f + e); }

template <> __device__ __forceinline__ void store8_nt<e4m3_t>(e4m3_t *p, const f32x8 &v) {
  typedef __attribute__((ext_vector_type(2))) int i32x2;
  i32x2 w;
  store8((e4m3_t *)&w, v);
  __builtin_nontemporal_store(w, (i32x2 *)p);
}

// e^(-z^2 / 2), with the square's rounding in the second part.
__device__ __forceinline__ float exp_half_square(float z) {
  const float s = z * z, h = s * (-0.5f * kLog2e);
  const float l = fmaf(s, -0.5f * kLog2eLow, fmaf(s, -0.5f * kLog2e, -h));
  return exp2_parts(h, fmaf(fmaf(z, z, -s), -0.5f * kLog2e, l));
}

// Phi(z), the normal distribution function, from e = e^(-z^2 / 2): Phi(-x) / e is a
// quotient of polynomials, fitted by least squares with weights that level the
// relative error (5.9e-9 on 0 <= x <= 14.5; e is 0 before x is 16). All coefficients
// are positive, so that nothing cancels, and the left tail keeps its relative
// accuracy: 30 units of 2^-24 at most. (8192^3 with gelu in the epilogue: 770 us with
// a formula whose tail was off by 1.6e-3 at z = -5, 790 with this one.)
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float x = fminf(fabsf(z), 16.0f);
  const float p = fmaf(fmaf(fmaf(fmaf(0.004116168134667482f, x, 0.04063235291871609f), x, 0.1832326667812138f), x, 0.43829180723955086f), x, 0.5f);
  const float q = fmaf(fmaf(fmaf(fmaf(fmaf(0.010317583677286739f, x, 0.10185665220121788f), x, 0.46946407313097654f), x, 1.2024931863050052f), x,
                            1.6744685953014102f), x, 1.0f);
  const float tail = e * (p * __builtin_amdgcn_rcpf(q));
  return z < 0.0f ? tail : 1.0f - tail;
}

static constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
static constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_f32(int32_t act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // keeps NaN
    case kActGelu: return times_p(z, normal_cdf(z, exp_half_square(z)));
    // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
    case kActGeluTanh: return times_p(z, logistic(exp_of_rounded(-z * (2.0f * kGeluC + 2.0f * kGeluC * kGeluA * (z * z)))));
    case kActSilu: return times_p(z, logistic(exp_f32(-z)));
    default: return z;
  }
}

// act_f32 of two rows' eight values, the activation decided once.
template <int ACT>
__device__ __forceinline__ void act16_as(f32x8 &a, f32x8 &b) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = act_f32(ACT, a[e]);
    b[e] = act_f32(ACT, b[e]);
  }
}
__device__ __forceinline__ void act16(int32_t act, f32x8 &a, f32x8 &b) {
  switch (act) {
    case kActRelu: act16_as<kActRelu>(a, b); break;
    case kActGelu: act16_as<kActGelu>(a, b); break;
    case kActGeluTanh: act16_as<kActGeluTanh>(a, b); break;
    case kActSilu: act16_as<kActSilu>(a, b); break;
    default: break;
  }
}

// d act / dz. The terms z f'(z) vanish faster than z grows; where the factor
// has underflowed to 0 the term is 0 (selected, so that infinite z gives no NaN).
__device__ __forceinline__ float act_grad_f32(int32_t act, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
    case kActGelu: {
      const float e = exp_half_square(z);
      return normal_cdf(z, e) + (e == 0.0f ? 0.0f : z * (0.39894228040143268f * e));
    }
    case kActGeluTanh: {
      const float p = logistic(exp_of_rounded(-2.0f * kGeluC * (z + kGeluA * z * z * z)));
      const float q = p * (1.0f - p);
      return p + (q == 0.0f ? 0.0f : 2.0f * kGeluC * z * (1.0f + 3.0f * kGeluA * z * z) * q);
    }
    case kActSilu: {
      const float p = logistic(exp_f32(-z));
      const float q = p * (1.0f - p);
      return p + (q == 0.0f ? 0.0f : z * q);
    }
    default: return 1.0f;
  }
}

// Sum (or, for bit patterns, unsigned maximum) over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

}  // namespace ptg
