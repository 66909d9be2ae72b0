// Sums of exponentials, shared by the kernels that end in a cross entropy's.
#pragma once

#include "layer_device.hpp"

namespace ptg {

// Sums of e^(z - top) as 2^(z log2 e - offset). What the offset's rounding left out of
// top log2 e is the same for all of a row's terms and is put right in their sum; the
// rest is |z - top| 2^-24 of a term, most where the term adds least. An infinite top
// (a block of nothing but -infinity, or a logit of +infinity) is not subtracted.
static constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float offset_of(float top) { return fabsf(top) < INFINITY ? top * kLog2E : 0.0f; }
__device__ __forceinline__ float put_right(float sum, float top, float offset) {
  return fabsf(top) < INFINITY ? fmaf(sum, -fmaf(top, kLog2E, -offset) * kLn2, sum) : sum;
}
// A sum of exponentials below one maximum, below another.
__device__ __forceinline__ float rescaled(float sum, float from, float to) {
  // (equal maxima are not subtracted: both may be infinite)
  return from == to ? sum : sum * __builtin_amdgcn_exp2f((from - to) * kLog2E);
}

}  // namespace ptg
