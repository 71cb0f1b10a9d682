// linear.cuh -- powers of a head's decay, shared by the linear attention kernels.
#pragma once

#include "fs_common.cuh"

namespace fs {

// exp(decay)^n as the sum of two fp32 numbers.
struct Factor {
  float hi, lo;
  __device__ __forceinline__ float times(float x, float plus) const {
    return fmaf(x, hi, fmaf(x, lo, plus));
  }
};

// decay <= 0, n >= 0.  The argument n * decay is a product kept whole (its rounding
// goes into lo).  Near 1, where a state is multiplied again and again, hi + lo comes from
// expm1 and is good to 2^-24 of 1 - lam; below 1/2 the exponential alone, 2^-22 of itself,
// is left: a state that is halved at every step remembers no errors.
__device__ __forceinline__ Factor decay_power(float decay, int n) {
  if (n == 0) return {1.f, 0.f};  // (also where decay is -inf)
  const float x = decay * (float)n;
  if (x < -1e30f) return {0.f, 0.f};
  const float rest = fmaf(decay, (float)n, -x);
  const float hi = expf(x);
  float lo = hi * rest;
  if (hi >= 0.5f) lo += expm1f(x) - (hi - 1.f);
  return {hi, lo};
}

}  // namespace fs
