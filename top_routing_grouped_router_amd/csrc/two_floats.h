// 1 / rms as two floats, and the norm's products with it to more than fp32's bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// hi + lo, hi the nearest float
struct Rstd {
  float hi, lo;
};

// y = s rstd w to about 2^-45, rounded to odd, so that any later rounding to fewer
// bits is that of the sum itself
__host__ __device__ __forceinline__ float scaled_odd(float s, Rstd r, float w) {
  // as written: with y = n w joined into the sums that follow, what y's own rounding lost
  // would count twice
#pragma clang fp contract(off)
  const float n = s * r.hi, en = __builtin_fmaf(s, r.lo, __builtin_fmaf(s, r.hi, -n));
  const float y = n * w, ey = __builtin_fmaf(en, w, __builtin_fmaf(n, w, -y));
  const float hi = y + ey, lo = (y - hi) + ey;
  const uint32_t u = __builtin_bit_cast(uint32_t, hi);
  const int away = static_cast<int>(u ^ __builtin_bit_cast(uint32_t, lo)) < 0 ? -1 : 1;
  return __builtin_bit_cast(float, lo != 0.0f && !(u & 1) ? u + away : u);
}

}  // namespace moe
