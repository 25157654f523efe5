// Rounding to 8-bit integers and storing them, shared by the kernels that quantise rows.
#pragma once

#include <cmath>
#include <cstdint>

namespace flce {

constexpr float kToInt = 12582912.0f;  // 1.5 * 2^23: adding it rounds to whole numbers

// x / scale rounded to whole numbers, halves to even, plus kToInt (the integer
// is in the low byte). Values of a short type are multiples of few scales, and
// halves are common: the quotient has to be the correctly rounded one. It is,
// from a product with the correctly rounded reciprocal and one correction by
// the exact remainder (Markstein 1990, theorem on division), where nothing
// leaves the normal range: quotients below a half need no more than to stay
// there.
__device__ __forceinline__ void round8(float (&x)[8], float scale, float inv) {
  if (scale >= 1.0e-28f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = x[j] * inv;
      x[j] = fmaf(fmaf(-q, scale, x[j]), inv, q) + kToInt;
    }
    return;
  }
  // a tiny scale, 0 or NaN
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = scale > 0.0f ? rintf(__fdiv_rn(x[j], scale)) : 0.0f;
    x[j] = fminf(127.0f, fmaxf(-127.0f, q)) + kToInt;
  }
}

__device__ __forceinline__ void put_bytes(int8_t* q, int64_t e, int64_t h, bool vec,
                                          const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __byte_perm(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), 0x40);
    const uint32_t hi =
        __byte_perm(__float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]), 0x40);
    w[i] = __byte_perm(lo, hi, 0x5410);
  }
  if (vec && e + 8 <= h) {
    *reinterpret_cast<uint2*>(q + e) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < h) q[e + j] = static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
  }
}

}  // namespace flce
