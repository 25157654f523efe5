// What the orthogonalising kernels share.
#pragma once

#include <cmath>

namespace flce {

// x = src / (|src| + eps) as src * 2^-exponent times a factor in (1/2, 1], from
// the sum of squares. A norm that is not finite has the factor NaN: every
// result is NaN.
__device__ __forceinline__ void norm_factor(double squares, float eps, int& exponent,
                                            float& factor) {
  const double norm = sqrt(squares) + static_cast<double>(eps);
  exponent = 0;
  factor = NAN;
  if (norm < INFINITY) {
    exponent = ilogb(norm);
    factor = static_cast<float>(scalbn(1.0 / norm, exponent));
  }
}

}  // namespace flce
