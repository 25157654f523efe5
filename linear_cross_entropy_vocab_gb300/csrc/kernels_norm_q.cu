// The root-mean-square norm with the residual's addition, output in 8-bit
// integers with a scale for each row.
#include "norm_fwd.cuh"

namespace flce {

cudaError_t launch_rms_norm_q(const NormParams& p, int dtype, cudaStream_t s) {
  return launch_norm<true>(p, dtype, s);
}

}  // namespace flce
