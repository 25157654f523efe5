// The root-mean-square norm with the residual's addition, output in the input's
// type.
#include "norm_fwd.cuh"

namespace flce {

cudaError_t launch_rms_norm(const NormParams& p, int dtype, cudaStream_t s) {
  return launch_norm<false>(p, dtype, s);
}

}  // namespace flce
