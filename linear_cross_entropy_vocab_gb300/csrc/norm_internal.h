// Parameters of the root-mean-square norm's kernels (kernels_norm.cu,
// kernels_norm_q.cu, kernels_norm_bwd.cu), filled in by the entry points in
// norm_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {

struct NormParams {
  const void* x;         // of the problem's dtype
  const void* residual;  // or null; fp32 where wide, else dtype
  const void* weight;    // or null; fp32 where weight_wide, else dtype
  void* sum;             // with residual; rows h apart
  void* y;               // dtype, rows h apart (kernels_norm.cu)
  int8_t* q;             // kernels_norm_q.cu
  float* scale;
  float* rstd;           // or null
  int64_t n, h, x_pitch, residual_pitch, q_pitch;
  int32_t wide, weight_wide, sms;
  float eps;
};
cudaError_t launch_rms_norm(const NormParams& p, int dtype, cudaStream_t s);
cudaError_t launch_rms_norm_q(const NormParams& p, int dtype, cudaStream_t s);

struct NormBwdParams {
  const void* grad_y;    // dtype, rows h apart
  const void* grad_sum;  // or null; fp32 where wide, else dtype, rows h apart
  const void* total;     // what was normalised; fp32 where wide, else dtype
  const void* weight;    // or null
  const float* rstd;
  void* grad_x;          // or null; dtype, rows h apart
  void* grad_residual;   // or null; fp32 (wide only), rows h apart
  void* grad_weight;     // or null; the weight's type
  float* partial;        // [parts][h] sums for grad_weight
  float* along;          // [n], rows too long for one CTA only
  int64_t n, h, total_pitch;
  int32_t wide, weight_wide;
};
// The most CTAs that each leave one row of partial sums.
int64_t norm_bwd_parts(int64_t n, int64_t h, int sms);
// Rows of more values go through `along`.
constexpr int64_t kNormBwdMaxH = 16384;
cudaError_t launch_rms_norm_bwd(const NormBwdParams& p, int dtype, int sms, cudaStream_t s);

}  // namespace flce
