// Parameters of the 8-bit integer kernels (kernels_int8.cu), filled in by the
// entry points in int8_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "flce.h"
#include "flce_math.cuh"

namespace flce {

struct QuantParams {
  const void* x;
  int64_t n, h, x_pitch;
  int8_t* q;
  int64_t q_pitch;
  float* scale;
};
cudaError_t launch_quantize_rows(const QuantParams& p, int dtype, cudaStream_t s);

struct QLinearParams {
  const int8_t* x;
  const float* x_scale;
  const int8_t* weight;
  const float* weight_scale;
  const void* bias;  // or null
  void* out;
  int64_t n, h, v;
  int64_t x_pitch, weight_pitch, out_pitch;
  int32_t out_dtype, bias_dtype;
  LogitXform xf;
};
cudaError_t launch_qlinear_simple(const QLinearParams& p, cudaStream_t s);

}  // namespace flce
