// Parameters of the 8-bit integer kernels (kernels_int8.cu, kernels_qlinear.cu),
// filled in by the entry points in int8_api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce.h"
#include "flce_math.cuh"

namespace flce {

// Rows to 8-bit integers (q), or to the same integers as halves in the order
// that the linear kernel's tensor-memory operand has (wide: 0, 2, 1, 3 in each
// four, zeros from h to wide_pitch, a multiple of 64).
struct QuantParams {
  const void* x;        // of type dtype; FLCE_Q_I8: integers already (wide only)
  int64_t n, h, x_pitch;
  int8_t* q;
  int64_t q_pitch;
  void* wide;
  int64_t wide_pitch;
  float* scale;         // not written for FLCE_Q_I8
};
cudaError_t launch_quantize_rows(const QuantParams& p, int dtype, cudaStream_t s);
cudaError_t launch_widen_rows(const QuantParams& p, int dtype, cudaStream_t s);

// Rows of h bytes copied to rows of a pitch that TMA can read.
cudaError_t launch_align_rows(const int8_t* src, int64_t rows, int64_t h, int64_t src_pitch,
                              int8_t* dst, int64_t dst_pitch, cudaStream_t s);

struct QLinearTcParams {
  CUtensorMap w_map;  // weight, bytes [v][h], box {128, 128}
  CUtensorMap x_map;  // widened x, halves [n][64-multiple], box {64, nt / CG}
  const float* x_scale;
  const float* weight_scale;
  const void* bias;  // or null
  void* out;
  int64_t n, v, out_pitch;
  int32_t bias_dtype;
  int32_t nt;                 // rows of x in a tile
  int32_t n_tiles, v_tiles;   // tiles along x and along the weight
  int32_t band;               // tiles of x that run through the weight together
  int32_t k_blocks;           // 64-deep blocks of h
  int32_t w_stages, x_stages; // set by the launcher
  int* err_word;
  LogitXform xf;
};
// cg: 1, or 2 for pairs of CTAs (256 weight rows).
cudaError_t launch_qlinear_tc(const QLinearTcParams& p, int cg, int out_dtype, int sms,
                              cudaStream_t s);

}  // namespace flce
