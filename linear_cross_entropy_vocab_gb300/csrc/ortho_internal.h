// Parameters of the orthogonalising kernels (kernels_ortho.cu), filled in by
// the entry points in ortho_api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {

// The matrices as the caller has them, and their copy in halves: x[b] is
// [m_pad][n_pad] with m <= n, the transpose of src[b] where `tall`, zeros
// outside [m][n] up to row m_rows; what lies in the rows after that is read
// into rows and columns of tiles that are not stored.
struct OrthoCopyParams {
  const void* src;
  int64_t batch_stride, row_pitch;  // elements
  int32_t batch, rows, cols;        // of src
  int32_t tall;
  int32_t m, n, m_pad, n_pad;
  void* x;
  double* partial;   // [batch][parts] sums of squares
  int32_t parts;
  float eps;
  int32_t x_shift;   // x holds src / norm times 2^x_shift, but for factor
  int32_t m_rows;    // rows of x that are filled: a multiple of 64
  int32_t* arrived;  // cleared for the products
  int32_t arrived_count;
  float* factor;     // [batch]: x = src / (norm + eps) is factor times what x holds
};
cudaError_t launch_ortho_norm(const OrthoCopyParams& p, int dtype, cudaStream_t s);
cudaError_t launch_ortho_copy(const OrthoCopyParams& p, int dtype, cudaStream_t s);

enum class OrthoOp {
  kGram,     // c = x x^T
  kPoly,     // c = a I + b g + c g g
  kMul,      // c = p x
  kOutWide,  // out = p x
  kOutTall,  // out = x^T p, of the transposed copy of a tall matrix
};

// One product over all matrices of the batch. Sides are padded to tiles; the
// loads' maps are boxes of 64 x 128 (contraction contiguous) or 64 x 64
// (contraction across rows), the store's 32 x 32 with 64-byte swizzle.
struct OrthoGemmParams {
  CUtensorMap a_map, b_map, c_map;
  int32_t batch, m_tiles, n_tiles, k_iters;
  int32_t units;                     // pairs of CTAs
  int32_t whole_tiles, split_tiles;  // of all tiles, in this order
  void* shares;      // sums of cut tiles: two of 256 KB for each pair
  int32_t* arrived;  // [split_tiles][2 CTAs][8 warps], zeros before and after
  int32_t a_stride, b_stride;  // rows of a map between two matrices
  int32_t m_pad;               // rows of c between two matrices
  float acc_scale;             // of the accumulator
  const float* factor;         // or null: [batch], its power is in factor_square
  int32_t factor_square;
  float old_scale, diag;       // kPoly: of the gram's halves, and on the diagonal
  const void* old;             // kPoly: the gram, rows m_pad apart
  void* out;                   // kOut*: rows x cols of out_dtype, dense
  int32_t out_mapped;          // kOut*: through c_map, of out [batch][rows][cols]
  int32_t rows, cols;          // of out, or of c: what is stored of a matrix
  int32_t* err_word;
};
cudaError_t launch_ortho_gemm(const OrthoGemmParams& p, OrthoOp op, int out_dtype,
                              cudaStream_t s);

constexpr int kOrthoTile = 256;
constexpr int kOrthoWarps = 8;  // that store a tile, in each CTA
constexpr int kOrthoShareBytes = kOrthoTile * kOrthoTile * 4;

}  // namespace flce
