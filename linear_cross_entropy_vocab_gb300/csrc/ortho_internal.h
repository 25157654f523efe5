// Parameters of the orthogonalising kernels (kernels_ortho.cu), filled in by
// the entry points in ortho_api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {

constexpr int kOrthoTile = 256;  // or half of it
constexpr int kOrthoWarps = 8;  // that store a tile, in each CTA
constexpr int kOrthoShareBytes = kOrthoTile * kOrthoTile * 4;
constexpr int kOrthoMaxSteps = 64;
// The SMs that the norm's and the copy's shares are planned for. The workspace and
// the order of the norm's sums go by it, so it is not the device's own number:
// with that, results and sizes would depend on the device.
constexpr int kOrthoPlanSms = 152;

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
  int32_t* count;    // cleared for the products
  int32_t counts;
  float* factor;     // [batch]: x = src / (norm + eps) is factor times what x holds
};
cudaError_t launch_ortho_norm(const OrthoCopyParams& p, int dtype, cudaStream_t s);
cudaError_t launch_ortho_copy(const OrthoCopyParams& p, int dtype, cudaStream_t s);

// What turns a step's accumulators into halves of the next operand's scale.
struct OrthoStep {
  float gram;             // x x^T
  float poly, old, diag;  // the square, the gram's halves, and on the diagonal
  float product;
};

enum class OrthoOp : int {
  kGram,     // c = a a^T over x's columns
  kSquare,   // c = a b of polynomials of one gram, which commute: symmetric
  kPoly,     // c = diag I + old a + a a, a the gram
  kMul,      // c = a x
  kOutWide,  // out = a x
  kOutTall,  // out = x^T b, of the transposed copy of a tall matrix
};
// The operands and results of products: two copies of x and four m x m
// matrices; the result of the last.
enum OrthoBuffer { kOrthoX0, kOrthoX1, kOrthoGram, kOrthoP0, kOrthoP1, kOrthoP2, kOrthoBuffers,
                   kOrthoOut = kOrthoBuffers };
struct OrthoProduct {
  int8_t op, a, b, c;  // OrthoOp, OrthoBuffer
  int8_t cut;          // of the cuts: 0 kGram, 1 symmetric ones else, 2 with x
  int8_t power;        // of the norm's factor
  float scale;         // of the sums
  float old, diag;     // kPoly
  int32_t need;        // what a matrix (or all: joint) has counted before
};
// Three steps a group (see ortho_api.cu) are eleven products.
constexpr int kOrthoMaxProducts = 240;

// Of a product's tiles over the whole batch, `whole` are taken whole and `cut`
// along their contraction, among `units` pairs of CTAs (or CTAs).
struct OrthoCut {
  int32_t units, whole, cut;
};

// All steps over all matrices. Sides are padded to tiles; `along` maps have boxes
// of 64 along the contraction x 128 rows, `across` (of x) of 64 x 64 with the
// contraction across rows, `store` of 32 x 32 with 64-byte swizzle.
struct OrthoRunParams {
  CUtensorMap along[kOrthoBuffers], across[2];
  CUtensorMap store[kOrthoBuffers + 1];  // the last: out [batch][rows][cols], where out_mapped
  OrthoProduct product[kOrthoMaxProducts];
  OrthoCut cut[3];
  int32_t products, batch;
  int32_t units, items;  // pairs of CTAs in the grid, and what they draw
  int32_t* ticket;       // 0 before
  int32_t pairs;       // tiles of 256 by CTA pairs, else of 128 by CTAs
  int32_t m_tiles, n_tiles;
  int32_t k_n, k_m;    // 64-deep stages along n and along m
  int32_t m_pad, m_rows, n_pad;
  int32_t out_mapped, rows, cols;  // of out
  int32_t joint;       // matrices count together (where tiles are cut)
  const float* factor; // [batch]
  const void* gram;
  void* out;           // dense
  void* shares;        // sums of cut tiles: two of 256 KB for each pair (64 for each CTA)
  int32_t* arrived;    // [cut][CTAs of a tile][8 warps], zeros before and after
  int32_t* finished;   // [batch], zeros before
  uint64_t wait_ns;    // after which a wait gives up
  int32_t* err_word;
};
cudaError_t launch_ortho_run(const OrthoRunParams& p, int out_dtype, cudaStream_t s);

// Matrices with one side of at most 128, each in the shared memory of a cluster
// of CTAs with `slab` columns each (a multiple of 64, at most 512).
constexpr int kOrthoMaxCluster = 8;
struct OrthoSmallParams {
  OrthoStep step[kOrthoMaxSteps];
  const void* src;
  int64_t batch_stride, row_pitch;
  void* out;  // dense
  int32_t batch, rows, cols, tall, steps, cluster, slab;
  int32_t x_shift, out_bf16;
  float eps;
  int32_t* err_word;
};
cudaError_t launch_ortho_small(const OrthoSmallParams& p, int dtype, cudaStream_t s);

}  // namespace flce
