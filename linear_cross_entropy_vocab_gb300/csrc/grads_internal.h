// The table of tensors that the gradient kernels get by value, and their
// launchers (kernels_grads.cu), used by the entry points in grads_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {

// Source bytes of one chunk: what a CTA takes at a time.
constexpr int kGradChunkBytes = 32768;
// CTAs per SM of the norm and of the clip: the kernels are compiled to fit that
// many, and the grids are that large. The clip holds a chunk's 16-byte loads and
// the places of its stores, 128 registers a thread; four CTAs of 64 spill, and
// 640 MB read and written take 270 us in fp32 and 216 in bf16, against 209 and
// 212 with two.
constexpr int kGradNormCtasPerSm = 4;
constexpr int kGradClipCtasPerSm = 2;
// Tensors in one launch. Kernel parameters end at 32,764 bytes; the smaller
// tables keep the parameters of a call with few tensors short (59 small ones:
// 65 us a clip in place with the medium table, 69 with the large).
constexpr int kGradTableSmall = 32;
constexpr int kGradTableMedium = 128;
constexpr int kGradTableLarge = 500;

struct GradEntry {
  const void* src;
  void* dst;          // null for the norm alone
  int64_t n;          // elements
  int64_t cols;       // contiguous elements of a row (n: the tensor is one run)
  int64_t src_pitch;  // elements from row to row
  int64_t dst_pitch;
  int32_t src_dtype;
  int32_t dst_dtype;
};

template <int CAP>
struct GradTable {
  GradEntry t[CAP];
  uint32_t first[CAP + 1];  // first chunk of each tensor; first[count]: all chunks
  int32_t count;
  int32_t in_place;  // every dst is its src: nothing to write where the factor is 1
};
static_assert(sizeof(GradTable<kGradTableLarge>) + 64 <= 32764, "kernel parameters");

template <int CAP>
cudaError_t launch_grad_partials(const GradTable<CAP>& tab, int p, int max_ctas, double* partials,
                                 int* n_partials, cudaStream_t s);
cudaError_t launch_grad_norm(const double* partials, int n, int p, float* norm_out,
                             cudaStream_t s);
// Norm and clip in one launch, by a cluster of kGradCluster CTAs.
constexpr int kGradCluster = 8;
cudaError_t launch_grad_clip_cluster(const GradTable<kGradTableSmall>& tab, int p, float max_norm,
                                     float eps, float* norm_out, cudaStream_t s);
template <int CAP>
cudaError_t launch_grad_clip(const GradTable<CAP>& tab, const double* partials, int n, int p,
                             float max_norm, float eps, float* norm_out, bool write_norm,
                             int max_ctas, cudaStream_t s);

}  // namespace flce
