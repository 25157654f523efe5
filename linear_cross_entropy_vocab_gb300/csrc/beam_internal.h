// Parameters of the beam search kernels (kernels_beam.cu), filled in by the
// entry points in beam_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {

constexpr int kBeamMaxCandidates = 256;
constexpr int kBeamMaxBeams = 64;  // of a reordering
constexpr int kBeamMaxSelectBeams = 1024;

// A selection CTA (256 threads) holds tiles of 16 bytes or of 16 logits for
// each thread.
constexpr int kTileSmallBytes = 256 * 16;
constexpr int kTileLarge = 256 * 16;

struct BeamSelectParams {
  const void* logits;
  int64_t stride_b, stride_k;  // elements
  const uint8_t* allowed;      // or null
  int64_t allowed_b, allowed_k;
  const float* beam_scores;    // [B][K]
  const uint8_t* finished;     // [B][K] or null
  int32_t batch, beams, m, splits;
  int32_t slice_len;           // logits of a slice, a multiple of 8 (the last may be shorter)
  int32_t groups;              // the power of two from m on, at most 256
  int32_t shifted;             // some row starts elsewhere than at a multiple of 16 bytes
  int64_t v;
  int64_t pad_token;
  // per (row, slice): its M best keys, best first, 0 where there are fewer,
  // and its maximum and sum of exponentials
  uint64_t* keys;
  float2* stats;
  float* scores_out;      // [B][M]
  int64_t* parents_out;   // [B][M]
  int64_t* tokens_out;    // [B][M]
  int32_t* err_word;
};

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, bool large,
                               cudaStream_t s);

constexpr int kReorderDims = 4;
// States of one launch: the small table keeps the parameters of a call with
// few states short.
constexpr int kReorderSmall = 8;
constexpr int kReorderLarge = 256;

// One state: `total` vectors of `width` bytes in runs of `run`, at the places
// that the (at most 4) outer extents and strides give, for each of
// batch x beams beams `beam_stride` bytes apart.
struct ReorderEntry {
  uint8_t* data;
  int64_t beam_stride;
  int64_t stride[kReorderDims];  // bytes, outermost first
  uint32_t size[kReorderDims];   // 1 where unused
  uint32_t run;                  // vectors in one contiguous run
  uint32_t total;                // vectors of one beam
  uint32_t width;                // 16 (at most 32 beams), 8, 4, 2 or 1
};

template <int CAP>
struct ReorderTable {
  ReorderEntry e[CAP];
  uint32_t first[CAP + 1];  // first block of each state
  int32_t count;
  int32_t batch, beams;
  const int64_t* parents;
  int32_t* err_word;
};
static_assert(sizeof(ReorderTable<kReorderLarge>) <= 32764, "kernel parameters");

template <int CAP>
cudaError_t launch_beam_reorder(const ReorderTable<CAP>& t, int64_t blocks, cudaStream_t s);

// Vectors of one beam that a block takes.
constexpr int kReorderBlock = 256;

}  // namespace flce
