// C entry points of the beam search operators (include/flce.h): argument
// checks, workspace and launches. Nothing is allocated on the device and
// nothing waits for it.
#include <algorithm>
#include <new>

#include "beam_internal.h"
#include "flce.h"
#include "host_common.h"

namespace {

using namespace flce::host;

// CTAs that a selection is cut into: most of what the GPU holds at a time (four
// on an SM for fp32, six for 16-bit types). Fewer leave SMs without work; more
// spend their time on the start and the end of a slice (64 x 8 rows of 128256,
// fp32 and bf16: 512 CTAs 85 and 77 us, 1024 92 and 82, 1536 108 and 107). A
// call that cannot have kFewCtas large tiles takes small ones: four rows of
// 128256 bf16 take 11 us with 32 slices each and 18 with 63, of which there is
// more to choose from.
constexpr int64_t kSelectCtas = 512;
constexpr int64_t kFewCtas = 100;

// A slice may be a whole row: its length in whole tiles, and the end of the tile
// after the next, stay in 32 bits.
constexpr int64_t kMaxV = 0x7fffffff - 2 * flce::kTileLarge;

struct SelectPlan {
  bool large;
  int64_t splits, slice_len;
  size_t stats, total;  // offset of the slice statistics; bytes in all
};

flce_status check_select(const flce_beam_problem* p) {
  if (p == nullptr) return fail(FLCE_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != FLCE_F32 && p->dtype != FLCE_BF16 && p->dtype != FLCE_F16)
    return fail(FLCE_ERR_INVALID_ARG, "dtype %d is not an flce_dtype", p->dtype);
  if (p->reserved != 0) return fail(FLCE_ERR_INVALID_ARG, "reserved must be 0");
  if (p->batch < 0 || p->batch > 0x7fffffff)
    return fail(FLCE_ERR_INVALID_ARG, "batch %lld", (long long)p->batch);
  if (p->beams < 1 || p->beams > flce::kBeamMaxSelectBeams)
    return fail(FLCE_ERR_UNSUPPORTED, "1 to %d beams are supported, not %lld",
                flce::kBeamMaxSelectBeams, (long long)p->beams);
  if (p->v < 1 || p->v > kMaxV)
    return fail(FLCE_ERR_INVALID_ARG, "vocabulary of %lld tokens", (long long)p->v);
  if (p->candidates < 1 || p->candidates > flce::kBeamMaxCandidates)
    return fail(FLCE_ERR_UNSUPPORTED, "1 to %d candidates are supported, not %lld",
                flce::kBeamMaxCandidates, (long long)p->candidates);
  if (p->pad_token < 0 || p->pad_token >= p->v)
    return fail(FLCE_ERR_INVALID_ARG, "pad_token %lld is not a token", (long long)p->pad_token);
  if (p->stride_batch < 0 || p->stride_beam < 0 || p->allowed_stride_batch < 0 ||
      p->allowed_stride_beam < 0)
    return fail(FLCE_ERR_INVALID_ARG, "strides must not be negative");
  return FLCE_OK;
}

SelectPlan plan_select(const flce_beam_problem* p) {
  SelectPlan q;
  const int64_t rows = p->batch * p->beams;
  const int64_t es = p->dtype == FLCE_F32 ? 4 : 2;
  q.large = rows * ceil_div(p->v, flce::kTileLarge) >= kFewCtas;
  const int64_t tile = q.large ? flce::kTileLarge : flce::kTileSmallBytes / es;
  const int64_t tiles = ceil_div(p->v, tile);
  // slices of whole tiles, as equal as that allows
  const int64_t wanted = ceil_div(kSelectCtas, std::max<int64_t>(rows, 1));
  q.splits = std::max<int64_t>(1, std::min(tiles, wanted));
  q.slice_len = ceil_div(tiles, q.splits) * tile;
  if (q.splits == tiles) q.slice_len = ceil_div(ceil_div(p->v, tiles), 8) * 8;  // alike
  q.splits = ceil_div(p->v, q.slice_len);
  q.stats = align_256(static_cast<size_t>(rows * q.splits * p->candidates) * sizeof(uint64_t));
  q.total = q.stats + align_256(static_cast<size_t>(rows * q.splits) * sizeof(float2));
  return q;
}

// Bytes that a thread moves at a time: the widest that divides the address,
// every stride and the contiguous run.
int width_of(const flce_beam_state& s) {
  uint64_t bits = reinterpret_cast<uintptr_t>(s.data) | static_cast<uint64_t>(s.beam_stride) |
                  static_cast<uint64_t>(s.run_bytes);
  for (int d = 0; d < flce::kReorderDims; ++d)
    if (s.size[d] > 1) bits |= static_cast<uint64_t>(s.stride[d]);
  int w = 16;
  while (w > 1 && (bits % static_cast<uint64_t>(w)) != 0) w /= 2;
  return w;
}

flce_status check_state(const flce_beam_state& s, int64_t i, int64_t rows, bool* empty) {
  int64_t total = s.run_bytes;
  if (s.run_bytes < 0) return fail(FLCE_ERR_INVALID_ARG, "state %lld: run_bytes", (long long)i);
  for (int d = 0; d < flce::kReorderDims; ++d) {
    if (s.size[d] < 0) return fail(FLCE_ERR_INVALID_ARG, "state %lld: size", (long long)i);
    if (s.size[d] > 0xffffffffll || (total > 0 && s.size[d] > (int64_t(1) << 46) / total))
      return fail(FLCE_ERR_UNSUPPORTED, "state %lld is too large", (long long)i);
    total *= s.size[d];
  }
  *empty = total == 0 || rows == 0;
  if (*empty) return FLCE_OK;
  if (s.data == nullptr)
    return fail(FLCE_ERR_INVALID_ARG, "state %lld: data is NULL", (long long)i);
  // every beam's bytes lie apart: sorted by stride, each axis steps over all
  // that the axes inside it span
  int64_t size[flce::kReorderDims + 1], stride[flce::kReorderDims + 1];
  int n = 0;
  for (int d = 0; d < flce::kReorderDims; ++d)
    if (s.size[d] > 1) {
      size[n] = s.size[d];
      stride[n++] = s.stride[d];
    }
  if (rows > 1) {
    size[n] = rows;
    stride[n++] = s.beam_stride;
  }
  for (int a = 1; a < n; ++a)
    for (int b = a; b > 0 && stride[b] < stride[b - 1]; --b) {
      std::swap(stride[b], stride[b - 1]);
      std::swap(size[b], size[b - 1]);
    }
  int64_t span = s.run_bytes;
  for (int a = 0; a < n; ++a) {
    if (stride[a] < span)
      return fail(FLCE_ERR_INVALID_ARG, "state %lld: elements overlap", (long long)i);
    if (size[a] > (int64_t(1) << 46) / stride[a])
      return fail(FLCE_ERR_UNSUPPORTED, "state %lld is too large", (long long)i);
    span += (size[a] - 1) * stride[a];
  }
  return FLCE_OK;
}

// No two states that hold anything start at one address: the second would move
// what the first moves, in no order. States that share memory otherwise are the
// caller's to avoid; views that interleave in one buffer are ordinary.
flce_status check_repeats(const flce_beam_state* states, int64_t count) {
  constexpr int64_t kFew = 64;
  const void* few[kFew];
  const void** const at = count <= kFew ? few : new (std::nothrow) const void*[count];
  if (at == nullptr)
    return fail(FLCE_ERR_INVALID_ARG, "no host memory for %lld states", (long long)count);
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    const flce_beam_state& s = states[i];
    if (s.run_bytes != 0 && s.size[0] != 0 && s.size[1] != 0 && s.size[2] != 0 && s.size[3] != 0)
      at[n++] = s.data;
  }
  std::sort(at, at + n);
  const bool twice = std::adjacent_find(at, at + n) != at + n;
  if (at != few) delete[] at;
  return twice ? fail(FLCE_ERR_INVALID_ARG, "a state is listed twice") : FLCE_OK;
}

// Launches for states that have been checked, each with as many as fit.
template <int CAP>
flce_status reorder(const flce_beam_state* states, int64_t count, const int64_t* parents,
                    int64_t batch, int64_t beams, int max_width, int32_t* err_word,
                    cudaStream_t stream) {
  flce::ReorderTable<CAP> t;
  t.batch = static_cast<int32_t>(batch);
  t.beams = static_cast<int32_t>(beams);
  t.parents = parents;
  t.err_word = err_word;
  t.count = 0;
  int64_t blocks = 0;
  for (int64_t i = 0; i <= count; ++i) {
    int64_t vecs = 0, need = 0;
    int width = 1;
    if (i < count) {
      vecs = states[i].run_bytes;
      for (int d = 0; d < flce::kReorderDims; ++d) vecs *= states[i].size[d];
      if (vecs == 0) continue;
      width = std::min(max_width, width_of(states[i]));
      vecs /= width;
      need = ceil_div(vecs, flce::kReorderBlock) * batch;
    }
    if (t.count > 0 && (i == count || t.count == CAP || blocks + need > 0x7fffffffll)) {
      t.first[t.count] = static_cast<uint32_t>(blocks);
      const cudaError_t e = flce::launch_beam_reorder(t, blocks, stream);
      if (e != cudaSuccess) return cuda_fail(e, "beam reordering kernel");
      t.count = 0;
      blocks = 0;
    }
    if (i == count) break;
    const flce_beam_state& s = states[i];
    flce::ReorderEntry& r = t.e[t.count];
    r.data = static_cast<uint8_t*>(s.data);
    r.beam_stride = s.beam_stride;
    for (int d = 0; d < flce::kReorderDims; ++d) {
      r.size[d] = static_cast<uint32_t>(s.size[d]);
      r.stride[d] = s.stride[d];
    }
    r.run = static_cast<uint32_t>(s.run_bytes / width);
    r.total = static_cast<uint32_t>(vecs);
    r.width = static_cast<uint32_t>(width);
    t.first[t.count++] = static_cast<uint32_t>(blocks);
    blocks += need;
  }
  return FLCE_OK;
}

}  // namespace

extern "C" {

size_t flce_beam_select_workspace_size(const flce_beam_problem* p) {
  if (check_select(p) != FLCE_OK) return 0;
  return plan_select(p).total;
}

flce_status flce_beam_select(const flce_beam_problem* p, const void* logits,
                             const float* beam_scores, const uint8_t* finished,
                             const uint8_t* allowed, float* scores_out, int64_t* parents_out,
                             int64_t* tokens_out, int32_t* err_word, void* workspace,
                             size_t workspace_bytes, void* stream) {
  clear_error();
  flce_status st = check_select(p);
  if (st != FLCE_OK) return st;
  const SelectPlan plan = plan_select(p);
  if (p->batch > 0) {
    if (logits == nullptr || beam_scores == nullptr || scores_out == nullptr ||
        parents_out == nullptr || tokens_out == nullptr)
      return fail(FLCE_ERR_INVALID_ARG,
                  "logits, beam_scores, scores_out, parents_out and tokens_out are required");
    if (!aligned_to(logits, p->dtype == FLCE_F32 ? 4 : 2) || !aligned_to(beam_scores, 4) ||
        !aligned_to(scores_out, 4) || !aligned_to(parents_out, 8) || !aligned_to(tokens_out, 8) ||
        !aligned_to(err_word, 4))
      return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  }
  st = check_workspace(workspace, workspace_bytes, plan.total);
  if (st != FLCE_OK) return st;
  if (p->batch * p->beams * plan.splits > 0x7fffffffll)
    return fail(FLCE_ERR_UNSUPPORTED, "more than 2^31 row slices");
  if (p->beams * plan.splits * p->candidates > 0x7fffffffll)
    return fail(FLCE_ERR_UNSUPPORTED, "more than 2^31 candidates of a prompt's slices");
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || p->batch == 0) return st;
  flce::BeamSelectParams k{};
  k.logits = logits;
  k.stride_b = p->stride_batch;
  k.stride_k = p->stride_beam;
  k.allowed = allowed;
  k.allowed_b = p->allowed_stride_batch;
  k.allowed_k = p->allowed_stride_beam;
  k.beam_scores = beam_scores;
  k.finished = finished;
  k.batch = static_cast<int32_t>(p->batch);
  k.beams = static_cast<int32_t>(p->beams);
  k.m = static_cast<int32_t>(p->candidates);
  k.splits = static_cast<int32_t>(plan.splits);
  const int64_t es = p->dtype == FLCE_F32 ? 4 : 2;
  k.shifted = !aligned_to(logits, 16) || (p->batch > 1 && p->stride_batch * es % 16 != 0) ||
              (p->beams > 1 && p->stride_beam * es % 16 != 0);
  k.groups = 1;
  while (k.groups < k.m) k.groups *= 2;
  k.slice_len = static_cast<int32_t>(plan.slice_len);
  k.v = p->v;
  k.pad_token = p->pad_token;
  k.keys = static_cast<uint64_t*>(workspace);
  k.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan.stats);
  k.scores_out = scores_out;
  k.parents_out = parents_out;
  k.tokens_out = tokens_out;
  k.err_word = err_word;
  const cudaError_t e =
      flce::launch_beam_select(k, p->dtype, plan.large, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "beam selection kernels");
}

flce_status flce_beam_reorder(const flce_beam_state* states, int64_t count,
                              const int64_t* parents, int64_t batch, int64_t beams,
                              int32_t* err_word, void* stream) {
  clear_error();
  if (count < 0 || (count > 0 && states == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "states are NULL, or their count is negative");
  if (batch < 0 || batch > 0x7fffffff)
    return fail(FLCE_ERR_INVALID_ARG, "batch %lld", (long long)batch);
  if (beams < 1 || beams > flce::kBeamMaxBeams)
    return fail(FLCE_ERR_UNSUPPORTED, "1 to %d beams are supported, not %lld",
                flce::kBeamMaxBeams, (long long)beams);
  if (batch > 0 && parents == nullptr) return fail(FLCE_ERR_INVALID_ARG, "parents is NULL");
  if (!aligned_to(parents, 8) || !aligned_to(err_word, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  const int max_width = beams > 32 ? 8 : 16;  // a thread holds one vector of each beam
  for (int64_t i = 0; i < count; ++i) {
    bool empty = false;
    const flce_status st = check_state(states[i], i, batch * beams, &empty);
    if (st != FLCE_OK) return st;
    if (empty) continue;
    int64_t vecs = states[i].run_bytes / std::min(max_width, width_of(states[i]));
    for (int d = 0; d < flce::kReorderDims; ++d) vecs *= states[i].size[d];
    // the kernel rounds a beam's vectors up to whole blocks in 32 bits
    if (vecs > 0xffffffffll / flce::kReorderBlock * flce::kReorderBlock ||
        ceil_div(vecs, flce::kReorderBlock) * batch > 0x7fffffffll)
      return fail(FLCE_ERR_UNSUPPORTED, "state %lld is too large", (long long)i);
  }
  if (batch > 0 && beams > 1 && count > 1) {
    const flce_status st = check_repeats(states, count);
    if (st != FLCE_OK) return st;
  }
  int sms = 0;
  const flce_status dev = check_device(&sms);
  if (dev != FLCE_OK || batch == 0) return dev;
  if (count <= flce::kReorderSmall)
    return reorder<flce::kReorderSmall>(states, count, parents, batch, beams, max_width, err_word,
                                        static_cast<cudaStream_t>(stream));
  return reorder<flce::kReorderLarge>(states, count, parents, batch, beams, max_width, err_word,
                                      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
