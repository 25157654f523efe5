// C entry points of the gradient norm and clip (include/flce.h): argument
// checks, the chunk tables, and the launch sequence. Nothing is allocated on
// the device and nothing waits for it.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>

#include "flce.h"
#include "grads_internal.h"
#include "host_common.h"

namespace {

using flce::GradEntry;
using flce::GradTable;
using flce::kGradTableLarge;
using flce::kGradTableMedium;
using flce::kGradTableSmall;
using namespace flce::host;

// Upper bound of the CTAs of one launch: the workspace holds one partial each.
constexpr int kMaxCtas = 1024;
// Chunks of 32 KB up to which the cluster of eight CTAs takes a clip by itself.
// On the device that is the shorter way up to 8 or 12 (two tensors in a graph,
// cluster against two launches: fp32 8 chunks 4.4 against 5.1 us, 16 5.2 / 5.1,
// 24 5.7 / 5.1, 64 8.3 / 5.3; bf16 8 5.8 / 6.4, 16 7.3 / 6.4, 24 8.8 / 6.4, 64
// 15.7 / 6.5). A call of its own, where a second launch costs the host 5 us,
// takes 16.5 us instead of 21.7 at any of these sizes. Between the two, 24 gives
// up at most 2.4 us in a graph for those 5.
constexpr uint32_t kClusterChunks = 24;

constexpr int64_t kMaxExtent = int64_t(1) << 46;

int64_t elem_size(int32_t dtype) { return dtype == FLCE_F32 ? 4 : 2; }
bool dtype_ok(int32_t d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }

flce_status check_side(const char* what, int64_t i, const void* p, const flce_grad& g,
                       int64_t pitch, int32_t dtype, bool written) {
  if (!dtype_ok(dtype))
    return fail(FLCE_ERR_INVALID_ARG, "gradient %lld: %s dtype %d is not an flce_dtype",
                (long long)i, what, dtype);
  if (p == nullptr)
    return fail(FLCE_ERR_INVALID_ARG, "gradient %lld: %s is NULL", (long long)i, what);
  if (!aligned_to(p, static_cast<size_t>(elem_size(dtype))))
    return fail(FLCE_ERR_UNSUPPORTED, "gradient %lld: %s is misaligned", (long long)i, what);
  if (pitch < 0 || pitch > kMaxExtent || (written && g.rows > 1 && pitch < g.cols))
    return fail(FLCE_ERR_INVALID_ARG, "gradient %lld: %s pitch %lld with %lld columns",
                (long long)i, what, (long long)pitch, (long long)g.cols);
  if (g.rows > 1 && pitch > 0 && g.rows > kMaxExtent / pitch)
    return fail(FLCE_ERR_INVALID_ARG, "gradient %lld: %s extent is too large", (long long)i, what);
  return FLCE_OK;
}

// The bytes that one side of a gradient spans.
struct Span {
  uintptr_t lo, hi;
  int64_t owner;
  int64_t row_bytes, pitch_bytes;  // pitch 0: one run
  bool written;
};

Span span_of(const void* p, const flce_grad& g, int64_t pitch, int32_t dtype, int64_t owner,
             bool written) {
  const int64_t es = elem_size(dtype);
  Span s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>(((g.rows - 1) * pitch + g.cols) * es);
  s.owner = owner;
  s.row_bytes = g.cols * es;
  s.pitch_bytes = g.rows > 1 && pitch > g.cols ? pitch * es : 0;
  if (s.pitch_bytes == 0) s.row_bytes = static_cast<int64_t>(s.hi - s.lo);
  s.written = written;
  return s;
}

// Whether two overlapping spans share no byte: rows of one pitch, side by side.
bool side_by_side(const Span& a, const Span& b) {
  const int64_t pitch = a.pitch_bytes != 0 ? a.pitch_bytes : b.pitch_bytes;
  if (pitch == 0) return false;
  if (a.pitch_bytes != 0 && b.pitch_bytes != 0 && a.pitch_bytes != b.pitch_bytes) return false;
  const int64_t off = static_cast<int64_t>((b.lo - a.lo) % static_cast<uintptr_t>(pitch));
  return off >= a.row_bytes && off + b.row_bytes <= pitch;
}

// No element that the clip writes is read or written for another place.
flce_status check_overlap(const flce_grad* g, int64_t count) {
  Span* const spans = new (std::nothrow) Span[2 * static_cast<size_t>(count)];
  Span* const open = new (std::nothrow) Span[2 * static_cast<size_t>(count)];
  flce_status st = FLCE_OK;
  if (spans == nullptr || open == nullptr) {
    st = fail(FLCE_ERR_INVALID_ARG, "no host memory for %lld gradients", (long long)count);
  } else {
    int64_t n = 0, n_open = 0;
    for (int64_t i = 0; i < count; ++i) {
      if (g[i].rows == 0 || g[i].cols == 0) continue;
      const bool in_place = g[i].src == g[i].dst && g[i].src_dtype == g[i].dst_dtype &&
                            (g[i].rows == 1 || g[i].src_pitch == g[i].dst_pitch);
      spans[n++] = span_of(g[i].dst, g[i], g[i].dst_pitch, g[i].dst_dtype, i, true);
      if (!in_place)
        spans[n++] = span_of(g[i].src, g[i], g[i].src_pitch, g[i].src_dtype, i, false);
    }
    std::sort(spans, spans + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    for (int64_t i = 0; i < n && st == FLCE_OK; ++i) {
      int64_t kept = 0;
      for (int64_t k = 0; k < n_open; ++k) {
        if (open[k].hi <= spans[i].lo) continue;
        if ((open[k].written || spans[i].written) && !side_by_side(open[k], spans[i])) {
          st = fail(FLCE_ERR_INVALID_ARG,
                    "gradients %lld and %lld overlap in memory that the clip writes",
                    (long long)open[k].owner, (long long)spans[i].owner);
          break;
        }
        open[kept++] = open[k];
      }
      n_open = kept;
      open[n_open++] = spans[i];
    }
  }
  delete[] spans;
  delete[] open;
  return st;
}

int norm_code(int32_t norm) {
  return norm == FLCE_NORM_INF ? 0 : norm == FLCE_NORM_L1 ? 1 : norm == FLCE_NORM_L2 ? 2 : -1;
}

flce_status check_args(const flce_grad* g, int64_t count, int32_t norm, const float* norm_out,
                       void* workspace, size_t workspace_bytes, bool clip) {
  if (count < 0 || (count > 0 && g == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "gradients are NULL, or their count is negative");
  if (norm_code(norm) < 0)
    return fail(FLCE_ERR_INVALID_ARG, "norm %d is not an flce_norm", norm);
  if (norm_out == nullptr) return fail(FLCE_ERR_INVALID_ARG, "norm_out is NULL");
  if (!aligned_to(norm_out, 4)) return fail(FLCE_ERR_UNSUPPORTED, "norm_out is misaligned");
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].rows < 0 || g[i].cols < 0 || g[i].cols > kMaxExtent ||
        (g[i].cols > 0 && g[i].rows > kMaxExtent / g[i].cols))
      return fail(FLCE_ERR_INVALID_ARG, "gradient %lld: %lld rows of %lld elements", (long long)i,
                  (long long)g[i].rows, (long long)g[i].cols);
    if (g[i].rows == 0 || g[i].cols == 0) continue;
    flce_status st = check_side("src", i, g[i].src, g[i], g[i].src_pitch, g[i].src_dtype, false);
    if (st == FLCE_OK && clip) {
      st = check_side("dst", i, g[i].dst, g[i], g[i].dst_pitch, g[i].dst_dtype, true);
      if (st == FLCE_OK && g[i].dst_dtype != g[i].src_dtype && g[i].dst_dtype != FLCE_F32)
        st = fail(FLCE_ERR_INVALID_ARG, "gradient %lld: dst has src's dtype or fp32",
                  (long long)i);
    }
    if (st != FLCE_OK) return st;
  }
  flce_status st = check_workspace(workspace, workspace_bytes, flce_grad_workspace_size(count));
  if (st == FLCE_OK && clip) st = check_overlap(g, count);
  return st;
}

// The gradients [*next, ...) that fit into one table; *next moves past them.
template <int CAP>
flce_status fill(GradTable<CAP>& tab, const flce_grad* g, int64_t count, int64_t* next,
                 bool clip) {
  uint64_t chunks = 0;
  int n = 0;
  tab.in_place = 1;
  for (; *next < count && n < CAP; ++*next) {
    const flce_grad& x = g[*next];
    const int64_t total = x.rows * x.cols;
    if (total == 0) continue;
    GradEntry& t = tab.t[n];
    const bool flat = x.rows == 1 || (x.src_pitch == x.cols && (!clip || x.dst_pitch == x.cols));
    t.src = x.src;
    t.dst = clip ? x.dst : nullptr;
    t.n = total;
    t.cols = flat ? total : x.cols;
    t.src_pitch = x.src_pitch;
    t.dst_pitch = x.dst_pitch;
    t.src_dtype = x.src_dtype;
    t.dst_dtype = x.dst_dtype;
    if (x.src != x.dst) tab.in_place = 0;
    tab.first[n++] = static_cast<uint32_t>(chunks);
    chunks += static_cast<uint64_t>(
        ceil_div(total, flce::kGradChunkBytes / elem_size(x.src_dtype)));
    if (chunks > 0x7fffffffull)
      return fail(FLCE_ERR_INVALID_ARG, "gradients of more than 2^31 chunks of %d bytes",
                  flce::kGradChunkBytes);
  }
  tab.count = n;
  tab.first[n] = static_cast<uint32_t>(chunks);
  return FLCE_OK;
}

template <int CAP>
flce_status run(const flce_grad* g, int64_t count, int p, bool clip, float max_norm, float eps,
                float* norm_out, double* partials, int sms, cudaStream_t s) {
  const int norm_ctas = std::min(kMaxCtas, flce::kGradNormCtasPerSm * sms);
  const int clip_ctas = std::min(kMaxCtas, flce::kGradClipCtasPerSm * sms);
  GradTable<CAP> tab;
  int n_partials = 0;
  for (int64_t next = 0; next < count;) {
    const flce_status st = fill(tab, g, count, &next, clip);
    if (st != FLCE_OK) return st;
    if (tab.count == 0) continue;
    if constexpr (CAP == kGradTableSmall) {
      if (clip && next == count && n_partials == 0 && tab.first[tab.count] <= kClusterChunks) {
        const cudaError_t e =
            flce::launch_grad_clip_cluster(tab, p, max_norm, eps, norm_out, s);
        return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "gradient clip kernel (cluster)");
      }
    }
    int n = 0;
    const cudaError_t e =
        flce::launch_grad_partials(tab, p, norm_ctas, partials + n_partials, &n, s);
    if (e != cudaSuccess) return cuda_fail(e, "gradient norm kernel");
    n_partials += n;
  }
  if (!clip || n_partials == 0) {
    const cudaError_t e = flce::launch_grad_norm(partials, n_partials, p, norm_out, s);
    return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "gradient norm reduction");
  }
  bool first = true;
  for (int64_t next = 0; next < count;) {
    const flce_status st = fill(tab, g, count, &next, clip);
    if (st != FLCE_OK) return st;
    if (tab.count == 0) continue;
    const cudaError_t e = flce::launch_grad_clip(tab, partials, n_partials, p, max_norm, eps,
                                                 norm_out, first, clip_ctas, s);
    if (e != cudaSuccess) return cuda_fail(e, "gradient clip kernel");
    first = false;
  }
  return FLCE_OK;
}

flce_status enter(const flce_grad* g, int64_t count, int32_t norm, bool clip, float max_norm,
                  float eps, float* norm_out, void* workspace, size_t workspace_bytes,
                  void* stream) {
  clear_error();
  flce_status st = check_args(g, count, norm, norm_out, workspace, workspace_bytes, clip);
  if (st != FLCE_OK) return st;
  if (clip && !(max_norm >= 0.0f && std::isfinite(max_norm)))
    return fail(FLCE_ERR_INVALID_ARG, "max_norm must be finite and not negative");
  if (clip && !(eps >= 0.0f && std::isfinite(eps)))
    return fail(FLCE_ERR_INVALID_ARG, "eps must be finite and not negative");
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK) return st;
  double* const partials = static_cast<double*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int p = norm_code(norm);
  if (count <= kGradTableSmall)
    return run<kGradTableSmall>(g, count, p, clip, max_norm, eps, norm_out, partials, sms, s);
  if (count <= kGradTableMedium)
    return run<kGradTableMedium>(g, count, p, clip, max_norm, eps, norm_out, partials, sms, s);
  return run<kGradTableLarge>(g, count, p, clip, max_norm, eps, norm_out, partials, sms, s);
}

}  // namespace

extern "C" {

size_t flce_grad_workspace_size(int64_t count) {
  if (count < 0) return 0;
  const int64_t launches = ceil_div(std::max<int64_t>(count, 1), kGradTableLarge);
  return static_cast<size_t>(launches) * kMaxCtas * sizeof(double);
}

flce_status flce_grad_norm(const flce_grad* grads, int64_t count, int32_t norm, float* norm_out,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return enter(grads, count, norm, false, 0.0f, 0.0f, norm_out, workspace, workspace_bytes,
               stream);
}

flce_status flce_grad_clip(const flce_grad* grads, int64_t count, int32_t norm, float max_norm,
                           float eps, float* norm_out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return enter(grads, count, norm, true, max_norm, eps, norm_out, workspace, workspace_bytes,
               stream);
}

}  // extern "C"
