// C entry points of the 8-bit integer operators (include/flce.h): argument
// checks, workspace and launches. Nothing is allocated on the device and
// nothing waits for it.
#include <algorithm>
#include <cmath>

#include "flce.h"
#include "host_common.h"
#include "int8_internal.h"

namespace {

using namespace flce::host;

// Keeps the sums of h products below 2^31, where the last place of the 32-bit
// accumulator, which each step of 16 products may lose beyond 2^24, is at most
// 128.
constexpr int64_t kMaxH = 131071;
constexpr int64_t kMaxRows = 0x7fffff00;  // a tile may end 255 rows further

bool float_type(int32_t d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }
size_t size_of(int32_t d) { return d == FLCE_F32 ? 4 : d == FLCE_Q_I8 ? 1 : 2; }

flce_status check_qproblem(const flce_qproblem* p) {
  if (p == nullptr) return fail(FLCE_ERR_INVALID_ARG, "problem is NULL");
  if (p->n < 0 || p->n > kMaxRows || p->v < 0 || p->v > kMaxRows)
    return fail(FLCE_ERR_INVALID_ARG, "n = %lld, v = %lld", (long long)p->n, (long long)p->v);
  if (p->h < 1 || p->h > kMaxH)
    return fail(FLCE_ERR_UNSUPPORTED, "h must be in 1 to %lld, not %lld", (long long)kMaxH,
                (long long)p->h);
  if (!float_type(p->x_dtype) && p->x_dtype != FLCE_Q_I8)
    return fail(FLCE_ERR_INVALID_ARG, "x_dtype %d", p->x_dtype);
  if (!float_type(p->out_dtype)) return fail(FLCE_ERR_INVALID_ARG, "out_dtype %d", p->out_dtype);
  if (p->has_bias != 0 && p->has_bias != 1)
    return fail(FLCE_ERR_INVALID_ARG, "has_bias must be 0 or 1");
  if (p->has_bias && !float_type(p->bias_dtype))
    return fail(FLCE_ERR_INVALID_ARG, "bias_dtype %d", p->bias_dtype);
  if (p->x_pitch < p->h || p->weight_pitch < p->h || p->out_pitch < p->v)
    return fail(FLCE_ERR_INVALID_ARG, "a pitch is smaller than its rows");
  if (!std::isfinite(p->logit_scale) || !std::isfinite(p->softcap))
    return fail(FLCE_ERR_INVALID_ARG, "logit_scale and softcap must be finite");
  if (p->softcap > 0.0f && !std::isfinite(1.0f / p->softcap))
    return fail(FLCE_ERR_INVALID_ARG, "softcap is too small to divide by");
  if ((p->flags & ~FLCE_Q_LAY_OUT_WEIGHT) != 0 || p->reserved != 0)
    return fail(FLCE_ERR_INVALID_ARG, "unknown flags, or reserved is not 0");
  return FLCE_OK;
}

// Rows of x that a tile takes, and whether CTA pairs take it. A tile of up to
// 128 rows runs on single CTAs, whose accumulator drains behind the next
// tile's products (128 rows of the Llama-3 head: 114 us, 126 by pairs; 16 rows
// alike); more rows run on pairs, which share the tile of x, in the fewest
// tiles of at most 256 rows, each as small as that many allow.
struct QTile {
  int cg;
  int64_t nt, n_tiles;
};

QTile tile_of(int64_t n) {
  QTile t;
  t.cg = n <= 128 ? 1 : 2;
  t.n_tiles = ceil_div(n, t.cg == 1 ? 128 : 256);
  const int64_t step = 16 * t.cg;
  t.nt = ceil_div(ceil_div(n, t.n_tiles), step) * step;
  t.n_tiles = ceil_div(n, t.nt);
  return t;
}

// Bytes of widened x that go through the whole weight together: they stay in
// L2 while the weight streams. 8192 rows of the Llama-3 head under the power
// cap: 4.73 ms with bands of 16 tiles (32 MB), 4.77 with 8, 4.91 with 4, which
// read the weight more often, and 4.97 without bands (32 tiles).
constexpr int64_t kBandBytes = int64_t(32) << 20;

struct QPlan {
  size_t wide, scale, weight, total;
  int64_t wide_pitch, weight_pitch;
  bool align;  // the weight is laid out in the workspace first
};

// TMA reads rows that start at multiples of 16 bytes: others are laid out
// anew, which reads and writes the weight once more.
QPlan plan_qlinear(const flce_qproblem* p) {
  QPlan q{};
  const bool align = p->weight_pitch % 16 != 0 || (p->flags & FLCE_Q_LAY_OUT_WEIGHT) != 0;
  q.align = align;
  q.wide_pitch = ceil_div(p->h, 64) * 64;
  q.scale = align_256(static_cast<size_t>(p->n) * static_cast<size_t>(q.wide_pitch) * 2);
  q.weight = q.scale + align_256(static_cast<size_t>(p->n) * 4);
  q.weight_pitch = align ? ceil_div(p->h, 16) * 16 : p->weight_pitch;
  q.total = q.weight +
            (align ? align_256(static_cast<size_t>(p->v) * static_cast<size_t>(q.weight_pitch))
                   : 0);
  return q;
}

bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t inner,
              int64_t outer, int64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) {
    fail(FLCE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fail(FLCE_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d (%lld x %lld, pitch %lld)",
         static_cast<int>(r), (long long)inner, (long long)outer, (long long)pitch_bytes);
    return false;
  }
  return true;
}

}  // namespace

extern "C" {

flce_status flce_quantize_rows(const void* x, int32_t dtype, int64_t n, int64_t h,
                               int64_t x_pitch, int8_t* q, int64_t q_pitch, float* scale,
                               void* stream) {
  clear_error();
  if (!float_type(dtype)) return fail(FLCE_ERR_INVALID_ARG, "dtype %d is not an flce_dtype", dtype);
  if (n < 0 || n > kMaxRows || h < 1 || h > (int64_t(1) << 40))
    return fail(FLCE_ERR_INVALID_ARG, "n = %lld, h = %lld", (long long)n, (long long)h);
  if (x_pitch < h || q_pitch < h)
    return fail(FLCE_ERR_INVALID_ARG, "a pitch is smaller than its rows");
  if (n > 0 && (x == nullptr || q == nullptr || scale == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "x, q and scale are required");
  if (!aligned_to(x, size_of(dtype)) || !aligned_to(scale, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  int sms = 0;
  const flce_status st = check_device(&sms);
  if (st != FLCE_OK || n == 0) return st;
  flce::QuantParams k{};
  k.x = x;
  k.n = n;
  k.h = h;
  k.x_pitch = x_pitch;
  k.q = q;
  k.q_pitch = q_pitch;
  k.scale = scale;
  const cudaError_t e = flce::launch_quantize_rows(k, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "row quantisation kernel");
}

size_t flce_qlinear_workspace_size(const flce_qproblem* p) {
  if (check_qproblem(p) != FLCE_OK) return 0;
  return plan_qlinear(p).total;
}

flce_status flce_qlinear(const flce_qproblem* p, const void* x, const float* x_scale,
                         const int8_t* weight, const float* weight_scale, const void* bias,
                         void* out, int32_t* err_word, void* workspace, size_t workspace_bytes,
                         void* stream) {
  clear_error();
  flce_status st = check_qproblem(p);
  if (st != FLCE_OK) return st;
  const bool dynamic = p->x_dtype != FLCE_Q_I8;
  if (p->n > 0 && p->v > 0) {
    if (x == nullptr || weight == nullptr || weight_scale == nullptr || out == nullptr)
      return fail(FLCE_ERR_INVALID_ARG, "x, weight, weight_scale and out are required");
    if (dynamic != (x_scale == nullptr))
      return fail(FLCE_ERR_INVALID_ARG, "x_scale goes with FLCE_Q_I8, and only with it");
    if ((p->has_bias != 0) != (bias != nullptr))
      return fail(FLCE_ERR_INVALID_ARG, "bias and has_bias differ");
    if (!aligned_to(x, size_of(p->x_dtype)) || !aligned_to(x_scale, 4) ||
        !aligned_to(weight_scale, 4) || !aligned_to(out, size_of(p->out_dtype)) ||
        !aligned_to(bias, p->has_bias ? size_of(p->bias_dtype) : 1) || !aligned_to(err_word, 4))
      return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  }
  const QPlan plan = plan_qlinear(p);
  if (p->n > 0 && p->v > 0 && !plan.align && !aligned_to(weight, 16))
    return fail(FLCE_ERR_UNSUPPORTED,
                "weight does not start at a multiple of 16 bytes (FLCE_Q_LAY_OUT_WEIGHT)");
  st = check_workspace(workspace, workspace_bytes, plan.total);
  if (st != FLCE_OK) return st;
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || p->n == 0 || p->v == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  cudaError_t e;
  if (plan.align) {
    int8_t* const laid = reinterpret_cast<int8_t*>(ws + plan.weight);
    e = flce::launch_align_rows(weight, p->v, p->h, p->weight_pitch, laid, plan.weight_pitch, s);
    if (e != cudaSuccess) return cuda_fail(e, "weight layout kernel");
    weight = laid;
  }
  flce::QuantParams q{};
  q.x = x;
  q.n = p->n;
  q.h = p->h;
  q.x_pitch = p->x_pitch;
  q.wide = ws + plan.wide;
  q.wide_pitch = plan.wide_pitch;
  q.scale = reinterpret_cast<float*>(ws + plan.scale);
  e = flce::launch_widen_rows(q, p->x_dtype, s);
  if (e != cudaSuccess) return cuda_fail(e, "row quantisation kernel");

  const QTile tile = tile_of(p->n);
  flce::QLinearTcParams k{};
  if (!make_map(&k.w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, weight, p->h, p->v, plan.weight_pitch,
                128, 128) ||
      !make_map(&k.x_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q.wide, plan.wide_pitch, p->n,
                plan.wide_pitch * 2, 64, static_cast<uint32_t>(tile.nt / tile.cg)))
    return FLCE_ERR_CUDA;
  const int64_t v_tiles = ceil_div(p->v, 128 * tile.cg);
  if (v_tiles * tile.n_tiles > 0x7fffffff)
    return fail(FLCE_ERR_UNSUPPORTED, "more than 2^31 output tiles");
  k.x_scale = dynamic ? q.scale : x_scale;
  k.weight_scale = weight_scale;
  k.bias = bias;
  k.out = out;
  k.n = p->n;
  k.v = p->v;
  k.out_pitch = p->out_pitch;
  k.bias_dtype = p->bias_dtype;
  k.nt = static_cast<int32_t>(tile.nt);
  k.n_tiles = static_cast<int32_t>(tile.n_tiles);
  k.v_tiles = static_cast<int32_t>(v_tiles);
  k.band = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>(tile.n_tiles, kBandBytes / (tile.nt * plan.wide_pitch * 2))));
  k.k_blocks = static_cast<int32_t>(ceil_div(p->h, 64));
  k.err_word = err_word;
  k.xf.scale = p->logit_scale;
  k.xf.has_cap = p->softcap > 0.0f ? 1 : 0;
  k.xf.softcap = k.xf.has_cap ? p->softcap : 1.0f;
  k.xf.inv_softcap = 1.0f / k.xf.softcap;
  e = flce::launch_qlinear_tc(k, tile.cg, p->out_dtype, sms, s);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "8-bit linear kernel");
}

}  // extern "C"
