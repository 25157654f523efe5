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

constexpr int64_t kMaxH = 131071;  // 128 * 128 * h stays below 2^31
constexpr int64_t kMaxRows = 0x7fffffff;

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
  return FLCE_OK;
}

struct QPlan {
  size_t q, scale, total;
  int64_t q_pitch;
};

QPlan plan_qlinear(const flce_qproblem* p) {
  QPlan q{};
  q.q_pitch = (p->h + 15) / 16 * 16;
  if (p->x_dtype != FLCE_Q_I8) {
    q.scale = align_256(static_cast<size_t>(p->n) * static_cast<size_t>(q.q_pitch));
    q.total = q.scale + align_256(static_cast<size_t>(p->n) * 4);
  }
  return q;
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
  const flce::QuantParams k{x, n, h, x_pitch, q, q_pitch, scale};
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
  st = check_workspace(workspace, workspace_bytes, plan.total);
  if (st != FLCE_OK) return st;
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || p->n == 0 || p->v == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  flce::QLinearParams k{};
  if (dynamic) {
    const flce::QuantParams q{x, p->n, p->h, p->x_pitch, reinterpret_cast<int8_t*>(ws + plan.q),
                              plan.q_pitch, reinterpret_cast<float*>(ws + plan.scale)};
    const cudaError_t e = flce::launch_quantize_rows(q, p->x_dtype, s);
    if (e != cudaSuccess) return cuda_fail(e, "row quantisation kernel");
    k.x = q.q;
    k.x_scale = q.scale;
    k.x_pitch = q.q_pitch;
  } else {
    k.x = static_cast<const int8_t*>(x);
    k.x_scale = x_scale;
    k.x_pitch = p->x_pitch;
  }
  k.weight = weight;
  k.weight_scale = weight_scale;
  k.bias = bias;
  k.out = out;
  k.n = p->n;
  k.h = p->h;
  k.v = p->v;
  k.weight_pitch = p->weight_pitch;
  k.out_pitch = p->out_pitch;
  k.out_dtype = p->out_dtype;
  k.bias_dtype = p->bias_dtype;
  k.xf.scale = p->logit_scale;
  k.xf.has_cap = p->softcap > 0.0f ? 1 : 0;
  k.xf.softcap = k.xf.has_cap ? p->softcap : 1.0f;
  k.xf.inv_softcap = 1.0f / k.xf.softcap;
  const cudaError_t e = flce::launch_qlinear_simple(k, s);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "8-bit linear kernel");
}

}  // extern "C"
