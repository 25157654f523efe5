// C entry points of the root-mean-square norm (include/flce.h): argument
// checks, workspace and launches. Nothing is allocated on the device and
// nothing waits for it.
#include <cfloat>
#include <cmath>

#include "flce.h"
#include "host_common.h"
#include "norm_internal.h"

namespace {

using namespace flce::host;

constexpr int64_t kMaxRows = 0x7fffff00;
constexpr int64_t kMaxH = int64_t(1) << 24;

bool float_type(int32_t d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }
size_t size_of(int32_t d) { return d == FLCE_F32 ? 4 : 2; }

flce_status check_problem(const flce_norm_problem* p) {
  if (p == nullptr) return fail(FLCE_ERR_INVALID_ARG, "problem is NULL");
  if (p->n < 0 || p->n > kMaxRows) return fail(FLCE_ERR_INVALID_ARG, "n = %lld", (long long)p->n);
  if (p->h < 1 || p->h > kMaxH)
    return fail(FLCE_ERR_UNSUPPORTED, "h must be in 1 to %lld, not %lld", (long long)kMaxH,
                (long long)p->h);
  if (!float_type(p->dtype))
    return fail(FLCE_ERR_INVALID_ARG, "dtype %d is not an flce_dtype", p->dtype);
  if ((p->sum_dtype != p->dtype && p->sum_dtype != FLCE_F32) ||
      (p->weight_dtype != p->dtype && p->weight_dtype != FLCE_F32))
    return fail(FLCE_ERR_INVALID_ARG, "sum_dtype and weight_dtype must be dtype or FLCE_F32");
  if (p->x_pitch < p->h || p->residual_pitch < p->h)
    return fail(FLCE_ERR_INVALID_ARG, "a pitch is smaller than its rows");
  if (p->x_pitch > (int64_t(1) << 40) || p->residual_pitch > (int64_t(1) << 40))
    return fail(FLCE_ERR_INVALID_ARG, "a pitch is too large");
  if (!(p->eps >= FLT_MIN) || !std::isfinite(p->eps))
    return fail(FLCE_ERR_INVALID_ARG, "eps must be finite and at least %g", (double)FLT_MIN);
  if (p->reserved != 0) return fail(FLCE_ERR_INVALID_ARG, "reserved is not 0");
  return FLCE_OK;
}

// The parts of a forward call that both outputs share.
flce_status check_forward(const flce_norm_problem* p, const void* x, const void* residual,
                          const void* weight, const void* sum) {
  if (p->n > 0 && x == nullptr) return fail(FLCE_ERR_INVALID_ARG, "x is required");
  if (p->n > 0 && (residual == nullptr) != (sum == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "sum_out goes with residual, and only with it");
  if (!aligned_to(x, size_of(p->dtype)) || !aligned_to(residual, size_of(p->sum_dtype)) ||
      !aligned_to(sum, size_of(p->sum_dtype)) || !aligned_to(weight, size_of(p->weight_dtype)))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  return FLCE_OK;
}

flce::NormParams forward_params(const flce_norm_problem* p, const void* x, const void* residual,
                                const void* weight, void* sum) {
  flce::NormParams k{};
  k.x = x;
  k.residual = residual;
  k.weight = weight;
  k.sum = sum;
  k.n = p->n;
  k.h = p->h;
  k.x_pitch = p->x_pitch;
  k.residual_pitch = p->residual_pitch;
  k.wide = p->sum_dtype == FLCE_F32 ? 1 : 0;
  k.weight_wide = p->weight_dtype == FLCE_F32 ? 1 : 0;
  k.eps = p->eps;
  return k;
}

// The SMs that a workspace is planned for: parts of grad_weight are never more
// than this many times the CTAs of an SM.
constexpr int kPlanSms = 160;

struct BwdPlan {
  size_t partial, along, total;
};
BwdPlan plan_backward(const flce_norm_problem* p) {
  BwdPlan b{};
  const int64_t parts = flce::norm_bwd_parts(p->n, p->h, kPlanSms);
  b.partial = 0;
  b.along = align_256(static_cast<size_t>(parts) * static_cast<size_t>(p->h) * 4);
  b.total = b.along +
            (p->h > flce::kNormBwdMaxH ? align_256(static_cast<size_t>(p->n) * 4) : 0);
  return b;
}

}  // namespace

extern "C" {

flce_status flce_rms_norm(const flce_norm_problem* p, const void* x, const void* residual,
                          const void* weight, void* y, void* sum_out, float* rstd_out,
                          void* stream) {
  clear_error();
  flce_status st = check_problem(p);
  if (st != FLCE_OK) return st;
  st = check_forward(p, x, residual, weight, sum_out);
  if (st != FLCE_OK) return st;
  if (p->n > 0 && y == nullptr) return fail(FLCE_ERR_INVALID_ARG, "y is required");
  if (!aligned_to(y, size_of(p->dtype)) || !aligned_to(rstd_out, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || p->n == 0) return st;
  flce::NormParams k = forward_params(p, x, residual, weight, sum_out);
  k.y = y;
  k.sms = sms;
  k.rstd = rstd_out;
  const cudaError_t e = flce::launch_rms_norm(k, p->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "norm kernel");
}

flce_status flce_rms_norm_quantize(const flce_norm_problem* p, const void* x,
                                   const void* residual, const void* weight, int8_t* q,
                                   int64_t q_pitch, float* scale, void* sum_out, void* stream) {
  clear_error();
  flce_status st = check_problem(p);
  if (st != FLCE_OK) return st;
  st = check_forward(p, x, residual, weight, sum_out);
  if (st != FLCE_OK) return st;
  if (q_pitch < p->h || q_pitch > (int64_t(1) << 40))
    return fail(FLCE_ERR_INVALID_ARG, "q_pitch = %lld", (long long)q_pitch);
  if (p->n > 0 && (q == nullptr || scale == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "q and scale are required");
  if (!aligned_to(scale, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || p->n == 0) return st;
  flce::NormParams k = forward_params(p, x, residual, weight, sum_out);
  k.q = q;
  k.sms = sms;
  k.q_pitch = q_pitch;
  k.scale = scale;
  const cudaError_t e = flce::launch_rms_norm_q(k, p->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "norm and row quantisation kernel");
}

size_t flce_rms_norm_backward_workspace_size(const flce_norm_problem* p) {
  if (check_problem(p) != FLCE_OK) return 0;
  return plan_backward(p).total;
}

flce_status flce_rms_norm_backward(const flce_norm_problem* p, const void* grad_y,
                                   const void* grad_sum, const void* total, const void* weight,
                                   const float* rstd, void* grad_x, void* grad_residual,
                                   void* grad_weight, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  clear_error();
  flce_status st = check_problem(p);
  if (st != FLCE_OK) return st;
  if (p->n > 0 && (grad_y == nullptr || total == nullptr || rstd == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "grad_y, total and rstd are required");
  if (grad_weight != nullptr && weight == nullptr)
    return fail(FLCE_ERR_INVALID_ARG, "grad_weight without a weight");
  if (grad_residual != nullptr && p->sum_dtype != FLCE_F32)
    return fail(FLCE_ERR_INVALID_ARG,
                "grad_residual is for an fp32 sum: in one type it is grad_x");
  const size_t e = size_of(p->dtype), ew = size_of(p->sum_dtype);
  if (!aligned_to(grad_y, e) || !aligned_to(grad_sum, ew) || !aligned_to(total, ew) ||
      !aligned_to(weight, size_of(p->weight_dtype)) || !aligned_to(rstd, 4) ||
      !aligned_to(grad_x, e) || !aligned_to(grad_residual, 4) ||
      !aligned_to(grad_weight, size_of(p->weight_dtype)))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  const BwdPlan plan = plan_backward(p);
  st = check_workspace(workspace, workspace_bytes, plan.total);
  if (st != FLCE_OK) return st;
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->n == 0) {
    if (grad_weight == nullptr) return FLCE_OK;
    const cudaError_t err =
        cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(p->h) * size_of(p->weight_dtype), s);
    return err == cudaSuccess ? FLCE_OK : cuda_fail(err, "zeroing grad_weight");
  }
  flce::NormBwdParams k{};
  k.grad_y = grad_y;
  k.grad_sum = grad_sum;
  k.total = total;
  k.weight = weight;
  k.rstd = rstd;
  k.grad_x = grad_x;
  k.grad_residual = grad_residual;
  k.grad_weight = grad_weight;
  k.partial = static_cast<float*>(workspace);
  k.along = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.along);
  k.n = p->n;
  k.h = p->h;
  k.total_pitch = p->x_pitch;
  k.wide = p->sum_dtype == FLCE_F32 ? 1 : 0;
  k.weight_wide = p->weight_dtype == FLCE_F32 ? 1 : 0;
  const cudaError_t err = flce::launch_rms_norm_bwd(k, p->dtype, sms < kPlanSms ? sms : kPlanSms, s);
  return err == cudaSuccess ? FLCE_OK : cuda_fail(err, "norm backward kernels");
}

}  // extern "C"
