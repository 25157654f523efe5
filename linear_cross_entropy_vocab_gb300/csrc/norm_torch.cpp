// The root-mean-square norm as PyTorch operators over the C ABI: allocation of
// results, the current stream, and the autograd node. In C++ because these calls
// are shorter than Python's share of them: autograd runs a node in a thread of
// its own, where a node written in Python took 100 us more than this one.
//
// rms_norm calls the library itself for ordinary tensors. Where something
// listens to what is dispatched (tracing, torch.compile, fake tensors, a mode) it
// calls rms_norm_forward and rms_norm_backward through the dispatcher, which have
// a form for tensors without data.
#include <ATen/ATen.h>
#include <ATen/TensorSubclassLikeUtils.h>
#include <ATen/core/dispatch/Dispatcher.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/library.h>

#include <memory>
#include <optional>
#include <tuple>
#include <vector>

#include "flce.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

int32_t code_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat:
      return FLCE_F32;
    case at::kBFloat16:
      return FLCE_BF16;
    case at::kHalf:
      return FLCE_F16;
    default:
      TORCH_CHECK_TYPE(false, "unsupported dtype ", t.scalar_type());
  }
}

void check(flce_status status, const char* call) {
  TORCH_CHECK(status == FLCE_OK, call, ": ", flce_status_string(status), ": ", flce_last_error());
}

void* stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

const void* pointer(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* writable(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Shapes, for calls of the operators themselves: the Python layer has checked its
// own. The kernels go by x's shape (total's, backwards).
void check_like(const char* name, const Tensor& t, const Tensor& x) {
  TORCH_CHECK_VALUE(t.sym_sizes() == x.sym_sizes() && t.device() == x.device(), name,
                    " must be of x's shape and on its device");
}
void check_inputs(const Tensor& x, const std::optional<Tensor>& weight,
                  const std::optional<Tensor>& residual) {
  TORCH_CHECK_VALUE(x.dim() >= 1 && x.sym_sizes().back() >= 1,
                    "x must be (..., H) with H of at least 1");
  if (weight)
    TORCH_CHECK_VALUE(weight->dim() == 1 && weight->sym_sizes()[0] == x.sym_sizes().back() &&
                          weight->device() == x.device(),
                      "weight must be (H,) and on x's device");
  if (residual) check_like("residual", *residual, x);
}
void check_gradients(const Tensor& grad_y, const std::optional<Tensor>& grad_sum,
                     const Tensor& total, const std::optional<Tensor>& weight, const Tensor& rstd,
                     bool need_weight) {
  check_inputs(total, weight, grad_sum);
  check_like("grad_y", grad_y, total);
  TORCH_CHECK_VALUE(rstd.scalar_type() == at::kFloat && rstd.dim() == 1 && rstd.is_contiguous() &&
                        rstd.sym_numel() * total.sym_sizes().back() == total.sym_numel() &&
                        rstd.device() == total.device(),
                    "rstd must have a float32 for each row");
  TORCH_CHECK_VALUE(!grad_sum || grad_sum->scalar_type() == total.scalar_type(),
                    "grad_sum must be of total's type");
  TORCH_CHECK_VALUE(weight || !need_weight, "a gradient of no weight is asked for");
}

// t [..., H] as rows of contiguous elements at one pitch: as it is, where its
// leading dimensions are steps of one (a slice of wider rows), or a copy.
Tensor rows_of(const Tensor& t, int64_t& pitch) {
  const int64_t h = t.size(-1);
  pitch = h;
  if (t.is_contiguous()) return t;
  bool rows = t.dim() > 1 && (t.stride(-1) == 1 || h == 1) && t.stride(-2) >= h;
  for (int64_t i = 0; rows && i + 2 < t.dim(); ++i)
    rows = t.stride(i) == t.stride(i + 1) * t.size(i + 1);
  if (!rows) return t.contiguous();
  pitch = t.stride(-2);
  return t;
}

Tensor empty_as(const Tensor& shape_of, const Tensor& like) {
  return at::empty(shape_of.sizes(), like.options());
}

// Inputs as the library takes them.
struct Inputs {
  Tensor x, weight, residual;
  flce_norm_problem problem{};
};
Inputs prepare(const Tensor& x, const std::optional<Tensor>& weight, double eps,
               const std::optional<Tensor>& residual) {
  Inputs in;
  flce_norm_problem& p = in.problem;
  in.x = rows_of(x, p.x_pitch);
  p.h = x.size(-1);
  p.n = x.numel() / p.h;
  p.dtype = p.sum_dtype = p.weight_dtype = code_of(x);
  p.residual_pitch = p.h;
  p.eps = static_cast<float>(eps);
  if (residual) {
    in.residual = rows_of(*residual, p.residual_pitch);
    p.sum_dtype = code_of(in.residual);
  }
  if (weight) {
    in.weight = weight->contiguous();
    p.weight_dtype = code_of(in.weight);
  }
  return in;
}

// (y, sum or undefined); fills rstd where it is defined.
std::tuple<Tensor, Tensor> forward(const Inputs& in, const Tensor& rstd) {
  const c10::cuda::CUDAGuard guard(in.x.device());
  const Tensor y = empty_as(in.x, in.x);
  const Tensor sum = in.residual.defined() ? empty_as(in.x, in.residual) : Tensor();
  check(flce_rms_norm(&in.problem, pointer(in.x), pointer(in.residual), pointer(in.weight),
                      writable(y), writable(sum), static_cast<float*>(writable(rstd)),
                      stream_of(in.x)),
        "flce_rms_norm");
  return {y, sum};
}
Tensor empty_rstd(const Inputs& in) {
  return at::empty({in.problem.n}, in.x.options().dtype(at::kFloat));
}

struct Gradients {
  Tensor x, residual, weight;  // those that are asked for
};
// In one type the gradients of x and of the residual are one tensor, `x`.
Gradients gradients(const Tensor& upstream, const Tensor& upstream_sum, const Tensor& normalised,
                    const Tensor& gain, const Tensor& rstd, double eps, bool need_x,
                    bool need_residual, bool need_weight) {
  const c10::cuda::CUDAGuard guard(normalised.device());
  flce_norm_problem p{};
  const Tensor total = rows_of(normalised, p.x_pitch), grad_y = upstream.contiguous();
  const Tensor grad_sum = upstream_sum.defined() ? upstream_sum.contiguous() : upstream_sum;
  const Tensor weight = gain.defined() ? gain.contiguous() : gain;
  Gradients g;
  if (need_x) g.x = empty_as(total, grad_y);
  if (need_residual) g.residual = empty_as(total, total);
  if (need_weight) g.weight = at::empty_like(weight);
  p.h = total.size(-1);
  p.n = rstd.numel();
  p.residual_pitch = p.h;
  p.dtype = code_of(grad_y);
  p.sum_dtype = code_of(total);
  p.weight_dtype = weight.defined() ? code_of(weight) : p.dtype;
  p.eps = static_cast<float>(eps);
  const size_t bytes = flce_rms_norm_backward_workspace_size(&p);
  const Tensor workspace =
      at::empty({static_cast<int64_t>(bytes)}, total.options().dtype(at::kByte));
  check(flce_rms_norm_backward(&p, pointer(grad_y), pointer(grad_sum), pointer(total),
                               pointer(weight), static_cast<const float*>(pointer(rstd)),
                               writable(g.x), writable(g.residual), writable(g.weight),
                               writable(workspace), bytes, stream_of(total)),
        "flce_rms_norm_backward");
  return g;
}

// The same as operators without an autograd formula: (y, rstd) or (y, rstd, sum),
// and those gradients that are asked for, in the order of their flags.
std::vector<Tensor> rms_norm_forward(const Tensor& x, const std::optional<Tensor>& weight,
                                     double eps, const std::optional<Tensor>& residual) {
  check_inputs(x, weight, residual);
  const Inputs in = prepare(x, weight, eps, residual);
  const Tensor rstd = empty_rstd(in);
  auto [y, sum] = forward(in, rstd);
  if (residual) return {y, rstd, sum};
  return {y, rstd};
}
std::vector<Tensor> rms_norm_forward_meta(const Tensor& x, const std::optional<Tensor>& weight,
                                          double, const std::optional<Tensor>& residual) {
  check_inputs(x, weight, residual);
  const auto sizes = x.sym_sizes();
  const c10::SymInt n = x.sym_numel() / sizes.back();
  std::vector<Tensor> out{at::empty_symint(sizes, x.options()),
                          at::empty_symint({n}, x.options().dtype(at::kFloat))};
  if (residual) out.push_back(at::empty_symint(sizes, residual->options()));
  return out;
}

std::vector<Tensor> defined(const Gradients& g) {
  std::vector<Tensor> out;
  for (const Tensor& t : {g.x, g.residual, g.weight})
    if (t.defined()) out.push_back(t);
  return out;
}
std::vector<Tensor> rms_norm_backward(const Tensor& grad_y, const std::optional<Tensor>& grad_sum,
                                      const Tensor& total, const std::optional<Tensor>& weight,
                                      const Tensor& rstd, double eps, bool need_x,
                                      bool need_residual, bool need_weight) {
  check_gradients(grad_y, grad_sum, total, weight, rstd, need_weight);
  return defined(gradients(grad_y, grad_sum.value_or(Tensor()), total, weight.value_or(Tensor()),
                           rstd, eps, need_x, need_residual, need_weight));
}
std::vector<Tensor> rms_norm_backward_meta(const Tensor& grad_y,
                                           const std::optional<Tensor>& grad_sum,
                                           const Tensor& total,
                                           const std::optional<Tensor>& weight,
                                           const Tensor& rstd, double, bool need_x,
                                           bool need_residual, bool need_weight) {
  check_gradients(grad_y, grad_sum, total, weight, rstd, need_weight);
  Gradients g;
  if (need_x) g.x = at::empty_symint(total.sym_sizes(), grad_y.options());
  if (need_residual) g.residual = at::empty_symint(total.sym_sizes(), total.options());
  if (need_weight) g.weight = at::empty_symint(weight->sym_sizes(), weight->options());
  return defined(g);
}

// Whether a call on these tensors goes through the dispatcher.
template <class... Optional>
bool listened_to(const Tensor& t, const Optional&... others) {
  return at::isTensorSubclassLike(t) || ((others && at::isTensorSubclassLike(*others)) || ...);
}
template <class F>
auto operator_of(const char* name) {
  return c10::Dispatcher::singleton().findSchemaOrThrow(name, "").typed<F>();
}
std::vector<Tensor> dispatch_forward(const Tensor& x, const std::optional<Tensor>& weight,
                                     double eps, const std::optional<Tensor>& residual) {
  static const auto op = operator_of<decltype(rms_norm_forward)>("flce::rms_norm_forward");
  return op.call(x, weight, eps, residual);
}
Gradients dispatch_gradients(const Tensor& grad_y, const Tensor& grad_sum, const Tensor& total,
                             const Tensor& weight, const Tensor& rstd, double eps, bool need_x,
                             bool need_residual, bool need_weight) {
  static const auto op = operator_of<decltype(rms_norm_backward)>("flce::rms_norm_backward");
  const auto given = [](const Tensor& t) {
    return t.defined() ? std::optional<Tensor>(t) : std::nullopt;
  };
  const std::vector<Tensor> got = op.call(grad_y, given(grad_sum), total, given(weight), rstd, eps,
                                          need_x, need_residual, need_weight);
  Gradients g;
  size_t next = 0;
  if (need_x) g.x = got[next++];
  if (need_residual) g.residual = got[next++];
  if (need_weight) g.weight = got[next++];
  return g;
}

// Refuses a backward that is captured while an eager graph of the same leaves
// lives: their accumulators keep the stream that they were made on, autograd
// would make that one wait for the captured one, and where it is the default
// stream the capture is lost and the process with it.
void refuse_lost_capture() {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
  const auto node = torch::autograd::get_current_node();
  if (node == nullptr) return;
  for (size_t i = 0; i < node->num_outputs(); ++i) {
    torch::autograd::Node* const next = node->next_edge(i).function.get();
    if (dynamic_cast<torch::autograd::AccumulateGrad*>(next) == nullptr ||
        !node->task_should_compute_output(i))
      continue;
    const auto stream = next->stream();
    TORCH_CHECK(!stream || *stream != c10::cuda::getDefaultCUDAStream(stream->device_index()),
                "rms_norm: a captured backward needs leaves without another graph; drop the "
                "outputs of earlier calls on the default stream before the capture, or make "
                "them on the captured stream");
  }
}

class RmsNorm : public torch::autograd::Function<RmsNorm> {
 public:
  static variable_list forward(AutogradContext* ctx, const Tensor& x,
                               const std::optional<Tensor>& weight, double eps,
                               const std::optional<Tensor>& residual) {
    Tensor y, sum;
    ctx->set_materialize_grads(false);
    if (listened_to(x, weight, residual)) {
      const std::vector<Tensor> got = dispatch_forward(x, weight, eps, residual);
      y = got[0];
      if (residual) sum = got[2];
      ctx->save_for_backward({residual ? sum : x, weight.value_or(Tensor()), got[1]});
    } else {
      const Inputs in = prepare(x, weight, eps, residual);
      const Tensor rstd = empty_rstd(in);
      std::tie(y, sum) = ::forward(in, rstd);
      ctx->save_for_backward({residual ? sum : in.x, in.weight, rstd});
    }
    ctx->saved_data["eps"] = eps;
    ctx->saved_data["dtype"] = static_cast<int64_t>(x.scalar_type());
    if (residual) return {y, sum};
    return {y};
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &total = saved[0], &weight = saved[1], &rstd = saved[2];
    const bool plain = !at::isTensorSubclassLike(grads[0].defined() ? grads[0] : total);
    if (plain) refuse_lost_capture();
    // inputs that are tensors are counted
    size_t input = 0;
    const bool need_x = ctx->needs_input_grad(input++);
    const bool need_weight = weight.defined() && ctx->needs_input_grad(input++);
    const bool need_residual = grads.size() > 1 && ctx->needs_input_grad(input);
    const Tensor grad_y = grads[0], grad_sum = grads.size() > 1 ? grads[1] : Tensor();
    const auto dtype = static_cast<at::ScalarType>(ctx->saved_data["dtype"].toInt());
    const bool wide = total.scalar_type() != dtype;
    Tensor grad_x, grad_weight, grad_residual;
    if (!grad_y.defined()) {  // y is not used: the sum's gradient passes through
      if (grad_sum.defined()) {
        if (need_x) grad_x = grad_sum.to(dtype);
        if (need_weight) grad_weight = at::zeros_like(weight);
        if (need_residual) grad_residual = grad_sum;
      }
    } else {
      // in one type the gradients of x and of the residual are one tensor
      Gradients g = (plain ? gradients : dispatch_gradients)(
          grad_y, grad_sum, total, weight, rstd, ctx->saved_data["eps"].toDouble(),
          need_x || (need_residual && !wide), need_residual && wide, need_weight);
      grad_x = g.x;
      grad_residual = g.residual;
      grad_weight = g.weight;
      if (need_residual && !wide) grad_residual = grad_x;
      if (!need_x) grad_x = Tensor();
    }
    variable_list out{grad_x, grad_weight, Tensor(), grad_residual};
    if (at::GradMode::is_enabled()) {
      // a graph of the backward is asked for: its outputs refuse to go further
      variable_list some;
      for (const Tensor& t : out)
        if (t.defined()) some.push_back(t);
      const auto refuse = std::make_shared<torch::autograd::DelayedError>(
          "rms_norm cannot be differentiated twice", static_cast<int64_t>(some.size()));
      for (Tensor& t : some) t = t.detach().requires_grad_();
      some = (*refuse)(std::move(some));
      size_t next = 0;
      for (Tensor& t : out)
        if (t.defined()) t = some[next++];
    }
    return out;
  }
};

std::vector<Tensor> rms_norm(const Tensor& x, const std::optional<Tensor>& weight, double eps,
                             const std::optional<Tensor>& residual, bool differentiable) {
  check_inputs(x, weight, residual);
  if (differentiable) return RmsNorm::apply(x, weight, eps, residual);
  if (listened_to(x, weight, residual)) {
    const std::vector<Tensor> got = dispatch_forward(x, weight, eps, residual);
    if (residual) return {got[0], got[2]};
    return {got[0]};
  }
  const Inputs in = prepare(x, weight, eps, residual);
  auto [y, sum] = forward(in, Tensor());
  if (residual) return {y, sum};
  return {y};
}

std::vector<Tensor> rms_norm_quantize(const Tensor& x, const std::optional<Tensor>& weight,
                                      double eps, const std::optional<Tensor>& residual) {
  check_inputs(x, weight, residual);
  const Inputs in = prepare(x, weight, eps, residual);
  const flce_norm_problem& p = in.problem;
  const c10::cuda::CUDAGuard guard(x.device());
  // rows at multiples of 16 bytes, as the 8-bit layer reads them best
  const int64_t pitch = (p.h + 15) / 16 * 16;
  Tensor q = at::empty({p.n, pitch}, x.options().dtype(at::kChar));
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  const Tensor scale = at::empty(lead, x.options().dtype(at::kFloat));
  const Tensor sum = residual ? empty_as(in.x, in.residual) : Tensor();
  check(flce_rms_norm_quantize(&p, pointer(in.x), pointer(in.residual), pointer(in.weight),
                               static_cast<int8_t*>(writable(q)), pitch,
                               static_cast<float*>(writable(scale)), writable(sum), stream_of(x)),
        "flce_rms_norm_quantize");
  if (pitch != p.h) q = q.narrow(1, 0, p.h);
  if (lead.empty())
    q = q.select(0, 0);
  else if (lead.size() > 1)
    q = q.unflatten(0, lead);
  if (residual) return {q, scale, sum};
  return {q, scale};
}
std::vector<Tensor> rms_norm_quantize_meta(const Tensor& x, const std::optional<Tensor>& weight,
                                           double, const std::optional<Tensor>& residual) {
  check_inputs(x, weight, residual);
  const auto sizes = x.sym_sizes();
  std::vector<c10::SymInt> strides(sizes.size(), 1);
  c10::SymInt stride = (sizes.back() + 15) / 16 * 16;
  for (size_t i = sizes.size() - 1; i-- > 0; stride = stride * sizes[i]) strides[i] = stride;
  std::vector<Tensor> out{
      at::empty_strided_symint(sizes, strides, x.options().dtype(at::kChar)),
      at::empty_symint(sizes.slice(0, sizes.size() - 1), x.options().dtype(at::kFloat))};
  if (residual) out.push_back(at::empty_symint(sizes, residual->options()));
  return out;
}

}  // namespace

TORCH_LIBRARY(flce, m) {
  m.def("rms_norm(Tensor x, Tensor? weight, float eps, Tensor? residual, bool differentiable) "
        "-> Tensor[]",
        &rms_norm);
  m.def("rms_norm_forward(Tensor x, Tensor? weight, float eps, Tensor? residual) -> Tensor[]");
  m.def("rms_norm_backward(Tensor grad_y, Tensor? grad_sum, Tensor total, Tensor? weight, "
        "Tensor rstd, float eps, bool need_x, bool need_residual, bool need_weight) -> Tensor[]");
  m.def("rms_norm_quantize(Tensor x, Tensor? weight, float eps, Tensor? residual) -> Tensor[]");
}
TORCH_LIBRARY_IMPL(flce, CUDA, m) {
  m.impl("rms_norm_forward", &rms_norm_forward);
  m.impl("rms_norm_backward", &rms_norm_backward);
  m.impl("rms_norm_quantize", &rms_norm_quantize);
}
// None of these has a formula of its own: autograd is passed over, which its
// fallback would do in some microseconds.
TORCH_LIBRARY_IMPL(flce, Autograd, m) {
  m.impl("rms_norm_forward", torch::CppFunction::makeFallthrough());
  m.impl("rms_norm_backward", torch::CppFunction::makeFallthrough());
  m.impl("rms_norm_quantize", torch::CppFunction::makeFallthrough());
}
TORCH_LIBRARY_IMPL(flce, Meta, m) {
  m.impl("rms_norm_forward", &rms_norm_forward_meta);
  m.impl("rms_norm_backward", &rms_norm_backward_meta);
  m.impl("rms_norm_quantize", &rms_norm_quantize_meta);
}
