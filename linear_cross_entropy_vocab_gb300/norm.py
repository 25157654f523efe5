"""The root-mean-square norm with the residual's addition, before the head and between layers.

    s = x + residual
    y = s * weight / sqrt(mean(s^2) + eps)

``rms_norm`` gives y (and s) with their gradients, ``rms_norm_quantize`` gives y in 8-bit integers
as int8_linear takes them. The work runs in libflce.so (``flce_rms_norm``,
``flce_rms_norm_quantize``, ``flce_rms_norm_backward``).
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import abi
from ._autograd import refuse_gradient
from ._stream import on_device, raw_stream

__all__ = ["rms_norm", "rms_norm_quantize"]

_DTYPES = {torch.float32: abi.FLCE_F32, torch.bfloat16: abi.FLCE_BF16,
           torch.float16: abi.FLCE_F16}


def _check_inputs(x, weight, eps, residual) -> None:
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16 or float16")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., H) with H of at least 1")
    if weight is not None:
        if weight.shape != x.shape[-1:]:
            raise ValueError("weight must be (H,)")
        if weight.dtype != x.dtype and weight.dtype != torch.float32:
            raise TypeError(f"weight must be {x.dtype} or float32, not {weight.dtype}")
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, x {tuple(x.shape)}")
        if residual.dtype != x.dtype and residual.dtype != torch.float32:
            raise TypeError(f"residual must be {x.dtype} or float32, not {residual.dtype}")
    if not 1.1754944e-38 <= eps <= 3.4028234e38:
        raise ValueError("eps must be finite and at least 2^-126")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    for name, t in (("weight", weight), ("residual", residual)):
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, x on {x.device}")


def _rows(t: torch.Tensor):
    """``t`` [..., H] as rows of contiguous elements at one pitch: (tensor, pitch)."""
    h = t.shape[-1]
    if t.is_contiguous():
        return t, h
    if t.dim() == 2 and (t.stride(1) == 1 or h == 1) and t.stride(0) >= h:
        return t, t.stride(0)
    return t.contiguous(), h


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _prepare(x, weight, eps, residual):
    """x, residual and weight as rows, and the problem that they make."""
    x, x_pitch = _rows(x)
    h = x.shape[-1]
    code = sum_code = weight_code = _DTYPES[x.dtype]
    residual_pitch = h
    if residual is not None:
        residual, residual_pitch = _rows(residual)
        sum_code = _DTYPES[residual.dtype]
    if weight is not None:
        weight_code = _DTYPES[weight.dtype]
        if not weight.is_contiguous():
            weight = weight.contiguous()
    problem = abi.flce_norm_problem(x.numel() // h, h, x_pitch, residual_pitch, code, sum_code,
                                    weight_code, eps, 0)
    return x, weight, residual, problem


def _forward(x, weight, residual, problem, rstd):
    """(y, sum or None); fills ``rstd`` where one is given."""
    dense = torch.contiguous_format
    y = torch.empty_like(x, memory_format=dense)
    total = None if residual is None else torch.empty_like(residual, memory_format=dense)
    dev = x.device
    with on_device(dev):
        abi.flce_rms_norm(problem, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(),
                          _ptr(total), _ptr(rstd), raw_stream(dev))
    return y, total


class _RmsNorm(torch.autograd.Function):
    # The backward runs in autograd's own thread, where Python takes several times as long: what
    # it needs to know is worked out here.
    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        ctx.set_materialize_grads(False)
        x, weight, residual, problem = _prepare(x, weight, eps, residual)
        rstd = x.new_empty(problem.n, dtype=torch.float32)
        y, total = _forward(x, weight, residual, problem, rstd)
        if residual is None:
            ctx.save_for_backward(x, weight, rstd)
        else:
            ctx.save_for_backward(total, weight, rstd)
            problem.x_pitch = problem.h  # of the sum
        ctx.plan = problem, abi.flce_rms_norm_backward_workspace_size(problem)
        return y if residual is None else (y, total)

    @staticmethod
    def backward(ctx, grad_y, grad_sum=None):
        if torch.is_grad_enabled():  # a graph of the backward is asked for
            return _backward_once(ctx, grad_y, grad_sum)
        return _backward(ctx, grad_y, grad_sum)


def _backward(ctx, grad_y, grad_sum):
    total, weight, rstd = ctx.saved_tensors
    need_x, need_weight, _, need_residual = ctx.needs_input_grad
    problem, ws_bytes = ctx.plan
    wide = problem.sum_dtype != problem.dtype
    if grad_y is None:  # y is not used: the sum's gradient passes through
        if grad_sum is None:
            return None, None, None, None
        dtype = next(t for t, code in _DTYPES.items() if code == problem.dtype)
        return (grad_sum.to(dtype) if need_x else None,
                torch.zeros_like(weight) if need_weight else None, None,
                grad_sum if need_residual else None)
    dev = grad_y.device
    if not grad_y.is_contiguous():
        grad_y = grad_y.contiguous()
    if grad_sum is not None and not grad_sum.is_contiguous():
        grad_sum = grad_sum.contiguous()
    # in one type the gradients of x and of the residual are one tensor
    grad_x = torch.empty_like(grad_y) if need_x or (need_residual and not wide) else None
    grad_residual = torch.empty_like(total) if need_residual and wide else None
    grad_weight = torch.empty_like(weight) if need_weight else None
    ws = rstd.new_empty((ws_bytes + 3) // 4)
    with on_device(dev):
        abi.flce_rms_norm_backward(
            problem, grad_y.data_ptr(), _ptr(grad_sum), total.data_ptr(), _ptr(weight),
            rstd.data_ptr(), _ptr(grad_x), _ptr(grad_residual), _ptr(grad_weight), ws.data_ptr(),
            ws_bytes, raw_stream(dev))
    return (grad_x if need_x else None, grad_weight, None,
            grad_residual if wide else grad_x if need_residual else None)


_backward_once = once_differentiable(_backward)


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
             residual: Optional[torch.Tensor] = None):
    """y, or (y, s) where a ``residual`` is given: s = x + residual, y = s * weight /
    sqrt(mean(s^2) + eps) over the last dimension.

    x [..., H] is float32, bfloat16 or float16, and y has its type. ``residual`` is of x's shape
    and of its type or float32; s has the residual's type. ``weight`` [H] is of x's type or
    float32 (None: ones). y is computed from the unrounded sum, in 32 bits. ``eps`` is at least
    2^-126; H is at most 2^24.

    x, weight and residual get gradients from those of y and s; the backward reads s as it is
    stored, and gives the same bits in every run. It cannot be differentiated again.
    """
    eps = float(eps)
    _check_inputs(x, weight, eps, residual)
    if forward_ad._current_level < 0 and not (torch.is_grad_enabled() and (
            x.requires_grad or weight is not None and weight.requires_grad
            or residual is not None and residual.requires_grad)):
        x, weight, residual, problem = _prepare(x, weight, eps, residual)
        y, total = _forward(x, weight, residual, problem, None)
        return y if residual is None else (y, total)
    return _RmsNorm.apply(x, weight, eps, residual)


def rms_norm_quantize(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, *, residual: Optional[torch.Tensor] = None):
    """:func:`rms_norm` with y in 8-bit integers, as :func:`quantize_rows` makes them of the
    unrounded y: (q int8 [..., H], scale float32 [...]), or (q, scale, s) where a ``residual`` is
    given. q and scale go into :func:`int8_linear` as ``x`` and ``x_scale``. A row whose y holds
    a NaN or an infinity has scale NaN. It has no gradient: inputs that ask for one are refused.
    """
    eps = float(eps)
    _check_inputs(x, weight, eps, residual)
    refuse_gradient("rms_norm_quantize", ("x", "weight", "residual"), x, weight, residual)
    lead, h = x.shape[:-1], x.shape[-1]
    x, weight, residual, problem = _prepare(x, weight, eps, residual)
    dev = x.device
    total = None if residual is None else torch.empty_like(
        residual, memory_format=torch.contiguous_format)
    q_pitch = (h + 15) // 16 * 16
    q = torch.empty(problem.n, q_pitch, dtype=torch.int8, device=dev)
    scale = x.new_empty(lead, dtype=torch.float32)
    with on_device(dev):
        abi.flce_rms_norm_quantize(problem, x.data_ptr(), _ptr(residual), _ptr(weight),
                                   q.data_ptr(), q_pitch, scale.data_ptr(), _ptr(total),
                                   raw_stream(dev))
    if q_pitch != h:
        q = q[:, :h]
    if len(lead) != 1:
        q = q.unflatten(0, lead) if lead else q[0]
    return (q, scale) if residual is None else (q, scale, total)
