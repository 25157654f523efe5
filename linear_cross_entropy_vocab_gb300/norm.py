"""The root-mean-square norm with the residual's addition, before the head and between layers.

    s = x + residual
    y = s * weight / sqrt(mean(s^2) + eps)

``rms_norm`` gives y (and s) with their gradients, ``rms_norm_quantize`` gives y in 8-bit integers
as int8_linear takes them. The work runs in libflce.so (``flce_rms_norm``,
``flce_rms_norm_quantize``, ``flce_rms_norm_backward``), called by the operators of
libflce_torch.so.
"""
from __future__ import annotations

import os
from typing import Optional

import torch
from torch.autograd import forward_ad

from . import abi, native_build
from ._autograd import refuse_gradient

__all__ = ["rms_norm", "rms_norm_quantize"]

_DTYPES = (torch.float32, torch.bfloat16, torch.float16)
_MAX_H = 1 << 24


def _check_inputs(x, weight, eps, residual) -> None:
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16 or float16")
    if x.dim() < 1 or not 1 <= x.shape[-1] <= _MAX_H:
        raise ValueError("x must be (..., H) with H of at least 1 and at most 2^24")
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


_ops = None


def _operators():
    """torch.ops.flce, which libflce_torch.so registers. Raises if it is missing."""
    global _ops
    if _ops is None:
        abi.load()
        path = native_build.TORCH_LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -m linear_cross_entropy_vocab_gb300.native_build)")
        why = native_build.torch_mismatch()
        if why is not None:
            raise RuntimeError(
                f"{path} is of another PyTorch ({why}): build the CUDA library again "
                "(python -m linear_cross_entropy_vocab_gb300.native_build)")
        torch.ops.load_library(path)
        _ops = torch.ops.flce.rms_norm.default, torch.ops.flce.rms_norm_quantize.default
    return _ops


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
             residual: Optional[torch.Tensor] = None):
    """y, or (y, s) where a ``residual`` is given: s = x + residual, y = s * weight /
    sqrt(mean(s^2) + eps) over the last dimension.

    x [..., H] is float32, bfloat16 or float16, and y has its type. ``residual`` is of x's shape
    and of its type or float32; s has the residual's type. ``weight`` [H] is of x's type or
    float32 (None: ones). y is computed from the unrounded sum, in 32 bits; its last bit may
    depend on whether rows lie at 16-byte boundaries. ``eps`` is at least 2^-126; H is at most 2^24.

    x, weight and residual get gradients from those of y and s; the backward reads s as it is
    stored, and gives the same bits in every run. Where s leaves float16's range it is stored as an
    infinity, and the row's gradients and the weight's of that column are not finite, although y is:
    a float32 residual keeps them. It cannot be differentiated again. torch.compile and other tracers see ``flce::rms_norm_forward``
    and ``flce::rms_norm_backward``.
    """
    eps = float(eps)
    _check_inputs(x, weight, eps, residual)
    differentiable = forward_ad._current_level >= 0 or torch.is_grad_enabled() and (
        x.requires_grad or weight is not None and weight.requires_grad
        or residual is not None and residual.requires_grad)
    got = _operators()[0](x, weight, eps, residual, differentiable)
    return got[0] if residual is None else tuple(got)


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
    return tuple(_operators()[1](x, weight, eps, residual))
