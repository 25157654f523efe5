"""Rows in 8-bit integers with a scale each, and the linear layer on them: a head for answering,
at half the memory and half the memory traffic of a 16-bit one.

    scale[i] = max |x[i]| * (1/127),   q[i] = round(x[i] / scale[i])
    u = logit_scale * (scale[:, None] * weight_scale * (q @ weight.T) + bias)
    out = softcap * tanh(u / softcap)   if softcap, else u

The work runs in libflce.so (``flce_quantize_rows``, ``flce_qlinear``).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import abi
from ._autograd import refuse_gradient
from ._stream import on_device, raw_stream

__all__ = ["quantize_rows", "int8_linear"]

_DTYPES = {torch.float32: abi.FLCE_F32, torch.bfloat16: abi.FLCE_BF16,
           torch.float16: abi.FLCE_F16}


def _rows(x: torch.Tensor):
    """``x`` [..., H] as rows of contiguous elements at one pitch: (tensor, rows, pitch)."""
    h = x.shape[-1]
    n = x.numel() // h
    if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= h:
        return x, n, x.stride(0)
    x = x.contiguous()
    return x, n, h


def quantize_rows(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [..., H] (float32, bfloat16 or float16) -> (q int8 [..., H], scale float32 [...]), with
    x close to q * scale. Halves round to even; a row of zeros has scale 0, and a row that holds
    a NaN or an infinity has scale NaN. q's rows start at multiples of 16 bytes, as int8_linear
    reads them best: where H is no multiple of 16, q is a view of wider rows. It has no gradient:
    an x that asks for one is refused."""
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16 or float16")
    refuse_gradient("quantize_rows", ("x",), x)
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., H) with H of at least 1")
    lead, h = x.shape[:-1], x.shape[-1]
    x, n, pitch = _rows(x)
    q_pitch = (h + 15) // 16 * 16
    q = torch.empty(n, q_pitch, dtype=torch.int8, device=x.device)
    scale = torch.empty(n, dtype=torch.float32, device=x.device)
    with on_device(x.device):
        stream = raw_stream(x.device)
        abi.flce_quantize_rows(x.data_ptr(), code, n, h, pitch, q.data_ptr(), q_pitch,
                               scale.data_ptr(), stream)
    if q_pitch != h:
        q = q[:, :h]
    if len(lead) == 1:
        return q, scale
    return q.unflatten(0, lead) if lead else q[0], scale.reshape(lead)


def int8_linear(x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, *, x_scale: Optional[torch.Tensor] = None,
                logit_scale: float = 1.0, softcap: Optional[float] = None,
                out_dtype: Optional[torch.dtype] = None,
                err_word: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Logits [..., V] of x [..., H] against weight [V, H] (int8, weight_scale [V] float32; H at
    most 131071).

    x is float32, bfloat16 or float16 and is quantised row by row within the call, or int8 with
    ``x_scale`` [...] float32 from :func:`quantize_rows`. ``bias`` [V] is a float tensor.
    ``logit_scale`` and ``softcap`` are the losses'. The result is ``out_dtype``, by default x's
    type (float32 for int8). It has no gradient: inputs that ask for one are refused.
    Weight rows that start at multiples of 16 bytes, as quantize_rows makes them, are read where
    they are; others are laid out anew in every call.
    """
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be (..., H) and weight (V, H)")
    v, h = weight.shape
    if h < 1:
        raise ValueError("H must be at least 1")
    if weight.dtype != torch.int8:
        raise TypeError("weight must be int8")
    if weight_scale.shape != (v,) or weight_scale.dtype != torch.float32:
        raise ValueError("weight_scale must be (V,) float32")
    lead = x.shape[:-1]
    if x.dtype == torch.int8:
        code = abi.FLCE_Q_I8
        if x_scale is None or x_scale.shape != lead or x_scale.dtype != torch.float32:
            raise ValueError("int8 x needs x_scale, float32 with x's leading shape")
    else:
        code = _DTYPES.get(x.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16, float16 or int8")
        if x_scale is not None:
            raise ValueError("x_scale goes with int8 x only")
    out_dtype = (torch.float32 if x.dtype == torch.int8 else x.dtype) if out_dtype is None \
        else out_dtype
    if out_dtype not in _DTYPES:
        raise TypeError(f"unsupported out_dtype {out_dtype}")
    if bias is not None and (bias.shape != (v,) or bias.dtype not in _DTYPES):
        raise ValueError("bias must be (V,), float32, bfloat16 or float16")
    refuse_gradient("int8_linear", ("x", "weight_scale", "bias", "x_scale"), x, weight_scale, bias,
                    x_scale)
    dev = x.device
    for name, t in (("x", x), ("weight", weight), ("weight_scale", weight_scale),
                    ("bias", bias), ("x_scale", x_scale), ("err_word", err_word)):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, x on {dev}")
    if err_word is not None and (err_word.dtype != torch.int32 or err_word.numel() != 1):
        raise TypeError("err_word must be one int32")
    x, n, x_pitch = _rows(x)
    if v and (weight.stride(1) != 1 and h > 1 or weight.stride(0) < h):
        weight = weight.contiguous()
    w_pitch = max(weight.stride(0), h)
    weight_scale = weight_scale.contiguous()
    bias = None if bias is None else bias.contiguous()
    x_scale = None if x_scale is None else x_scale.contiguous()
    out = torch.empty(*lead, v, dtype=out_dtype, device=dev)
    prob = abi.flce_qproblem(n, h, v, x_pitch, w_pitch, v, code, _DTYPES[out_dtype],
                             0 if bias is None else _DTYPES[bias.dtype],
                             0 if bias is None else 1, float(logit_scale),
                             0.0 if softcap is None else float(softcap),
                             abi.FLCE_Q_LAY_OUT_WEIGHT if weight.data_ptr() % 16 else 0, 0)
    with on_device(dev):
        ws_bytes = abi.flce_qlinear_workspace_size(prob)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        stream = raw_stream(dev)
        abi.flce_qlinear(prob, x.data_ptr(), None if x_scale is None else x_scale.data_ptr(),
                         weight.data_ptr(), weight_scale.data_ptr(),
                         None if bias is None else bias.data_ptr(), out.data_ptr(),
                         None if err_word is None else err_word.data_ptr(), ws.data_ptr(),
                         ws_bytes, stream)
    return out
