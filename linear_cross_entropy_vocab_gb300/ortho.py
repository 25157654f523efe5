"""Matrices with their singular values taken towards 1, by Newton-Schulz products: what an
optimiser makes of a matrix's momentum before it adds it to the weights.

    x = g / (|g| + eps)                      |g|: root of the sum of squares
    x = a x + (b (x x^T) + c (x x^T)^2) x    for each step's a, b, c

The work runs in libflce.so (``flce_orthogonalize``).
"""
from __future__ import annotations

import array
import itertools
from typing import Optional, Sequence, Tuple

import torch

from . import abi
from ._autograd import refuse_gradient
from ._stream import on_device, raw_stream

__all__ = ["orthogonalize", "NEWTON_SCHULZ"]

_DTYPES = {torch.float32: abi.FLCE_F32, torch.bfloat16: abi.FLCE_BF16,
           torch.float16: abi.FLCE_F16}

# Five steps that lift small singular values quickly: those above 0.002 of the norm end between
# 0.68 and 1.21.
NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5


def _table(coefficients):
    """The coefficients as 32-bit floats in host memory, and the number of steps."""
    if any(len(triple) != 3 for triple in coefficients):
        raise ValueError("coefficients must be triples")
    if not 1 <= len(coefficients) <= 64:
        raise ValueError("coefficients must have 1 to 64 triples")
    return array.array("f", itertools.chain.from_iterable(coefficients)), len(coefficients)


def orthogonalize(x: torch.Tensor, *,
                  coefficients: Sequence[Tuple[float, float, float]] = NEWTON_SCHULZ,
                  eps: float = 1e-7, out_dtype: Optional[torch.dtype] = None,
                  err_word: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each matrix of x [..., M, N] with its singular values taken towards 1 and its singular
    vectors as they are; matrices of one shape are best given together.

    x is float32, bfloat16 or float16; the result [..., M, N] is bfloat16 or float16
    (``out_dtype``, by default x's type, bfloat16 for float32). ``coefficients`` has a triple for
    each step, at most 64. They have to keep the largest singular value, which is at most 1 before
    the first step, in 1e-4 to 16, and each step's a + b t + c t^2 (t its square) below 1e4 in
    magnitude, and both within 1.5 times that where every step finds its values larger by 2^-9:
    schedules that are tuned step by step need their safety factor (a / 1.01, b / 1.01^3,
    c / 1.01^5); without it they magnify roundings and are refused. Products are taken of 11-bit
    values with 32-bit sums: with the default steps the result of noise, or of noise with a few
    larger directions, is within 2.5e-3 of itself in the 2-norm (3e-3 in bfloat16). Where singular
    values lie far apart, noise comes to that in the directions of the smallest, of a 2-norm of
    2^-12 times the product of the a (0.12 with the default steps, where each singular value near 1
    counts 1). A matrix of zeros stays one; one that holds a NaN or an infinity becomes NaN. It has
    no gradient: an x that asks for one is refused. Sides are at most 2^20, and the matrices of a
    call at most 65535. ``err_word`` (one int32, which the caller clears and reads) gets
    FLCE_DEVERR_TIMEOUT if a kernel gave up waiting, after 4 seconds, and left the result
    incomplete; without it that is not reported.
    """
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}: use float32, bfloat16 or float16")
    if x.dim() < 2:
        raise ValueError("x must be (..., M, N)")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == torch.float32 else x.dtype
    if out_dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"out_dtype must be bfloat16 or float16, not {out_dtype}")
    table, steps = _table(coefficients)
    eps = float(eps)
    if not 1.1754944e-38 <= eps <= 3.4028234e38:
        raise ValueError("eps must be finite and at least 2^-126")
    refuse_gradient("orthogonalize", ("x",), x)
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dev = x.device
    if err_word is not None:
        if err_word.dtype != torch.int32 or err_word.numel() != 1:
            raise TypeError("err_word must be one int32")
        if err_word.device != dev:
            raise ValueError(f"err_word is on {err_word.device}, x on {dev}")
    lead, (m, n) = x.shape[:-2], x.shape[-2:]
    out = torch.empty(x.shape, dtype=out_dtype, device=dev)
    if out.numel() == 0:
        return out
    if x.stride(-1) != 1 and n > 1 or x.stride(-2) < n and m > 1:
        x = x.contiguous()
    if len(lead) != 1:
        x = x.reshape(-1, m, n) if lead else x.unsqueeze(0)
    prob = abi.flce_ortho_problem(x.shape[0], m, n, x.stride(0), max(x.stride(1), n), code,
                                  _DTYPES[out_dtype], steps, eps, table.buffer_info()[0], 0)
    with on_device(dev):
        ws_bytes = abi.flce_orthogonalize_workspace_size(prob)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        abi.flce_orthogonalize(prob, x.data_ptr(), out.data_ptr(),
                               None if err_word is None else err_word.data_ptr(), ws.data_ptr(),
                               ws_bytes, raw_stream(dev))
    return out
