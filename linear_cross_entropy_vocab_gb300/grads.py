"""The norm of a set of gradients taken together, and clipping by it.

    norm = (sum |g|^p)^(1/p) over every element of every gradient   (p = 1, 2)
    norm = max |g|                                                  (p = inf)
    clipped = g * min(1, max_norm / (norm + eps))

Two kernel launches for up to 500 tensors, one for a clip of few small ones, more in steps of 500;
the norm stays on the device and nothing waits for it, so a clip can be captured into a CUDA graph
with the step that it belongs to. Autograd records none of it: the norm is a constant. The work
runs in libflce.so (``flce_grad_norm``, ``flce_grad_clip``).
"""
from __future__ import annotations

import array
import math
from typing import Iterable, Optional, Sequence

import torch

from . import abi
from ._stream import on_device, raw_stream

__all__ = ["grad_norm", "clip_grads_", "clip_grads", "clip_grad_norm_"]

_DTYPES = {torch.float32: abi.FLCE_F32, torch.bfloat16: abi.FLCE_BF16,
           torch.float16: abi.FLCE_F16}
_NORMS = {1.0: abi.FLCE_NORM_L1, 2.0: abi.FLCE_NORM_L2, math.inf: abi.FLCE_NORM_INF}
_MAX_RUNS = 1 << 16  # of one tensor that is neither dense nor rows with a pitch


def _norm_code(norm_type) -> int:
    try:
        return _NORMS[float(norm_type)]
    except (KeyError, TypeError, ValueError):
        raise ValueError(f"norm_type must be 1, 2 or inf, not {norm_type!r}") from None


def _runs(g: torch.Tensor, o: torch.Tensor):
    """(byte offset in g, in o, rows, cols, pitch of g, of o) that cover two tensors of one
    shape."""
    dims = sorted(((s, a, b) for s, a, b in zip(g.shape, g.stride(), o.stride()) if s > 1),
                  key=lambda d: (-d[1], -d[2]))
    merged: list = []
    for s, a, b in dims:
        if merged and merged[-1][1] == a * s and merged[-1][2] == b * s:
            merged[-1] = (merged[-1][0] * s, a, b)
        else:
            merged.append((s, a, b))
    cols = 1
    if merged and merged[-1][1] == 1 and merged[-1][2] == 1:
        cols = merged.pop()[0]
    rows, pg, po = merged.pop() if merged else (1, cols, cols)
    outer = 1
    for s, _, _ in merged:
        outer *= s
    if outer > _MAX_RUNS:
        raise ValueError("a gradient has too many separate pieces: make it contiguous")
    starts = [(0, 0)]
    for s, a, b in merged:
        starts = [(x + i * a, y + i * b) for x, y in starts for i in range(s)]
    return [(x * g.element_size(), y * o.element_size(), rows, cols, pg, po) for x, y in starts]


def _table(grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]]):
    """The flce_grad structs of the gradients as 64-bit words, and the gradients' device."""
    words: list = []
    if not grads:
        return array.array("q"), None
    device, index = grads[0].device, grads[0].get_device()
    add, code_of = words.extend, _DTYPES.get
    for i, g in enumerate(grads):
        code = code_of(g.dtype)
        if code is None:
            raise TypeError(f"gradient {i} is {g.dtype}: use float32, bfloat16 or float16")
        if not g.is_cuda:
            raise ValueError(f"gradient {i} must be a CUDA tensor")
        if g.get_device() != index:
            raise ValueError(f"gradient {i} is on {g.device}, the first on {device}")
        if g.layout is not torch.strided:
            raise ValueError(f"gradient {i} must be a dense tensor, not {g.layout}")
        n = g.numel()
        if out is None:
            if n == 0:
                continue
            src = g.data_ptr()
            if g.is_contiguous():
                add((src, src, 1, n, n, n, code | code << 32))
            else:
                for x, y, rows, cols, pg, po in _runs(g, g):
                    add((src + x, src + y, rows, cols, pg, po, code | code << 32))
            continue
        o = out[i]
        if o.shape != g.shape:
            raise ValueError(f"out {i} is {tuple(o.shape)}, its gradient {tuple(g.shape)}")
        out_code = code_of(o.dtype)
        if out_code != code and out_code != abi.FLCE_F32:
            raise TypeError(f"out {i} must be {g.dtype} or float32, not {o.dtype}")
        if o.get_device() != index or o.layout is not torch.strided:
            raise ValueError(f"out {i} must be a dense tensor on {device}")
        if n == 0:
            continue
        src, dst, codes = g.data_ptr(), o.data_ptr(), code | out_code << 32
        if g.is_contiguous() and o.is_contiguous():
            add((src, dst, 1, n, n, n, codes))
        else:
            for x, y, rows, cols, pg, po in _runs(g, o):
                add((src + x, dst + y, rows, cols, pg, po, codes))
    return array.array("q", words), device


def _run(grads, out, norm_type, max_norm, eps) -> torch.Tensor:
    code = _norm_code(norm_type)
    table, device = _table(grads, out)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    count = len(table) // 7
    address = table.buffer_info()[0] if count else None
    with on_device(device):
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws_bytes = abi.flce_grad_workspace_size(count)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        stream = raw_stream(device)
        if max_norm is None:
            abi.flce_grad_norm(address, count, code, norm.data_ptr(), ws.data_ptr(), ws_bytes,
                               stream)
        else:
            abi.flce_grad_clip(address, count, code, max_norm, eps, norm.data_ptr(),
                               ws.data_ptr(), ws_bytes, stream)
    return norm


def _limits(max_norm, eps):
    max_norm, eps = float(max_norm), float(eps)
    if not (math.isfinite(max_norm) and max_norm >= 0):
        raise ValueError("max_norm must be finite and not negative")
    if not (math.isfinite(eps) and eps >= 0):
        raise ValueError("eps must be finite and not negative")
    return max_norm, eps


def _listed(tensors) -> list:
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


def grad_norm(grads: Iterable[torch.Tensor], norm_type: float = 2.0) -> torch.Tensor:
    """The norm over every element of ``grads`` (0-d fp32 on their device); 0 without any.
    Tensors may be of different types, shapes and strides; they are on one device."""
    return _run(_listed(grads), None, norm_type, None, None)


def clip_grads_(grads: Iterable[torch.Tensor], max_norm: float, norm_type: float = 2.0, *,
                eps: float = 1e-6) -> torch.Tensor:
    """Scale ``grads`` in place so that their norm is at most ``max_norm``; returns the norm that
    they had (0-d fp32, on the device). No two of them may share memory. Where the norm is small
    enough already, nothing is written. A NaN norm makes every gradient NaN, an infinite one makes
    the finite ones 0."""
    max_norm, eps = _limits(max_norm, eps)
    grads = _listed(grads)
    norm = _run(grads, None, norm_type, max_norm, eps)
    torch.autograd.graph.increment_version(grads)
    return norm


def clip_grads(grads: Iterable[torch.Tensor], max_norm: float, norm_type: float = 2.0, *,
               out: Iterable[torch.Tensor], eps: float = 1e-6) -> torch.Tensor:
    """As :func:`clip_grads_`, with the clipped gradients written to ``out``: tensors of the
    gradients' shapes, in their types or in float32 (an optimizer's 32-bit copies)."""
    max_norm, eps = _limits(max_norm, eps)
    grads, out = _listed(grads), _listed(out)
    if len(out) != len(grads):
        raise ValueError(f"{len(grads)} gradients and {len(out)} outputs")
    norm = _run(grads, out, norm_type, max_norm, eps)
    torch.autograd.graph.increment_version(out)
    return norm


def clip_grad_norm_(parameters: Iterable[torch.Tensor], max_norm: float, norm_type: float = 2.0,
                    error_if_nonfinite: bool = False, *, eps: float = 1e-6) -> torch.Tensor:
    """:func:`clip_grads_` over the ``.grad`` of ``parameters`` (those without one are left out).
    A ``max_norm`` of inf sets no limit: the norm is returned and the gradients stay as they are,
    whatever it is. ``error_if_nonfinite`` waits for the norm and raises before anything is scaled
    if it is not finite."""
    unlimited = max_norm == math.inf
    _limits(0.0 if unlimited else max_norm, eps)
    grads = [p.grad for p in _listed(parameters) if p.grad is not None]
    if error_if_nonfinite or unlimited:
        norm = grad_norm(grads, norm_type)
        if error_if_nonfinite and not math.isfinite(float(norm)):
            raise RuntimeError(f"the gradients' norm is {float(norm)}: they are not clipped")
        if unlimited:
            return norm
    return clip_grads_(grads, max_norm, norm_type, eps=eps)
