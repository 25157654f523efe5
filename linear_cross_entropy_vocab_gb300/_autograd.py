"""What an operator without a gradient does with inputs that ask for one."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

__all__ = ["refuse_gradient"]

_recording = torch.is_grad_enabled


def refuse_gradient(operator: str, names: tuple, *inputs) -> None:
    """Raise where autograd would record the call on one of ``inputs`` (tensors or None) or carry
    a forward-mode tangent through it: the result would silently be a constant."""
    if _recording():
        for i, t in enumerate(inputs):
            if t is not None and t.requires_grad:
                raise RuntimeError(f"{operator} has no gradient, and {names[i]} asks for one: "
                                   "call it under torch.no_grad() or on a detached tensor")
    if forward_ad._current_level >= 0:
        for i, t in enumerate(inputs):
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{operator} has no gradient, and {names[i]} carries a "
                                   "forward-mode tangent")
