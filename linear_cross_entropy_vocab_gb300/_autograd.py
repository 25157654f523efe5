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
        for t in inputs:
            if t is not None and t.requires_grad:
                name = next(n for n, x in zip(names, inputs) if x is t)
                raise RuntimeError(f"{operator} has no gradient, and {name} asks for one: call it "
                                   "under torch.no_grad() or on a detached tensor")
    if forward_ad._current_level >= 0:
        for name, t in zip(names, inputs):
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{operator} has no gradient, and {name} carries a forward-mode "
                                   "tangent")
