"""What an operator without a gradient does with inputs that ask for one."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

__all__ = ["refuse_gradient"]


def refuse_gradient(operator: str, **inputs) -> None:
    """Raise where autograd would record the call on one of ``inputs`` (tensors or None) or carry
    a forward-mode tangent through it: the result would silently be a constant."""
    recorded = torch.is_grad_enabled()
    dual = forward_ad._current_level >= 0
    if not (recorded or dual):
        return
    for name, t in inputs.items():
        if t is None:
            continue
        if recorded and t.requires_grad:
            raise RuntimeError(f"{operator} has no gradient, and {name} asks for one: call it "
                               "under torch.no_grad() or on a detached tensor")
        if dual and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{operator} has no gradient, and {name} carries a forward-mode "
                               "tangent")
