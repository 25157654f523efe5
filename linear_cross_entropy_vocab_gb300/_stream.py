"""The device and stream that a call runs on, for entry points whose work is shorter than the
bookkeeping around it."""
from __future__ import annotations

import contextlib

import torch

__all__ = ["on_device", "raw_stream"]

_HERE = contextlib.nullcontext()


def on_device(dev: torch.device):
    """A context in which ``dev`` is the current device; free of charge where it is already."""
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def raw_stream(dev: torch.device) -> int:
    """The cudaStream_t of ``dev``'s current stream (without a Stream object around it)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)
