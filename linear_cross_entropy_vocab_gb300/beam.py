"""One step of a beam search over the vocabulary: the choice among all continuations of a
prompt's beams, and the reordering of what is kept for each beam.

    score[b, k, v] = beam_scores[b, k] + logits[b, k, v] - logsumexp(logits[b, k])

The work runs in libflce.so (``flce_beam_select``, ``flce_beam_reorder``).
"""
from __future__ import annotations

import array
from typing import Iterable, NamedTuple, Optional, Union

import torch

from . import abi
from ._autograd import refuse_gradient
from ._stream import on_device, raw_stream

__all__ = ["BeamSelection", "beam_select", "beam_reorder_"]

_DTYPES = {torch.float32: abi.FLCE_F32, torch.bfloat16: abi.FLCE_BF16,
           torch.float16: abi.FLCE_F16}


class BeamSelection(NamedTuple):
    """[B, M] each, best first: the score (fp32), the beam that is continued and the token
    (int64)."""

    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor


def _on(name: str, t: torch.Tensor, device) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _err_ptr(err_word: Optional[torch.Tensor], device):
    if err_word is None:
        return None
    if err_word.dtype != torch.int32 or err_word.numel() != 1:
        raise TypeError("err_word must be one int32")
    _on("err_word", err_word, device)
    return err_word.data_ptr()


def beam_select(logits: torch.Tensor, beam_scores: torch.Tensor,
                num_candidates: Optional[int] = None, *,
                finished: Optional[torch.Tensor] = None,
                allowed: Optional[torch.Tensor] = None, pad_token: int = 0,
                err_word: Optional[torch.Tensor] = None) -> BeamSelection:
    """The ``num_candidates`` (default K; at most 256) best continuations of each prompt.

    logits [B, K, V] (float32, bfloat16 or float16; K at most 1024, V below 2^31 - 8192) and
    beam_scores [B, K] (float32, the log probability of each beam so far). Scores that are equal
    are taken in the order of k * V + v.

    ``allowed`` (bool, broadcast to [B, K, V]): tokens that may come; the others count as logits
    of -inf, whatever they hold. ``finished`` (bool [B, K]): beams at their end; each offers
    itself alone, its score unchanged, under ``pad_token``. Beams with score -inf and beams whose
    mask leaves nothing offer nothing; places that nothing fills hold score -inf, parent 0 and
    ``pad_token``. ``err_word`` (one int32, which the caller clears and reads) gets
    FLCE_DEVERR_NOT_FINITE where an allowed logit or a beam score is NaN or +inf; that beam
    offers nothing. The scores have no gradient: logits or beam scores that ask for one are
    refused.
    """
    if logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    b, k, v = logits.shape
    code = _DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {logits.dtype}: use float32, bfloat16 or float16")
    if k < 1 or v < 1:
        raise ValueError("logits need at least one beam and one token")
    refuse_gradient("beam_select", ("logits", "beam_scores"), logits, beam_scores)
    dev = logits.device
    _on("logits", logits, dev)
    if beam_scores.shape != (b, k):
        raise ValueError("beam_scores must be (B, K)")
    if beam_scores.dtype != torch.float32:
        raise TypeError("beam_scores must be float32")
    _on("beam_scores", beam_scores, dev)
    if logits.stride(2) != 1 and v > 1:
        logits = logits.contiguous()
    beam_scores = beam_scores.contiguous()
    fin_ptr = ok_ptr = None
    ok_b = ok_k = 0
    if finished is not None:
        if finished.shape != (b, k):
            raise ValueError("finished must be (B, K)")
        if finished.dtype != torch.bool:
            raise TypeError("finished must be bool")
        _on("finished", finished, dev)
        finished = finished.contiguous()
        fin_ptr = finished.data_ptr()
    if allowed is not None:
        if allowed.dtype != torch.bool:
            raise TypeError("allowed must be bool")
        _on("allowed", allowed, dev)
        if allowed.dim() == 0 or allowed.shape[-1] != v:
            raise ValueError("allowed must be broadcastable to (B, K, V), with V of its own")
        if allowed.stride(-1) != 1 and v > 1:
            allowed = allowed.contiguous()
        try:
            allowed = allowed.expand(b, k, v)
        except RuntimeError:
            raise ValueError(f"allowed {tuple(allowed.shape)} cannot be broadcast to "
                             f"{(b, k, v)}") from None
        ok_ptr = allowed.data_ptr()
        ok_b, ok_k = allowed.stride(0), allowed.stride(1)
    m = k if num_candidates is None else int(num_candidates)
    prob = abi.flce_beam_problem(b, k, v, m, logits.stride(0), logits.stride(1), ok_b, ok_k,
                                 int(pad_token), code, 0)
    if m < 1:
        raise ValueError("num_candidates must be at least 1")
    scores = torch.empty(b, m, dtype=torch.float32, device=dev)
    parents = torch.empty(b, m, dtype=torch.int64, device=dev)
    tokens = torch.empty(b, m, dtype=torch.int64, device=dev)
    with on_device(dev):
        ws_bytes = abi.flce_beam_select_workspace_size(prob)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        stream = raw_stream(dev)
        abi.flce_beam_select(prob, logits.data_ptr(), beam_scores.data_ptr(), fin_ptr, ok_ptr,
                             scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                             _err_ptr(err_word, dev), ws.data_ptr(), ws_bytes, stream)
    return BeamSelection(scores, parents, tokens)


_NO_STATE = (0, 0, 1, 1, 1, 1, 0, 0, 0, 0, 0)  # nothing to move


def _state_words(i: int, t: torch.Tensor, dim: int, rows: int) -> tuple:
    """The flce_beam_state of a tensor whose axis ``dim`` counts the beams."""
    if not -t.dim() <= dim < t.dim():
        raise ValueError(f"state {i} has no dimension {dim}")
    dim %= t.dim()
    if t.shape[dim] != rows:
        raise ValueError(f"state {i} has {t.shape[dim]} rows along dimension {dim}, not {rows}")
    es = t.element_size()
    strides = t.stride()
    # (stride, size) of the other axes from the widest stride to the narrowest, neighbours that
    # make one axis joined
    dims = [(st, s) for d, (s, st) in enumerate(zip(t.shape, strides)) if d != dim and s != 1]
    if any(s == 0 for _, s in dims) or rows == 0:
        return _NO_STATE
    dims.sort(reverse=True)
    merged: list = []
    for st, s in dims:
        if merged and merged[-1][0] == st * s:
            merged[-1] = (st, merged[-1][1] * s)
        else:
            merged.append((st, s))
    run = es
    if merged and merged[-1][0] == 1:
        run = merged.pop()[1] * es
    n = len(merged)
    if n == 0:
        return (t.data_ptr(), strides[dim] * es, 1, 1, 1, 1, 0, 0, 0, 0, run)
    if n == 1:
        (st, s), = merged
        return (t.data_ptr(), strides[dim] * es, 1, 1, 1, s, 0, 0, 0, st * es, run)
    pad = abi.BEAM_STATE_DIMS - n
    if pad < 0:
        raise ValueError(f"state {i} lies in too many separate pieces: make it contiguous")
    return (t.data_ptr(), strides[dim] * es, *(1,) * pad, *(s for _, s in merged),
            *(0,) * pad, *(st * es for st, _ in merged), run)


def beam_reorder_(states: Union[torch.Tensor, Iterable[torch.Tensor]], parents: torch.Tensor,
                  dim: int = 0, *, err_word: Optional[torch.Tensor] = None) -> None:
    """Reorder what is kept for each beam, in place: along ``dim``, which counts the B * K beams
    of every state, row b * K + j becomes what row b * K + parents[b, j] was.

    ``states`` is a tensor or several, of any types, shapes and strides (views of the filled part
    of a cache among them), that share no memory (one that is listed twice is refused, other
    sharing is not looked for); parents [B, K] int64. Beams that continue themselves are neither
    read nor written. K is at most 64. A parent outside [0, K) leaves its beam as it is and sets
    FLCE_DEVERR_PARENT_RANGE in ``err_word`` (one int32, which the caller clears and reads).
    """
    if parents.dim() != 2:
        raise ValueError("parents must be (B, K)")
    if parents.dtype != torch.int64:
        raise TypeError("parents must be int64")
    b, k = parents.shape
    if k < 1:
        raise ValueError("parents must name at least one beam")
    dev = parents.device
    _on("parents", parents, dev)
    parents = parents.contiguous()
    states = [states] if isinstance(states, torch.Tensor) else list(states)
    words: list = []
    for i, t in enumerate(states):
        if t.layout != torch.strided:
            raise ValueError(f"state {i} must be a dense tensor, not {t.layout}")
        _on(f"state {i}", t, dev)
        words += _state_words(i, t, dim, b * k)
    table = array.array("q", words)
    with on_device(dev):
        stream = raw_stream(dev)
        abi.flce_beam_reorder(table.buffer_info()[0] if states else None, len(states),
                              parents.data_ptr(), b, k, _err_ptr(err_word, dev), stream)
    torch.autograd.graph.increment_version(states)
