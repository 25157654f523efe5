"""Fused linear cross-entropy for one GB300 GPU (sm_103a).

``fused_linear_cross_entropy`` computes the cross-entropy of
``softcap(logit_scale * (hidden @ weight.T + bias))`` against ``targets``
without materialising the (N, V) logits, with the metrics and gradients of
the "fused-linear-ce" model card (trl-lib). The compute runs in the
hand-written CUDA kernels of ``libflce.so`` (C ABI: include/flce.h); this
package marshals tensors to it. ``fused_linear_kl_div`` is the same fused
projection with a KL divergence against teacher probabilities
(FusedLinearKLDivLoss pull request, Liger-Kernel #1423).

Beside the losses: ``clip_grad_norm_`` and its parts (the norm of many gradients
and clipping by it, for the training step), ``orthogonalize`` (an update whose
singular values are near 1), ``int8_linear`` and
``quantize_rows`` (the head in 8-bit integers) and ``beam_select`` and
``beam_reorder_`` (a beam search's choice over the vocabulary and the
reordering of its states). In front of the head: ``rms_norm`` and
``rms_norm_quantize`` (the norm with the residual's addition, with gradients or
in 8-bit integers).
"""
from .api import (  # noqa: F401
    flce_backward_tensors, flce_forward_tensors, flce_kl_backward_tensors,
    flce_kl_forward_tensors, fused_linear_cross_entropy, fused_linear_kl_div)
from .beam import BeamSelection, beam_reorder_, beam_select  # noqa: F401
from .grads import clip_grad_norm_, clip_grads, clip_grads_, grad_norm  # noqa: F401
from .int8 import int8_linear, quantize_rows  # noqa: F401
from .norm import rms_norm, rms_norm_quantize  # noqa: F401
from .ortho import orthogonalize  # noqa: F401
from .native_build import build  # noqa: F401

__all__ = ["fused_linear_cross_entropy", "flce_forward_tensors", "flce_backward_tensors",
           "fused_linear_kl_div", "flce_kl_forward_tensors", "flce_kl_backward_tensors",
           "grad_norm", "clip_grads_", "clip_grads", "clip_grad_norm_",
           "BeamSelection", "beam_select", "beam_reorder_", "quantize_rows", "int8_linear",
           "rms_norm", "rms_norm_quantize", "orthogonalize",
           "build"]
