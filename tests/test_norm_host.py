"""Refusals of the root-mean-square norm, which need no GPU: the C entry points return their status
before any CUDA call, and the Python layer raises before it calls them."""
import ctypes
import math

import pytest
import torch

import linear_cross_entropy_vocab_gb300 as package
from linear_cross_entropy_vocab_gb300 import abi, native_build

FAKE = 0x10000  # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = (abi.FLCE_ERR_INVALID_ARG, abi.FLCE_ERR_UNSUPPORTED,
                                   abi.FLCE_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def lib():
    native_build.build()
    return abi.load()


def _problem(**kw):
    args = dict(n=5, h=100, x_pitch=100, residual_pitch=100, dtype=abi.FLCE_BF16,
                sum_dtype=abi.FLCE_BF16, weight_dtype=abi.FLCE_BF16, eps=1e-6, reserved=0)
    args.update(kw)
    return abi.flce_norm_problem(**args)


BAD = [dict(n=-1), dict(n=1 << 31), dict(dtype=3), dict(sum_dtype=abi.FLCE_F16),
       dict(weight_dtype=abi.FLCE_F16), dict(x_pitch=99), dict(residual_pitch=99),
       dict(x_pitch=1 << 60), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan),
       dict(eps=math.inf), dict(eps=1e-39), dict(reserved=1)]


def _norm(p, x=FAKE, r=None, w=None, y=FAKE, s=None, rstd=None):
    return abi.flce_rms_norm(p, x, r, w, y, s, rstd, None, check=False)


def _quant(p, x=FAKE, r=None, w=None, q=FAKE, pitch=112, scale=FAKE, s=None):
    return abi.flce_rms_norm_quantize(p, x, r, w, q, pitch, scale, s, None, check=False)


def _back(p, dy=FAKE, ds=None, total=FAKE, w=FAKE, rstd=FAKE, gx=FAKE, gr=None, gw=FAKE, ws=FAKE,
          size=1 << 40):
    return abi.flce_rms_norm_backward(p, dy, ds, total, w, rstd, gx, gr, gw, ws, size, None,
                                      check=False)


def test_struct_layout():
    assert ctypes.sizeof(abi.flce_norm_problem) == 56


def test_problem_refusals():
    for bad in BAD:
        for call in (_norm, _quant, _back):
            assert call(_problem(**bad)) == INVALID, bad
        assert abi.flce_rms_norm_backward_workspace_size(_problem(**bad)) == 0
    for h in (0, -4, (1 << 24) + 1):
        p = _problem(h=h, x_pitch=1 << 30, residual_pitch=1 << 30)
        for call in (_norm, _quant, _back):
            assert call(p) == UNSUPPORTED


def test_pointer_refusals():
    p = _problem()
    assert _norm(p, x=None) == INVALID
    assert _norm(p, y=None) == INVALID
    assert _norm(p, r=FAKE) == INVALID
    assert _norm(p, s=FAKE) == INVALID
    for name in ("x", "y", "w"):
        assert _norm(p, **{name: FAKE + 1}) == UNSUPPORTED
    assert _norm(p, r=FAKE + 1, s=FAKE) == UNSUPPORTED
    assert _norm(_problem(sum_dtype=abi.FLCE_F32), r=FAKE, s=FAKE + 2) == UNSUPPORTED
    assert _norm(p, rstd=FAKE + 2) == UNSUPPORTED
    assert _quant(p, q=None) == INVALID
    assert _quant(p, scale=None) == INVALID
    assert _quant(p, pitch=99) == INVALID
    assert _quant(p, scale=FAKE + 2) == UNSUPPORTED
    for name in ("dy", "total", "rstd"):
        assert _back(p, **{name: None}) == INVALID
    assert _back(p, w=None) == INVALID
    assert _back(p, gr=FAKE) == INVALID  # the sum is not fp32
    for name in ("dy", "ds", "total", "w", "rstd", "gx", "gw"):
        assert _back(p, **{name: FAKE + 1}) == UNSUPPORTED
    assert _back(p, size=8) == WORKSPACE
    assert _back(p, ws=None) == WORKSPACE
    assert _back(p, ws=FAKE + 8) == WORKSPACE


def test_python_refusals():
    x, w = torch.zeros(3, 8), torch.ones(8)
    for call in (package.rms_norm, package.rms_norm_quantize):
        with pytest.raises(ValueError, match="CUDA"):
            call(x, w)
        with pytest.raises(TypeError):
            call(x.double())
        with pytest.raises(TypeError):
            call(x.long())
        with pytest.raises(ValueError, match="weight"):
            call(x, torch.ones(7))
        with pytest.raises(TypeError, match="weight"):
            call(x, w.bfloat16())
        with pytest.raises(ValueError, match="residual"):
            call(x, w, residual=torch.zeros(8))
        with pytest.raises(TypeError, match="residual"):
            call(x, w, residual=x.half())
        with pytest.raises(ValueError, match="H of at least 1"):
            call(torch.zeros(3, 0))
        with pytest.raises(ValueError, match="H of at least 1"):
            call(torch.zeros(()))
        for eps in (0.0, -1.0, math.nan, math.inf, 1e-39):
            with pytest.raises(ValueError, match="eps"):
                call(x, w, eps)
