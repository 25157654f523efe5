"""Refusals of the orthogonalising operator, which need no GPU: the C entry point returns its status
before any CUDA call, and the Python layer raises before it calls it."""
import ctypes
import math

import pytest
import torch

import linear_cross_entropy_vocab_gb300 as package
from linear_cross_entropy_vocab_gb300 import abi, native_build

FAKE = 0x10000  # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = (abi.FLCE_ERR_INVALID_ARG, abi.FLCE_ERR_UNSUPPORTED,
                                   abi.FLCE_ERR_WORKSPACE)
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def lib():
    native_build.build()
    return abi.load()


def _problem(triples=(QUINTIC,) * 5, **kw):
    flat = [v for triple in triples for v in triple]
    table = (ctypes.c_float * max(len(flat), 1))(*flat)
    args = dict(batch=2, rows=300, cols=200, batch_stride=60000, row_pitch=200, dtype=abi.FLCE_F32,
                out_dtype=abi.FLCE_BF16, steps=len(triples), eps=1e-7,
                coefficients=ctypes.addressof(table), reserved=0)
    args.update(kw)
    p = abi.flce_ortho_problem(**args)
    p.table = table  # kept alive
    return p


def _call(p, src=FAKE, out=FAKE, err=None, ws=FAKE, size=1 << 50):
    return abi.flce_orthogonalize(p, src, out, err, ws, size, None, check=False)


def test_struct_layout():
    assert ctypes.sizeof(abi.flce_ortho_problem) == 72


def test_problem_refusals():
    for bad in (dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(dtype=3), dict(out_dtype=3),
                dict(out_dtype=abi.FLCE_F32), dict(row_pitch=199), dict(batch_stride=-1),
                dict(row_pitch=1 << 50), dict(batch_stride=1 << 60), dict(eps=0.0),
                dict(eps=math.nan), dict(eps=math.inf), dict(steps=0), dict(steps=65),
                dict(coefficients=None), dict(reserved=1)):
        p = _problem(**bad)
        assert _call(p) == INVALID, bad
        assert abi.flce_orthogonalize_workspace_size(p) == 0
    for bad in (dict(batch=65536), dict(rows=(1 << 20) + 1),
                dict(cols=(1 << 20) + 1, row_pitch=1 << 21)):
        assert _call(_problem(**bad)) == UNSUPPORTED, bad
    assert _call(_problem(batch=60000, rows=1 << 20, cols=1 << 20, row_pitch=1 << 20)) \
        == UNSUPPORTED


def test_coefficients_that_leave_the_range():
    for bad in ((20.0, 0.0, 0.0), (3.0, 30.0, 0.0), (math.nan, 0.0, 0.0), (1.0, math.inf, 0.0),
                (0.0, 0.0, 0.0), (1e-5, 0.0, 0.0), (3e38, -3e38, 3e38)):
        assert _call(_problem((bad,))) == UNSUPPORTED, bad
    # each step is fine by itself
    assert _call(_problem(((5.0, 0.0, 0.0),) * 2)) == UNSUPPORTED
    assert _call(_problem(((5.0, 0.0, 0.0), (0.5, 0.0, 0.0))), size=8) == WORKSPACE
    # the largest value lies inside the range: 3 s - 3 s^5 at s = (1/5)^(1/4)
    assert _call(_problem(((9.0, 0.0, -9.0),)), size=8) == WORKSPACE
    assert _call(_problem(((35.0, 0.0, -35.0),))) == UNSUPPORTED


def test_pointer_refusals():
    p = _problem()
    assert _call(p, src=None) == INVALID
    assert _call(p, out=None) == INVALID
    assert _call(p, src=FAKE + 2) == UNSUPPORTED
    assert _call(p, out=FAKE + 1) == UNSUPPORTED
    assert _call(p, err=FAKE + 2) == UNSUPPORTED
    assert _call(p, size=8) == WORKSPACE
    assert _call(p, ws=None) == WORKSPACE
    assert _call(p, ws=FAKE + 8) == WORKSPACE


def test_workspace_size():
    p = _problem(batch=3, rows=14336, cols=4096, row_pitch=4096)
    size = abi.flce_orthogonalize_workspace_size(p)
    held = 3 * (2 * 2 * 4096 * 14336 + 4 * 2 * 4096 * 4096)
    # and the sums of tiles whose contraction is cut
    assert held <= size <= held + (1 << 20) + 160 * 256 * 1024
    small = _problem(batch=1, rows=256, cols=200, row_pitch=200)
    assert abi.flce_orthogonalize_workspace_size(small) <= 3 << 20
    # none for matrices that stay in shared memory
    assert abi.flce_orthogonalize_workspace_size(_problem(rows=128, cols=4096, row_pitch=4096)) == 0
    assert _call(_problem(rows=128), src=None) == INVALID


def test_python_refusals():
    x = torch.zeros(3, 8)
    call = package.orthogonalize
    with pytest.raises(ValueError, match="CUDA"):
        call(x)
    with pytest.raises(TypeError):
        call(x.double())
    with pytest.raises(TypeError, match="out_dtype"):
        call(x, out_dtype=torch.float32)
    with pytest.raises(ValueError, match=r"\(\.\.\., M, N\)"):
        call(torch.zeros(3))
    with pytest.raises(ValueError, match="triples"):
        call(x, coefficients=((1.0, 2.0),))
    for bad in ((), (QUINTIC,) * 65):
        with pytest.raises(ValueError, match="1 to 64"):
            call(x, coefficients=bad)
    for eps in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(ValueError, match="eps"):
            call(x, eps=eps)
    with pytest.raises(RuntimeError, match="no gradient"):
        call(x.requires_grad_())
