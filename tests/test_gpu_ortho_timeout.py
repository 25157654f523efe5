"""What orthogonalising does when a wait runs out: it reports and returns, and the next call is
right. The second product waits for a count that nothing makes; nothing faults."""
import ctypes
import time

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import abi, orthogonalize
from linear_cross_entropy_vocab_gb300.ortho import NEWTON_SCHULZ

pytestmark = pytest.mark.gpu


def _problem(x):
    flat = [v for triple in NEWTON_SCHULZ for v in triple]
    table = (ctypes.c_float * len(flat))(*flat)
    p = abi.flce_ortho_problem(x.shape[0], x.shape[1], x.shape[2], x.stride(0), x.stride(1),
                               abi.FLCE_F32, abi.FLCE_F16, len(NEWTON_SCHULZ), 1e-7,
                               ctypes.addressof(table), 0)
    p.table = table  # kept alive
    return p


# tiles of 128 by CTAs, cut or in a batch, and of 256 by pairs, with groups of steps and without
@pytest.mark.parametrize("batch,m,n", [(1, 300, 520), (3, 200, 900), (1, 2300, 2200),
                                       (8, 1000, 2700)])
def test_a_lost_count_is_reported(batch, m, n):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(batch, m, n, generator=g, device="cuda")
    want = orthogonalize(x, out_dtype=torch.float16)
    p = _problem(x)
    size = abi.flce_orthogonalize_workspace_size(p)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    start = time.perf_counter()
    abi.flce_selftest_orthogonalize_timeout(p, x.data_ptr(), out.data_ptr(), err.data_ptr(),
                                            ws.data_ptr(), size, 0.05, stream)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    assert int(err) & abi.FLCE_DEVERR_TIMEOUT
    assert 0.05 <= took < 5.0, took
    # the same workspace again, with nothing lost
    err.zero_()
    abi.flce_orthogonalize(p, x.data_ptr(), out.data_ptr(), err.data_ptr(), ws.data_ptr(), size,
                           stream)
    assert int(err) == 0 and torch.equal(out, want)


def test_argument_checks():
    x = torch.zeros(1, 300, 520, device="cuda")
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    p = _problem(x)

    def call(p, err, budget):
        return abi.flce_selftest_orthogonalize_timeout(p, x.data_ptr(), x.data_ptr(), err, None, 0,
                                                       budget, None, check=False)

    for bad in (0.0, -1.0, 2.0):
        assert call(p, err.data_ptr(), bad) == abi.FLCE_ERR_INVALID_ARG
    assert call(p, None, 0.05) == abi.FLCE_ERR_INVALID_ARG
    assert call(p, err.data_ptr(), 0.05) == abi.FLCE_ERR_WORKSPACE
    small = _problem(x[:, :100])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert abi.flce_selftest_orthogonalize_timeout(
        small, x.data_ptr(), x.data_ptr(), err.data_ptr(), ws.data_ptr(), 1 << 20, 0.05, None,
        check=False) == abi.FLCE_ERR_UNSUPPORTED
