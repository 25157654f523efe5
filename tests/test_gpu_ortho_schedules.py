"""Orthogonalising with schedules that are tuned step by step, against the steps in 64 bits.

Tolerance: 1 % of the result's 2-norm, whatever the kernels plan and however they group steps. Each
product's operands are halves, so a step moves a singular value by some 2^-12 of the polynomial's
largest value, which is four to eight times what it multiplies by; the next steps' polynomials rise
at most twelve times as fast as their value where they are steepest, and fall as fast between, so
that a few values of many are off by a per cent or two and most by 1e-3.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import orthogonalize
from linear_cross_entropy_vocab_gb300.abi import FlceError
from test_ortho_schedules_host import STEPWISE, TUNED, TUNED8, safe

pytestmark = pytest.mark.gpu

SCHEDULES = {"tuned5": safe(TUNED[:-1]) + TUNED[-1:], "tuned5_all": safe(TUNED),
             "tuned8": safe(TUNED8[:-1]) + TUNED8[-1:],
             "stepwise": STEPWISE, "top": ((1.0, 0.5, 0.0), (0.3, 0.163, 0.0)) * 3}
# in one CTA's shared memory, in a cluster's, by tiles of 128 and of 256, with steps that share a gram
SIZES = [(1, 100, 300), (2, 128, 1100), (2, 3000, 90), (1, 300, 520), (1, 2300, 2200),
         (1, 1000, 5100), (4, 3000, 700)]


def steps64(g, coefficients, eps=1e-7):
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in coefficients:
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def matrices(kind, batch, m, n, dtype=torch.float32):
    """Noise, noise with what many examples have in common, of some rank, or other spectra."""
    g = torch.Generator("cuda").manual_seed(m + 3 * n)
    x = torch.randn(batch, m, n, generator=g, device="cuda")
    if kind == "momentum":
        rank = max(1, min(m, n) // 32)
        u = torch.randn(batch, m, rank, generator=g, device="cuda")
        v = torch.randn(batch, rank, n, generator=g, device="cuda")
        x.baddbmm_(u, v, alpha=2.0 * rank ** -0.5)
    elif kind != "noise":
        u, values, v = torch.linalg.svd(x.double(), full_matrices=False)
        k = torch.arange(1, min(m, n) + 1, device="cuda", dtype=torch.float64)
        values = {"1/k": 1 / k, "1/k^2": 1 / k ** 2, "one far above": 0.01 + (k < 2) * 10.0,
                  "rank one": (k < 2) * 1.0}[kind]
        x = (u * values) @ v
    return (x * 1e-3).to(dtype)


@pytest.mark.parametrize("name", SCHEDULES)
@pytest.mark.parametrize("batch,m,n", SIZES)
def test_against_64_bits(batch, m, n, name):
    x = matrices("noise", batch, m, n)
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    got = orthogonalize(x, coefficients=SCHEDULES[name], out_dtype=torch.float16, err_word=err)
    for i in {0, batch - 1}:
        want = steps64(x[i], SCHEDULES[name])
        off = float((got[i].double() - want).norm() / want.norm())
        assert off <= 1e-2, off
    assert int(err) == 0


DEFAULT = ((3.4445, -4.7750, 2.0315),) * 5


@pytest.mark.parametrize("kind", ["noise", "momentum"])
@pytest.mark.parametrize("batch,m,n", SIZES + [(1, 1, 9), (5, 16, 40), (1, 4100, 2300)])
def test_the_precision_that_is_promised(batch, m, n, kind):
    """Three roundings a step, each of 2^-12.3 (2^-11 / 6^(1/2), the mean square over a half's
    numbers) magnified some three times, make 15^(1/2) * 3 * 2^-12.3 = 2.3e-3, a result in
    bfloat16 2^-8 / 6^(1/2) = 1.6e-3 more: 2.8e-3 together. Held to 4e-3."""
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        x = matrices(kind, batch, m, n, dtype)
        for out in (torch.float16, torch.bfloat16):
            err = torch.zeros((), dtype=torch.int32, device="cuda")
            got = orthogonalize(x, out_dtype=out, err_word=err)
            for i in {0, batch - 1}:
                want = steps64(x[i], DEFAULT)
                off = float((got[i].double() - want).norm() / want.norm())
                assert off <= 4e-3, (dtype, out, off)
            assert int(err) == 0


@pytest.mark.parametrize("kind", ["1/k", "1/k^2", "one far above", "rank one"])
@pytest.mark.parametrize("batch,m,n", [(1, 100, 300), (2, 120, 1100), (1, 300, 520),
                                       (1, 1000, 700), (1, 900, 6000)])
def test_singular_values_far_apart(batch, m, n, kind):
    """What a rounding adds is noise of 2^-12.3 of the matrix' 2-norm, which the steps magnify in
    the directions of small singular values, by the product of the a at most. The polynomial's and
    the gram's roundings give as much again a step, in steps after the first with fewer left: 2^-11
    times that product is held, beside what noise is held to."""
    x = matrices(kind, batch, m, n)
    for coefficients in (DEFAULT, SCHEDULES["tuned5"], SCHEDULES["tuned8"]):
        got = orthogonalize(x, coefficients=coefficients, out_dtype=torch.float16)
        grow = math.prod(a for a, _, _ in coefficients)
        for i in {0, batch - 1}:
            want = steps64(x[i], coefficients)
            off = float((got[i].double() - want).norm())
            assert off <= 1e-2 * float(want.norm()) + 2.0 ** -11 * grow, (off, float(want.norm()))


@pytest.mark.parametrize("m,n", [(100, 300), (300, 520), (700, 3000)])
def test_schedules_that_magnify_roundings_are_refused(m, n):
    x = matrices("noise", 1, m, n)
    for coefficients in (TUNED, TUNED8):
        with pytest.raises(FlceError, match="safety factor"):
            orthogonalize(x, coefficients=coefficients)
