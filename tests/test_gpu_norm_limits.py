"""What the norm's documentation says of sums beyond their type's range, and of rows that lie at
other addresses."""
import pytest
import torch

from linear_cross_entropy_vocab_gb300 import rms_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h", [64, 257, 4096, 20000])
def test_a_sum_beyond_float16(h):
    g = torch.Generator("cuda").manual_seed(h)
    x, r, dy = (torch.randn(5, h, generator=g, device="cuda").half() for _ in range(3))
    x[2, 7] = r[2, 7] = 6e4
    w = torch.rand(h, generator=g, device="cuda").half()
    for wide in (False, True):
        leaves = [t.clone().requires_grad_() for t in (x, r.float() if wide else r, w)]
        y, s = rms_norm(leaves[0], leaves[2], residual=leaves[1])
        s64 = x.double() + r.double()
        want = s64 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-6) * w.double()
        # products in 32 bits, and one rounding to float16 with its smallest step
        tol = want.abs() * (2.0 ** -11 + 2.0 ** -19) + 2.0 ** -25
        assert bool(((y.double() - want).abs() <= tol).all())
        assert bool(s[2, 7].isinf()) != wide
        gx, gr, gw = torch.autograd.grad(y, leaves, dy)
        others = [0, 1, 3, 4]
        columns = [c for c in range(h) if c != 7]
        assert bool(gx[others].isfinite().all()) and bool(gr[others].isfinite().all())
        assert bool(gw[columns].isfinite().all())
        assert bool(gx[2].isfinite().all()) == wide and bool(gr[2].isfinite().all()) == wide
        assert bool(gw[7].isfinite()) == wide


@pytest.mark.parametrize("h", [8, 1000, 4096, 16384])
def test_rows_at_other_addresses(h):
    """In fp32 a square's sum and the rounding of rstd may differ by 24 steps between the orders:
    up to 16 sums a thread and ten in the tree, halved by the root, and one each for the division
    and the products."""
    g = torch.Generator("cuda").manual_seed(h)
    base = torch.randn(6, h + 1, generator=g, device="cuda")
    view = base[:, 1:]
    a, b = rms_norm(view), rms_norm(view.contiguous())
    assert bool(((a - b).abs() <= 24 * 2.0 ** -24 * b.abs()).all())
