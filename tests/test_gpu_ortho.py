"""Orthogonalised matrices against the steps in 64 bits.

Tolerance. Sums are held in 32 bits and everything else that is computed is rounded to halves where
the kernels store it: the copy, the grams, the polynomials and what gathers them, x after a group of
steps, and the result. The steps magnify those roundings, by an amount that depends on the matrix.
So the same steps are done in 64 bits with each of these roundings, and the kernel's error is held
to 1.5 times the error that they make: it makes the same roundings, but for those of sums whose
32-bit error (k / 16 * 2^-23 of k products' magnitudes, against 2^-11 of a half) takes them across
the border between two halves. Single entries are held to 16 times the mean of that bound.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import (clip_grads_, fused_linear_cross_entropy,
                                              orthogonalize, rms_norm)
from linear_cross_entropy_vocab_gb300.abi import FlceError
from linear_cross_entropy_vocab_gb300.ortho import NEWTON_SCHULZ

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _groups(steps, together):
    """How many steps each gram serves: three, and two at the end."""
    sizes = []
    while sum(sizes) < steps:
        left = steps - sum(sizes)
        sizes.append(1 if not together else 2 if left == 4 else min(3, left))
    return sizes


def _shares_grams(batch, m, n):
    """The kernels' rule for steps that share a gram (sides of more than 128)."""
    m, n = sorted((m, n))
    return m > 128 and batch * m * m * (n - m) > 4e9


def _half(t, bound):
    """Halves with the power of two that takes values up to ``bound`` to 2^13 to 2^14."""
    scale = 2.0 ** (14 - math.frexp(bound)[1])
    return (t * scale).to(torch.float16).double() / scale


def _steps64(g, coefficients, eps, out_dtype, together, round_=True):
    """The steps with the kernels' roundings, or without any."""
    half = _half if round_ else lambda t, bound: t
    g = g.double()
    norm = torch.linalg.matrix_norm(g) + eps
    near = 2.0 ** math.floor(math.log2(float(norm)))  # the factor below is applied to sums
    x = g.t() if g.shape[0] > g.shape[1] else g
    x = half(x / near, 1.0) * (near / norm)
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    top, k = 1.0, 0
    for size in _groups(len(coefficients), together):
        gram = half(x @ x.t(), top * top)
        gathered, all_ = None, 1.0
        for s in range(size):
            a, b, c = coefficients[k]
            k += 1
            t = torch.linspace(0, top, 4001, dtype=torch.float64)
            q = float((a + b * t ** 2 + c * t ** 4).abs().max()) * 65 / 64
            p = half(a * eye + b * gram + c * (gram @ gram), q)
            new = float((t * (a + b * t ** 2 + c * t ** 4)).abs().max()) * 65 / 64
            if s + 1 < size:
                gram = half(half(p @ gram, q * top * top) @ p, new * new)
            all_ *= q
            gathered = p if gathered is None else half(p @ gathered, all_)
            top = new
        x = gathered @ x
        if k < len(coefficients):
            x = half(x, top)
    x = x.t() if g.shape[0] > g.shape[1] else x
    return x.to(out_dtype).double() if round_ else x


def _bound(g, coefficients, eps, out_dtype, together):
    """(result, bound on the 2-norm of the result's error) for one matrix."""
    want = _steps64(g, coefficients, eps, out_dtype, False, False)
    err = float((_steps64(g, coefficients, eps, out_dtype, together) - want).norm())
    # what halves cannot hold beside the largest values, and results below the type's smallest
    floor = 2.0 ** -25 * math.sqrt(want.numel())
    return want, 1.5 * err + floor


def _check(got, g, coefficients=NEWTON_SCHULZ, eps=1e-7, batch=1, spread=True):
    together = _shares_grams(batch, *g.shape)
    want, delta = _bound(g, coefficients, eps, got.dtype, together)
    err = got.double() - want
    assert float(err.norm()) <= delta, (float(err.norm()), delta, float(want.norm()))
    # a matrix whose error lies in few entries has no such mean: one entry can hold all of it
    assert not spread or float(err.abs().max()) <= 16 * delta / math.sqrt(want.numel())
    assert delta < 0.03 * float(want.norm()) + 1e-3


def _matrices(batch, m, n, dtype, seed=0, scale=1e-3):
    g = torch.Generator("cuda").manual_seed(seed + 7 * m + n)
    return (torch.randn(batch, m, n, generator=g, device="cuda") * scale).to(dtype)


SIZES = [(1, 1, 1), (1, 1, 9), (2, 5, 3), (1, 64, 64), (3, 100, 300), (1, 300, 100), (2, 256, 256),
         (1, 257, 511), (1, 130, 1000), (2, 513, 700), (1, 1000, 260), (5, 96, 64), (1, 1024, 600),
         (1, 64, 5000), (1, 3000, 33), (40, 16, 200), (1, 770, 1300),
         # one side in shared memory, in clusters of 1 to 8, and just not
         (1, 128, 512), (2, 128, 513), (3, 1500, 100), (1, 128, 4096), (2, 4090, 65), (1, 7, 4097),
         (2, 129, 600), (300, 8, 24),
         # tiles of 128 in two rounds, some cut, and just tiles of 256
         (1, 1300, 2500), (2, 1900, 1200), (1, 2300, 2200),
         # steps that share a gram
         (4, 3000, 700), (1, 1000, 5100), (30, 200, 4100),
         # tiles whose contraction is cut between CTAs: few, or more than a round
         (1, 1024, 2100), (4, 4000, 700), (90, 20, 1000), (80, 300, 900), (30, 100, 3000),
         (1, 300, 20000), (1, 400, 40000), (20, 640, 500),
         # tiles of 256, some in a batch, with steps that share a gram and without
         (8, 1000, 1000), (8, 1000, 2700), (2, 2701, 2050), (1, 4100, 2300), (17, 700, 4000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,m,n", SIZES)
def test_against_64_bits(batch, m, n, dtype):
    x = _matrices(batch, m, n, dtype)
    got = orthogonalize(x)
    assert got.shape == x.shape and got.is_contiguous()
    assert got.dtype == (torch.bfloat16 if dtype == torch.float32 else dtype)
    for i in {0, batch // 2, batch - 1}:
        _check(got[i], x[i], batch=batch)
    # matrices of a batch do not meet (alone, their sums may be cut elsewhere)
    for i in {0, batch - 1}:
        others = torch.full_like(x, math.nan)
        others[i] = x[i]
        assert torch.equal(got[i], orthogonalize(others)[i])
    assert torch.equal(got, orthogonalize(x))
    other = torch.float16 if got.dtype == torch.bfloat16 else torch.bfloat16
    got = orthogonalize(x, out_dtype=other)
    assert got.dtype == other
    _check(got[0], x[0], batch=batch)


@pytest.mark.parametrize("m,n", [(70, 200), (300, 128), (257, 300)])
def test_other_steps(m, n):
    x = _matrices(1, m, n, torch.float32)
    for coefficients in (((3.4445, -4.7750, 2.0315),), ((1.5, -0.5, 0.0),) * 2,
                         ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)),
                         ((0.01, 0.0, 0.0),), ((15.0, -20.0, 8.0), (0.5, 0.0, 0.001))):
        got = orthogonalize(x[0], coefficients=coefficients, eps=1e-3)
        _check(got, x[0], coefficients, 1e-3)
    # the first step's values reach 5.4, the second would take them to 45
    with pytest.raises(FlceError, match="singular values"):
        orthogonalize(x[0], coefficients=((15.0, -20.0, 8.0), (0.5, 0.0, 0.01)))
    # many steps end at an orthogonal matrix: singular values at 1, to the rounding of their place
    got = orthogonalize(x[0], coefficients=((1.5, -0.5, 0.0),) * 40, out_dtype=torch.float16)
    values = torch.linalg.svdvals(got.double())
    assert float((values - 1).abs().max()) < 2e-2


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 8])
def test_numbers_of_steps(steps):
    coefficients = tuple((3.0 - 0.2 * k, -3.5 + 0.3 * k, 1.4 - 0.1 * k) for k in range(steps))
    for x in (_matrices(3, 600, 5000, torch.bfloat16), _matrices(1, 300, 400, torch.bfloat16),
              _matrices(8, 1000, 2700, torch.bfloat16), _matrices(8, 1000, 1000, torch.bfloat16),
              _matrices(1, 100, 1000, torch.bfloat16)):
        _check(orthogonalize(x, coefficients=coefficients)[0], x[0], coefficients, batch=len(x))


def test_addresses_and_strides():
    base = _matrices(6, 130, 400, torch.bfloat16)
    views = [base[:, :, 1:301], base[1::2], base[:, ::3], base[:, :100, 8:308], base.transpose(1, 2),
             base[0], base[0, :, 1:200], base.view(2, 3, 130, 400), base[:1].expand(3, 130, 400),
             base[:, :1], base[:, :, :1], base.permute(1, 0, 2)]
    for x in views:
        got = orthogonalize(x)
        assert got.shape == x.shape
        flat, gots = x.reshape(-1, *x.shape[-2:]), got.view(-1, *x.shape[-2:])
        for i in range(min(2, len(flat))):
            _check(gots[i], flat[i])
        # not bit for bit what a dense copy gives: the squares of rows with a pitch are added in
        # another order, by which the norm's factor may differ in its last place (2^-24), and then
        # values next to a border of the halves round the other way, once for each rounding
        same = orthogonalize(x.contiguous())
        _, delta = _bound(flat[0], NEWTON_SCHULZ, 1e-7, got.dtype, False)
        again = same.view(-1, *x.shape[-2:])[0].double()
        assert float((gots[0].double() - again).norm()) <= 2 * delta
    for shape in ((0, 5, 6), (3, 0, 6), (3, 6, 0), (2, 0, 4, 4)):
        assert orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_what_surrounds_the_result_stays():
    """Sizes that end inside a tile: nothing is written past the result."""
    for m, n in ((100, 300), (300, 100), (33, 257), (700, 99), (130, 257), (300, 400)):
        x = _matrices(2, m, n, torch.bfloat16)
        want = orthogonalize(x)
        import linear_cross_entropy_vocab_gb300.ortho as ortho
        room = torch.full((2 * m * n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        empty = torch.empty

        def placed(*a, **k):
            if a and tuple(a[0]) == (2, m, n) if isinstance(a[0], (tuple, torch.Size)) else False:
                return room[2048:2048 + 2 * m * n].view(2, m, n)
            return empty(*a, **k)

        try:
            ortho.torch.empty = placed
            got = orthogonalize(x)
        finally:
            ortho.torch.empty = empty
        assert torch.equal(got, want) and got.data_ptr() == room[2048:].data_ptr()
        assert bool((room[:2048] == 7).all()) and bool((room[2048 + 2 * m * n:] == 7).all())


@pytest.mark.parametrize("m,n", [(90, 200), (90, 900), (150, 200)])
def test_extremes(m, n):
    x = _matrices(9, m, n, torch.float32, scale=1.0)
    x[0] = 0
    x[1] *= 1e36
    x[2] *= 1e-36
    x[3, 5, 7] = math.nan
    x[4, 0, 0] = math.inf
    x[5] = 0
    x[5, 3, 4] = -2.0
    x[6, 1:] = 0
    x[7] *= 1e-3
    x[7, 0, 0] = 1e30
    got = orthogonalize(x)
    assert not bool(got[0].any())
    for i in (1, 2, 5, 6, 8):
        _check(got[i], x[i], spread=i not in (5, 6))
    assert bool(got[3].isnan().all()) and bool(got[4].isnan().all())
    assert bool(got[7].isfinite().all()) and abs(float(got[7, 0, 0])) > 0.6
    # an eps beside the norm
    got = orthogonalize(x[8:] * 1e-6, eps=1e-4)
    _check(got[0], x[8] * 1e-6, eps=1e-4)
    # numbers that halves cannot hold well
    tiny = _matrices(1, 64, 64, torch.float16, scale=1e-6)
    _check(orthogonalize(tiny)[0], tiny[0])


@pytest.mark.parametrize("m,n", [(300, 520), (100, 1100), (2000, 2200)])
def test_streams_and_graphs(m, n):
    x = _matrices(2, m, n, torch.bfloat16)
    want = orthogonalize(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = orthogonalize(x)
    other = orthogonalize(x.transpose(1, 2))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graphs, outs, ins = [], [], []
    for i in range(2):
        ins.append(x.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(orthogonalize(ins[i] if i == 0 else ins[i].transpose(1, 2)))
    for seed in (3, 4):
        nx = _matrices(2, m, n, torch.bfloat16, seed)
        for i in range(2):
            ins[i].copy_(nx)
            graphs[i].replay()
        assert torch.equal(outs[0], orthogonalize(nx))
        assert torch.equal(outs[1], orthogonalize(nx.transpose(1, 2)))
    assert torch.equal(other, orthogonalize(x.transpose(1, 2)))


def test_a_training_step():
    """Norm, head, clip and update as a training step has them, against the same in 64 bits."""
    g = torch.Generator("cuda").manual_seed(3)
    n, h, v = 200, 128, 1000

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    x, r, w = rand(n, h), rand(n, h), 1 + rand(h, std=0.1)
    mix, head = rand(h, h, std=h ** -0.5), rand(v, h, std=h ** -0.5)
    targets = torch.randint(0, v, (n,), generator=g, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (mix, head, w)]
    y, _ = rms_norm(x @ leaves[0].t(), leaves[2], residual=r)
    fused_linear_cross_entropy(y, leaves[1], targets).backward()
    ref = [t.double().requires_grad_() for t in (mix, head, w)]
    s = (x @ mix.t()).double() + r.double()  # the product as it was rounded, with its gradient
    s = s + x.double() @ ref[0].t() - (x.double() @ ref[0].t()).detach()
    yy = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * ref[2]
    torch.nn.functional.cross_entropy(yy @ ref[1].t(), targets).backward()
    for a, b in zip(leaves, ref):
        # bf16 on the way: y, the gradients of the logits and of y, and the product's
        assert float((a.grad.double() - b.grad).norm()) <= 4 * 2.0 ** -8 * float(b.grad.norm())
    clip_grads_([t.grad for t in leaves], 1e-3)
    update = orthogonalize(leaves[0].grad)
    _check(update, leaves[0].grad)


def test_refusals_of_gradients():
    x = _matrices(1, 20, 30, torch.float32)[0].requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        orthogonalize(x)
    with torch.no_grad():
        orthogonalize(x)
