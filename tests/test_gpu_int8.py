"""The 8-bit linear layer against 64-bit products, and its quantisation bit for bit.

Tolerances. Integer products and sums up to 2^24 are exact; two products with the scales, the bias
and logit_scale round four times (2^-24 each of the magnitudes that meet there), the result once to
its type. Beyond 2^24 the sum over h may round at each of the h / 16 steps of the tensor core. The
softcap's tanh is within 1e-6 of the cap.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import int8_linear, quantize_rows

pytestmark = pytest.mark.gpu


def _quantize(x):
    """The definition in 32 bits on the host, where each operation rounds once."""
    x = x.float().cpu()
    peak = x.abs().amax(-1)
    scale = torch.where(torch.isfinite(peak), peak * (torch.ones(()) / 127.0), math.nan)
    s = scale.unsqueeze(-1)
    q = torch.where(s > 0, x / s, torch.zeros(())).nan_to_num().round().clamp(-127, 127)
    return q.to(torch.int8), scale


def _same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,h", [(1, 1), (3, 7), (5, 16), (130, 100), (2, 1023), (7, 1024),
                                 (3, 4096), (2, 4097), (3, 20001), (33, 255), (17, 256),
                                 (9, 257), (5, 2047), (6, 2048), (3, 2049), (1000, 40)])
def test_quantize(n, h, dtype):
    x = torch.randn(n, h, generator=torch.Generator().manual_seed(h)).to(dtype)
    q, scale = quantize_rows(x.cuda())
    wq, ws = _quantize(x)
    assert q.shape == (n, h) and scale.shape == (n,)
    assert torch.equal(scale.cpu(), ws) and torch.equal(q.cpu(), wq)
    assert q.stride(0) % 16 == 0 or n == 1


def test_quantize_edges():
    x = torch.randn(9, 50)
    x[0] = 0
    x[1, 3] = math.nan
    x[2, 4] = math.inf
    x[3, 5] = -math.inf
    x[4] = 3e38
    x[5] = 1e-38
    x[6] = torch.linspace(-127, 127, 50)
    x[7] = torch.arange(50) - 24.5  # halves
    x[7, 0] = 127.0
    x[8] = 1e-45
    q, scale = quantize_rows(x.cuda())
    wq, ws = _quantize(x)
    assert _same(scale.cpu(), ws)
    rows = [0, 4, 5, 6, 7]
    assert torch.equal(q.cpu()[rows], wq[rows])
    assert scale[0] == 0 and not bool(q[0].any())


def test_quantize_shapes_and_strides():
    base = torch.randn(6, 5, 40, device="cuda").bfloat16()
    for x in (base, base[:, 2], base[:, :, 3:20], base[0, 0], base.permute(2, 0, 1), base[:0],
              base[:, 0, 1:39]):
        q, scale = quantize_rows(x)
        assert q.shape == x.shape and scale.shape == x.shape[:-1]
        wq, ws = _quantize(x)
        assert torch.equal(q.cpu(), wq) and torch.equal(scale.cpu(), ws)


def _linear64(q, scale, wq, ws, bias=None, logit_scale=1.0, softcap=None):
    """(result, magnitude that the roundings are relative to, sum of |products|)"""
    acc = q.double() @ wq.double().t()
    gross = q.double().abs() @ wq.double().abs().t()
    f = scale.double().unsqueeze(-1) * ws.double()
    z, mag = acc * f, (acc * f).abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    z, mag = z * logit_scale, mag * abs(logit_scale)
    if softcap:
        z = softcap * torch.tanh(z / softcap)
    return z, mag, gross, (f * logit_scale).abs()


def _check(got, q, scale, wq, ws, bias=None, logit_scale=1.0, softcap=None):
    z, mag, gross, f = _linear64(q, scale, wq, ws, bias, logit_scale, softcap)
    h = q.shape[-1]
    tol = 5 * 2.0 ** -24 * mag + torch.finfo(got.dtype).eps / 2 * z.abs()
    tol = tol + torch.where(gross > 2.0 ** 24, (h / 16) * 2.0 ** -23 * gross * f, 0.0)
    if softcap:
        tol = tol + 1e-6 * softcap
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double() - z).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def _make(n, h, v, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + n + h + v)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    wq = torch.randint(-128, 128, (v, h), generator=g, device="cuda").to(torch.int8)
    ws = torch.rand(v, generator=g, device="cuda") * 0.01
    bias = torch.randn(v, generator=g, device="cuda")
    return x, wq, ws, bias


SIZES = [(1, 1, 1), (1, 16, 5), (3, 100, 130), (8, 64, 128), (16, 128, 129), (17, 96, 300),
         (32, 1024, 127), (33, 257, 1000), (64, 512, 256), (65, 80, 515), (128, 4096, 200),
         (129, 144, 640), (200, 1008, 333), (256, 64, 1024), (257, 112, 257), (500, 513, 700),
         (1030, 256, 400),
         (4700, 4096, 300)]  # more rows of x than run through the weight together


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,h,v", SIZES)
def test_linear(n, h, v, dtype):
    x, wq, ws, bias = _make(n, h, v, dtype)
    q, scale = quantize_rows(x)
    got = int8_linear(x, wq, ws)
    assert got.dtype == dtype and got.shape == (n, v)
    _check(got, q, scale, wq, ws)
    got = int8_linear(x, wq, ws, bias.to(dtype), logit_scale=0.7, softcap=20.0,
                      out_dtype=torch.float32)
    _check(got, q, scale, wq, ws, bias.to(dtype), 0.7, 20.0)
    # rows that were quantised before give the same as rows quantised within
    assert torch.equal(int8_linear(q, wq, ws, x_scale=scale, out_dtype=dtype),
                       int8_linear(x, wq, ws))


@pytest.mark.parametrize("h", [1, 15, 16, 17, 63, 64, 65, 127, 1000, 1001])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_pitches_and_addresses(n, h):
    """Weight rows padded, dense at any length, and starting at odd addresses."""
    x, wq, ws, bias = _make(n, h, 301, torch.bfloat16)
    q, scale = quantize_rows(x)
    want = int8_linear(x, wq, ws, bias)
    _check(want, q, scale, wq, ws, bias)
    wide = torch.full((301, (h + 31) // 16 * 16), 99, dtype=torch.int8, device="cuda")
    wide[:, :h] = wq
    assert torch.equal(int8_linear(x, wide[:, :h], ws, bias), want)
    flat = torch.full((301 * h + 64,), 99, dtype=torch.int8, device="cuda")
    odd = flat[3:3 + 301 * h].view(301, h)
    odd.copy_(wq)
    assert torch.equal(int8_linear(x, odd, ws, bias), want)
    assert torch.equal(int8_linear(x, wq.t().contiguous().t(), ws, bias), want)
    xs = torch.zeros(n, h + 5, dtype=torch.bfloat16, device="cuda")
    xs[:, 1:h + 1] = x
    assert torch.equal(int8_linear(xs[:, 1:h + 1], wq, ws, bias), want)
    qs = torch.full((n, h + 7), 77, dtype=torch.int8, device="cuda")
    qs[:, 3:h + 3] = q
    assert torch.equal(int8_linear(qs[:, 3:h + 3], wq, ws, bias, x_scale=scale,
                                   out_dtype=torch.bfloat16), want)


def test_extremes():
    """Every product at its largest, of one sign and of both."""
    for h in (1024, 4096, 20000):
        q = torch.full((5, h), 127, dtype=torch.int8, device="cuda")
        wq = torch.full((140, h), -128, dtype=torch.int8, device="cuda")
        wq[::2] = 127
        wq[1::4, ::2] = 127
        one, ws = torch.ones(5, device="cuda"), torch.ones(140, device="cuda")
        _check(int8_linear(q, wq, ws, x_scale=one), q, one, wq, ws)


def test_special_rows():
    x, wq, ws, bias = _make(6, 200, 300, torch.float32)
    x[0] = 0
    x[1, 7] = math.nan
    x[2, 8] = math.inf
    got = int8_linear(x, wq, ws, bias)
    assert torch.equal(got[0], bias)
    assert bool(got[1].isnan().all()) and bool(got[2].isnan().all())
    assert not bool(got[3:].isnan().any())
    q, scale = quantize_rows(x)
    _check(got[3:], q[3:], scale[3:], wq, ws, bias)


def test_shapes():
    x, wq, ws, bias = _make(24, 64, 100, torch.bfloat16)
    want = int8_linear(x, wq, ws)
    assert torch.equal(int8_linear(x.view(2, 3, 4, 64), wq, ws), want.view(2, 3, 4, 100))
    assert torch.equal(int8_linear(x[5], wq, ws), want[5])
    assert int8_linear(x[:0], wq, ws).shape == (0, 100)
    assert int8_linear(x, wq[:0], ws[:0]).shape == (24, 0)
    q, scale = quantize_rows(x.view(4, 6, 64))
    got = int8_linear(q, wq, ws, x_scale=scale)
    assert got.shape == (4, 6, 100) and got.dtype == torch.float32


def test_streams_and_graph():
    x, wq, ws, bias = _make(20, 512, 2000, torch.bfloat16)
    first = int8_linear(x, wq, ws, bias.bfloat16())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [int8_linear(x, wq, ws, bias.bfloat16()) for _ in range(10)]
    side.synchronize()
    assert all(torch.equal(first, a) for a in again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = int8_linear(x, wq, ws)
    for seed in range(3):
        x.copy_(_make(20, 512, 2000, torch.bfloat16, seed=seed + 1)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, int8_linear(x, wq, ws))


def test_close_to_the_unquantised_head():
    """What the layer is for: a head's logits, within what 8 bits lose."""
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(50, 512, generator=g, device="cuda").bfloat16()
    w = (torch.randn(1000, 512, generator=g, device="cuda") * 512 ** -0.5).bfloat16()
    wq, ws = quantize_rows(w)
    got = int8_linear(x, wq, ws, out_dtype=torch.float32).double()
    want = x.double() @ w.double().t()
    # steps of about 3.5 / 127 on both sides, each off by a uniform half step at most
    assert float((got - want).norm() / want.norm()) < 2 * 3.5 / 127 / math.sqrt(12) * 1.5


def test_refusals():
    x, wq, ws, bias = _make(4, 32, 50, torch.bfloat16)
    with pytest.raises(RuntimeError, match="no gradient"):
        int8_linear(x.clone().requires_grad_(True), wq, ws)
    with torch.no_grad():
        int8_linear(x.clone().requires_grad_(True), wq, ws)
    with pytest.raises(ValueError):
        int8_linear(x, wq, ws, x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        int8_linear(quantize_rows(x)[0], wq, ws)
    with pytest.raises(TypeError):
        int8_linear(x, wq.float(), ws)
    with pytest.raises(ValueError):
        int8_linear(x, wq[:, :31], ws)
    with pytest.raises(ValueError):
        int8_linear(x, wq, ws[:49])
    with pytest.raises(ValueError):
        int8_linear(x, wq, ws, bias[:49])
    with pytest.raises(ValueError):
        int8_linear(x, wq.cpu(), ws)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [6, 300])  # one CTA a tile, and pairs
def test_softcap_keeps_nan(n, out_dtype):
    """A NaN anywhere in a logit stays NaN under the cap; the other logits are the capped ones,
    large ones of either sign among them."""
    x, wq, ws, bias = _make(n, 200, 300, torch.float32)
    x[1, 7] = math.nan
    x[2, 8] = math.inf
    x[3] *= 1e6
    ws[40] = math.nan
    bias[50] = math.nan
    got = int8_linear(x, wq, ws, bias, softcap=20.0, out_dtype=out_dtype)
    rows = torch.arange(n, device="cuda")
    rows = (rows != 1) & (rows != 2)
    cols = torch.arange(300, device="cuda")
    cols = (cols != 40) & (cols != 50)
    assert bool(got[~rows].isnan().all()) and bool(got[:, ~cols].isnan().all())
    q, scale = quantize_rows(x)
    _check(got[rows][:, cols], q[rows], scale[rows], wq[cols], ws[cols], bias[cols], softcap=20.0)
    assert bool((got[3, cols] > 19.9).any()) and bool((got[3, cols] < -19.9).any())
    scale[4] = math.nan
    got = int8_linear(q, wq, ws, bias, x_scale=scale, softcap=20.0, out_dtype=out_dtype)
    assert bool(got[4].isnan().all())


@pytest.mark.parametrize("n", [1, 40, 300])
def test_scales_of_this_call(n):
    """Calls in a row whose scales take the same places in memory: each uses those that it made
    itself. The layer's kernel starts while the one that writes them still runs."""
    _, wq, ws, bias = _make(n, 96, 500, torch.float32)
    inputs = [_make(n, 96, 1, torch.float32, seed=i)[0] * 10.0 ** (i % 7 - 3) for i in range(40)]
    want = []
    for x in inputs:
        q, scale = quantize_rows(x)
        want.append(int8_linear(q, wq, ws, bias, x_scale=scale))
    torch.cuda.synchronize()
    got = [int8_linear(x, wq, ws, bias) for x in inputs]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [5, 300])
@pytest.mark.parametrize("size", [1e-6, 1e-3, 0.1, 1.0])
def test_softcap_of_small_logits(size, n):
    """Logits far below the cap keep their own precision: z rounds twice, its share of the cap
    twice, the product with the cap once (2^-24 each, none of which tanh magnifies), and tanh is
    within 10 * 2^-24: its rational form, evaluated in 32 bits over 2.2 million places on the
    host, is within 5, and the approximate reciprocal adds 2."""
    x, wq, ws, _ = _make(n, 128, 400, torch.float32)
    q, scale = quantize_rows(x)
    cap = 30.0
    ws = ws * (size * cap / float(((q.double() @ wq.double().t()) * scale.double().unsqueeze(-1)
                                  * ws.double()).abs().max()))
    z, _, gross, _ = _linear64(q, scale, wq, ws, softcap=cap)
    assert float(gross.max()) <= 2.0 ** 24  # the sums are exact
    got = int8_linear(x, wq, ws, softcap=cap).double()
    assert bool(((got - z).abs() <= 15 * 2.0 ** -24 * z.abs()).all())
    half = int8_linear(x, wq, ws, softcap=cap, out_dtype=torch.bfloat16).double()
    assert bool(((half - z).abs() <= (2.0 ** -8 + 16 * 2.0 ** -24) * z.abs()).all())
