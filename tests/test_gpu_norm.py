"""The root-mean-square norm with the residual's addition against its formulas in 64 bits.

Tolerances, in units of 2^-24 of the magnitudes that meet: the sum x + residual rounds once, each
thread adds up to 16 squares a sweep and the team's tree ten more, and their errors reach rstd by
half; three products follow. That is below 32 for rows of one sweep (16384 values), one more for
each further sweep. The gradient's mean has the same tree over products of three factors, and the
result two more products and sums: below 64 of |grad_sum| + rstd (|u| + |unit| mean|u unit|). A sum
over rows is added by CTAs of n / 152 rows at least and 32 warps after them. The result is rounded
once to its type. The references read the stored sum where the backward does.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import (int8_linear, quantize_rows, rms_norm,
                                              rms_norm_quantize)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [(1, 1), (3, 7), (5, 64), (130, 100), (2, 256), (33, 257), (7, 1000), (9, 1024), (4, 1025),
         (3, 2048), (5, 2049), (6, 4096), (3, 4097), (2, 8192), (3, 8193), (2, 16384), (2, 16385),
         (3, 40000), (1000, 40), (700, 512), (2500, 136)]


def _step(t):
    return torch.finfo(t).eps / 2


def _tiny(t):
    """Half the distance of the type's smallest numbers."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[t]


def _inputs(n, h, dtype, residual, seed=0, weight=True):
    g = torch.Generator("cuda").manual_seed(seed + 31 * n + h)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    r = None if residual is None else (3 * torch.randn(n, h, generator=g, device="cuda")).to(
        residual)
    w = (1 + 0.3 * torch.randn(h, generator=g, device="cuda")).to(dtype) if weight else None
    return x, r, w


def _forward64(x, r, w, eps):
    s = x.double() if r is None else x.double() + r.double()
    rstd = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, rstd, s * rstd * (1.0 if w is None else w.double())


def _within(got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def _check_forward(x, r, w, eps, y, total):
    s, _, want = _forward64(x, r, w, eps)
    if r is not None:
        assert torch.equal(total, (x.float() + r.float()).to(r.dtype))
    rel = (32 + x.shape[-1] / 16384) * U
    _within(y, want, want.abs() * (rel + _step(y.dtype)) + _tiny(y.dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", SIZES)
def test_forward(n, h, dtype):
    for residual in {None, dtype, torch.float32}:
        for weight in (True, False):
            x, r, w = _inputs(n, h, dtype, residual, weight=weight)
            got = rms_norm(x, w, 1e-6, residual=r)
            y, total = got if r is not None else (got, None)
            assert y.dtype == dtype and y.shape == (n, h)
            _check_forward(x, r, w, 1e-6, y, total)
    x, r, w = _inputs(n, h, dtype, dtype)
    y, total = rms_norm(x, w.float() * 1.0001, 0.5, residual=r)  # a weight in 32 bits
    _check_forward(x, r, w.float() * 1.0001, 0.5, y, total)


def _check_backward(x, r, w, eps, dy, ds, total, grads):
    s, rstd, _ = _forward64(x, r, w, eps)
    unit = (s if r is None else total.double()) * rstd
    u = dy.double() * (1.0 if w is None else w.double())
    mean = (u * unit).mean(-1, keepdim=True)
    grad = rstd * (u - unit * mean)
    mag = rstd * (u.abs() + unit.abs() * (u * unit).abs().mean(-1, keepdim=True))
    if ds is not None:
        grad, mag = grad + ds.double(), mag + ds.double().abs()
    tol = (64 + x.shape[-1] / 16384) * U * mag
    for name, got in grads.items():
        if name != "weight":
            _within(got, grad, tol + _step(got.dtype) * grad.abs() + _tiny(got.dtype))
    if w is not None:
        want, gross = (dy.double() * unit).sum(0), (dy.double() * unit).abs().sum(0)
        got = grads["weight"]
        n = x.shape[0]
        # shares: of rows too long for a CTA's registers 16
        rows = n / 16 if x.shape[-1] > 16384 else n / 152
        _within(got, want, (rows + 64) * U * gross + _step(got.dtype) * want.abs()
                + _tiny(got.dtype))


def _backward(x, r, w, dy, ds, eps=1e-6):
    leaves = {"x": x, "residual": r, "weight": w}
    leaves = {k: v.clone().requires_grad_() for k, v in leaves.items() if v is not None}
    got = rms_norm(leaves["x"], leaves.get("weight"), eps, residual=leaves.get("residual"))
    y, total = got if r is not None else (got, None)
    outs, ups = ([y], [dy]) if ds is None else ([y, total], [dy, ds])
    grads = torch.autograd.grad(outs, list(leaves.values()), ups)
    for leaf, grad in zip(leaves.values(), grads):
        assert grad.dtype == leaf.dtype and grad.shape == leaf.shape
    return y.detach(), None if total is None else total.detach(), dict(zip(leaves, grads))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", SIZES)
def test_backward(n, h, dtype):
    for residual in {None, dtype, torch.float32}:
        for weight in (True, False):
            x, r, w = _inputs(n, h, dtype, residual, 5, weight)
            g = torch.Generator("cuda").manual_seed(n + h)
            dy = torch.randn(n, h, generator=g, device="cuda").to(dtype)
            ds = None if r is None else torch.randn(n, h, generator=g, device="cuda").to(residual)
            for up in {None, ds}:
                y, total, grads = _backward(x, r, w, dy, up)
                _check_forward(x, r, w, 1e-6, y, total)
                _check_backward(x, r, w, 1e-6, dy, up, total, grads)


def test_backward_of_many_rows():
    x, r, w = _inputs(20011, 264, torch.bfloat16, torch.bfloat16)
    dy, ds = torch.randn_like(x), torch.randn_like(x)
    _, total, grads = _backward(x, r, w, dy, ds)
    _check_backward(x, r, w, 1e-6, dy, ds, total, grads)
    again = _backward(x, r, w, dy, ds)[2]
    assert all(torch.equal(grads[k], again[k]) for k in grads)
    assert grads["x"].data_ptr() == grads["residual"].data_ptr()  # one tensor for both


@pytest.mark.parametrize("h", [64, 513, 2050, 17000])
def test_backward_against_differences(h):
    """The derivative along random directions, from 64-bit differences of the formula."""
    x, r, w = _inputs(6, h, torch.float32, torch.float32)
    dy, ds = torch.randn_like(x), torch.randn_like(x)
    grads = _backward(x, r, w, dy, ds)[2]

    def value(x, r, w):
        s, _, y = _forward64(x, r, w, 1e-6)
        return float((y * dy.double()).sum() + (s * ds.double()).sum())

    inputs = {"x": x.double(), "residual": r.double(), "weight": w.double()}
    for name in inputs:
        along = torch.randn_like(inputs[name])
        step = 1e-5
        up, down = (value(**{**{k[0] if k != "residual" else "r": v for k, v in inputs.items()},
                             (name[0] if name != "residual" else "r"): inputs[name] + d * along})
                    for d in (step, -step))
        want = (up - down) / (2 * step)
        got = float((grads[name].double() * along).sum())
        # differences: step^2 times a third derivative, and 2^-53 of the value over the step;
        # the gradient: 64 * 2^-24 of each entry's magnitude
        mag = float((grads[name].double().abs() * along.abs()).sum())
        assert abs(got - want) <= 1e-5 * mag + 1e-5, (name, got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,h", SIZES)
def test_quantize(n, h, dtype):
    for residual in {None, dtype, torch.float32}:
        x, r, w = _inputs(n, h, dtype, residual, 9)
        got = rms_norm_quantize(x, w, 1e-6, residual=r)
        q, scale = got[:2]
        assert q.dtype == torch.int8 and q.shape == (n, h) and scale.shape == (n,)
        if r is not None:
            assert torch.equal(got[2], (x.float() + r.float()).to(r.dtype))
        # in 32 bits the norm's own output is what is quantised
        wide = rms_norm(x.float(), w.float(), 1e-6, residual=None if r is None else r.float())
        wide = wide if r is None else wide[0]
        want_q, want_scale = quantize_rows(wide)
        assert torch.equal(scale, want_scale) and torch.equal(q, want_q)
        _, _, y = _forward64(x, r, w, 1e-6)
        tol = 0.5 * scale.double()[:, None] + y.abs() * 64 * U
        _within(q.double() * scale.double()[:, None], y, tol)
        assert q.stride(0) % 16 == 0 or n == 1


def test_shapes_and_strides():
    base = torch.randn(6, 5, 48, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        b = base.to(dtype)
        for x in (b, b[:, 2], b[:, :, 3:20], b[0, 0], b.permute(2, 0, 1), b[:0], b[:, 0, 1:41],
                  b[:, 0, 8:40], b.transpose(1, 2)[..., :3], b[0].expand(7, 5, 48)):
            w = torch.randn(2 * x.shape[-1], device="cuda").to(dtype)[::2]
            r = torch.randn(x.shape, device="cuda").to(dtype)
            for residual in (None, r, r.transpose(0, -1).contiguous().transpose(0, -1)):
                got = rms_norm(x, w, residual=residual)
                y = got if residual is None else got[0]
                assert y.shape == x.shape and y.is_contiguous()
                if y.numel():
                    _check_forward(x, residual, w, 1e-6, y, None if residual is None else got[1])
                q, scale = rms_norm_quantize(x, w, residual=residual)[:2]
                assert q.shape == x.shape and scale.shape == x.shape[:-1]
                if residual is None and dtype == torch.float32:
                    want = quantize_rows(y)
                    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])
    # upstream gradients that are views
    x, r, w = _inputs(40, 96, torch.bfloat16, torch.bfloat16)
    dy = torch.randn(96, 40, device="cuda").bfloat16().t()
    ds = torch.randn(1, 96, device="cuda").bfloat16().expand(40, 96)
    _, total, grads = _backward(x, r, w, dy, ds)
    _check_backward(x, r, w, 1e-6, dy, ds, total, grads)
    # odd addresses
    flat = torch.randn(40 * 96 + 1, device="cuda").bfloat16()
    _, total, grads = _backward(flat[1:].view(40, 96), r, w, dy, ds)
    _check_backward(flat[1:].view(40, 96), r, w, 1e-6, dy, ds, total, grads)


def test_no_rows():
    x = torch.empty(0, 96, device="cuda").bfloat16()
    w = torch.ones(96, device="cuda").bfloat16()
    y, total, grads = _backward(x, x, w, x, x)
    assert y.shape == total.shape == (0, 96) and grads["x"].shape == (0, 96)
    assert grads["weight"].shape == (96,) and not bool(grads["weight"].any())
    q, scale = rms_norm_quantize(x, w)
    assert q.shape == (0, 96) and scale.shape == (0,)


@pytest.mark.parametrize("h", [200, 4096, 17000])
def test_extremes(h):
    x = torch.randn(8, h, device="cuda")
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-25
    x[3, h // 2] = math.nan
    x[4, 1] = math.inf
    x[5, h - 1] = -math.inf
    x[6] *= 1e18
    for eps in (1e-6, 1e-37):
        y = rms_norm(x, None, eps)
        fine = [0, 1, 2, 6, 7]
        _check_forward(x[fine], None, None, eps, y[fine], None)
        assert bool(y[3].isnan().all())
        # inf / inf, and everything else over infinity
        assert bool(y[4, 1].isnan()) and not bool(y[4, 2:].any())
        assert bool(y[5, h - 1].isnan()) and not bool(y[5, :h - 1].any())
        q, scale = rms_norm_quantize(x, None, eps)
        want_q, want_scale = quantize_rows(y)
        assert torch.equal(scale.isnan(), want_scale.isnan())
        assert torch.equal(scale.nan_to_num(), want_scale.nan_to_num())
        assert torch.equal(q[fine], want_q[fine])
        assert scale.isnan().tolist() == [False, False, False, True, True, True, False, False]


def test_some_gradients_only():
    x, r, w = _inputs(50, 520, torch.bfloat16, torch.float32)
    dy, ds = torch.randn_like(x), torch.randn(50, 520, device="cuda")
    full = _backward(x, r, w, dy, ds)[2]
    for names in (["x"], ["residual"], ["weight"], ["x", "weight"], ["residual", "weight"]):
        leaves = {"x": x, "residual": r, "weight": w}
        leaves = {k: v.clone().requires_grad_(k in names) for k, v in leaves.items()}
        y, total = rms_norm(leaves["x"], leaves["weight"], residual=leaves["residual"])
        got = torch.autograd.grad([y, total], [leaves[k] for k in names], [dy, ds],
                                  allow_unused=True)
        for k, v in zip(names, got):
            assert torch.equal(v, full[k])
    # the sum alone: its gradient passes through
    leaves = [v.clone().requires_grad_() for v in (x, r, w)]
    _, total = rms_norm(leaves[0], leaves[2], residual=leaves[1])
    gx, gr, gw = torch.autograd.grad(total, leaves, ds)
    assert torch.equal(gx, ds.bfloat16()) and torch.equal(gr, ds) and not bool(gw.any())


def test_one_tensor_in_two_places():
    x, _, w = _inputs(30, 264, torch.float32, torch.float32)
    dy, ds = torch.randn_like(x), torch.randn_like(x)
    want = _backward(x, x.clone(), w, dy, ds)[2]
    leaf, gain = x.clone().requires_grad_(), w.clone().requires_grad_()
    y, total = rms_norm(leaf, gain, residual=leaf)
    gx, gw = torch.autograd.grad([y, total], [leaf, gain], [dy, ds])
    assert torch.equal(gx, 2 * want["x"]) and torch.equal(gw, want["weight"])
    # accumulated into leaves, twice: the shared gradient is not written to
    leaves = [t.clone().requires_grad_() for t in (x, x, w)]
    for _ in range(2):
        y, total = rms_norm(leaves[0], leaves[2], residual=leaves[1])
        torch.autograd.backward([y, total], [dy, ds])
    assert torch.equal(leaves[0].grad, 2 * want["x"])
    assert torch.equal(leaves[1].grad, 2 * want["x"])
    # one after the other, through the stream
    y, total = rms_norm(leaf, gain, residual=x)
    y2, total2 = rms_norm(y, gain, residual=total)
    g = torch.autograd.grad([y2, total2], leaf, [dy, ds])[0]
    l64 = x.double().requires_grad_()
    s1 = l64 + x.double()
    u1 = s1 * torch.rsqrt((s1 * s1).mean(1, keepdim=True) + 1e-6) * w.double()
    s2 = u1 + s1
    u2 = s2 * torch.rsqrt((s2 * s2).mean(1, keepdim=True) + 1e-6) * w.double()
    ref = torch.autograd.grad((u2 * dy.double()).sum() + (s2 * ds.double()).sum(), l64)[0]
    # two layers of products of 32-bit values, 64 roundings each
    assert float((g.double() - ref).norm()) <= 128 * U * float(ref.norm()) * 2


def test_autograd_rules():
    x, r, w = _inputs(5, 64, torch.float32, torch.float32)
    leaf = x.clone().requires_grad_()
    y = rms_norm(leaf, w)
    (g,) = torch.autograd.grad(y.sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), leaf)
    # a sum that is changed after the call is not read by the backward
    y, total = rms_norm(leaf, w, residual=r)
    total.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()
    with pytest.raises(RuntimeError, match="no gradient"):
        rms_norm_quantize(leaf, w)
    with torch.no_grad():
        assert not rms_norm(leaf, w).requires_grad
        rms_norm_quantize(leaf, w)
    import torch.autograd.forward_ad as fwAD
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError):
            rms_norm(dual, w)
        with pytest.raises(RuntimeError, match="tangent"):
            rms_norm_quantize(dual, w)


def test_streams_and_graph():
    x, r, w = _inputs(300, 1000, torch.bfloat16, torch.bfloat16)
    dy, ds = torch.randn_like(x), torch.randn_like(x)
    want = _backward(x, r, w, dy, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _backward(x, r, w, dy, ds)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2]["weight"], want[2]["weight"])

    sx, sr = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total, grads = _backward(sx, sr, w, dy, ds)
        q, scale, _ = rms_norm_quantize(sx, w, residual=sr)
    for seed in (1, 2):
        nx, nr, _ = _inputs(300, 1000, torch.bfloat16, torch.bfloat16, seed)
        sx.copy_(nx)
        sr.copy_(nr)
        graph.replay()
        want = _backward(nx, nr, w, dy, ds)
        assert torch.equal(y, want[0]) and torch.equal(total, want[1])
        assert all(torch.equal(grads[k], want[2][k]) for k in grads)
        wq = rms_norm_quantize(nx, w, residual=nr)
        assert torch.equal(q, wq[0]) and torch.equal(scale, wq[1])


def test_slices_of_wider_rows():
    g = torch.Generator("cuda").manual_seed(3)
    wide = torch.randn(3, 5, 2 * 264, generator=g, device="cuda")
    dy, ds = (torch.randn(3, 5, 264, generator=g, device="cuda") for _ in range(2))
    w = 1 + 0.3 * torch.randn(264, generator=g, device="cuda")
    for part in (wide[..., 264:], wide[:, 1:4, :264], wide.transpose(0, 1)[..., :264],
                 wide[:, 2:3, :264], wide[..., ::2]):
        up, us = dy[:, :part.shape[1]], ds[:, :part.shape[1]]
        if part.shape[:2] != up.shape[:2]:
            up, us = dy.transpose(0, 1), ds.transpose(0, 1)
        results = []
        for view in (part, part.contiguous()):
            x, r = view.detach().requires_grad_(), (view * 2).detach().requires_grad_()
            outs = [rms_norm(x, w), *rms_norm(x, w, residual=view), *rms_norm(r, w, residual=x)]
            results.append(outs + list(torch.autograd.grad(
                outs, [x, r], [up, up, us, up, us])) + list(rms_norm_quantize(x.detach(), w)))
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_captured_backward_beside_an_eager_graph():
    x = torch.randn(8, 264, device="cuda").requires_grad_()
    dy = torch.randn(8, 264, device="cuda")
    kept = rms_norm(x)
    want, = torch.autograd.grad(rms_norm(x), x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured backward"):
        with torch.cuda.graph(graph):
            rms_norm(x).backward(dy)
    assert x.grad is None
    del kept
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rms_norm(x).backward(dy)
    x.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want)


def test_into_the_8_bit_head():
    x, r, w = _inputs(20, 1000, torch.bfloat16, torch.bfloat16)
    head_q, head_scale = quantize_rows(torch.randn(333, 1000, device="cuda").bfloat16())
    q, scale, _ = rms_norm_quantize(x, w, residual=r)
    logits = int8_linear(q, head_q, head_scale, x_scale=scale)
    _, _, y = _forward64(x, r, w, 1e-6)
    head = head_q.double() * head_scale.double()[:, None]
    # half a step of each row's scale on every value, at random
    tol = 6 * 0.5 * scale.double()[:, None] * head.norm(dim=1)
    _within(logits, y @ head.t(), tol)


def test_a_row_beyond_32_bits_of_offset():
    n, h = 70001, 32768  # 2.3 G values
    if torch.cuda.mem_get_info()[0] < 24e9:
        pytest.skip("needs 24 GB")
    x = torch.zeros(n, h, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(h, device="cuda")
    y = rms_norm(x)
    _check_forward(x[-1:], None, None, 1e-6, y[-1:], None)
    assert not bool(y[-2].any())
    del y
    q, scale = rms_norm_quantize(x)
    want = quantize_rows(rms_norm(x[-1:].float()))
    assert torch.equal(q[-1:], want[0]) and torch.equal(scale[-1:], want[1])
