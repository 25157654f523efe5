"""The gradients' norm and the clip by it against 64-bit sums.

Tolerances. A thread adds at most 16 terms into each of four 32-bit sums and joins those (18
roundings of 2^-24), everything above is 64-bit, and the norm is rounded once: 20 * 2^-24 relative
covers p = 1 (the root of p = 2 halves what the sum is off by); the maximum is exact. The factor
adds a sum and a quotient, the product one rounding, and the store half a step of its type.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import (clip_grad_norm_, clip_grads, clip_grads_,
                                              fused_linear_cross_entropy, grad_norm)

pytestmark = pytest.mark.gpu

NORM_REL = 20 * 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _norm64(grads, p):
    parts = [g.double().abs().reshape(-1) for g in grads if g.numel()]
    if not parts:
        return 0.0
    flat = torch.cat(parts)
    return float(flat.max() if p == math.inf else flat.pow(p).sum().pow(1.0 / p))


def _check_norm(got, grads, p, rel=NORM_REL):
    want = _norm64(grads, p)
    assert got.dtype == torch.float32 and got.shape == ()
    assert abs(float(got) - want) <= (0 if p == math.inf else rel) * want, (float(got), want)
    return want


def _check_clipped(got, was, norm, max_norm, eps=1e-6):
    factor = min(1.0, max_norm / (norm + eps))
    for o, g in zip(got, was):
        want = g.double() * factor
        half = torch.finfo(o.dtype).eps / 2
        # half a step of the smallest number that the type holds
        tiny = torch.finfo(o.dtype).smallest_normal * half
        err = (o.double() - want).abs()
        assert bool((err <= (half + NORM_REL + 3 * 2.0 ** -24) * want.abs() + tiny).all())


def _make(shapes, dtype, scale=1.0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(dtype) for s in shapes]


SHAPES = [
    [(1,)],
    [(7,), (0,), (3, 5), (1, 1)],
    [(8191,), (8192,), (8193,), (16384,), (16385,), (65537,)],
    [(257, 129), (1000,), (31, 4096), (5, 7, 11, 13)],
]


@pytest.mark.parametrize("p", [1.0, 2.0, math.inf])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shapes", SHAPES, ids=range(len(SHAPES)))
def test_norm_and_clip(shapes, dtype, p):
    grads = _make(shapes, dtype)
    want = _check_norm(grad_norm(grads, p), grads, p)
    for ratio in (0.25, 3.0):
        was = [g.clone() for g in grads]
        got = [g.clone() for g in grads]
        norm = clip_grads_(got, want * ratio, p)
        _check_norm(norm, was, p)
        _check_clipped(got, was, want, want * ratio)
        if ratio > 1:
            assert all(torch.equal(a, b) for a, b in zip(got, was))
        out = [torch.full_like(g, 7.0) for g in grads]
        _check_norm(clip_grads(grads, want * ratio, p, out=out), was, p)
        _check_clipped(out, was, want, want * ratio)
        assert all(torch.equal(a, b) for a, b in zip(grads, was))
        if dtype != torch.float32:
            out = [torch.full(g.shape, 7.0, device="cuda") for g in grads]
            clip_grads(grads, want * ratio, p, out=out)
            _check_clipped(out, was, want, want * ratio)


def test_types_together_and_many_tensors():
    grads = []
    for i in range(1203):  # three launches' worth
        grads += _make([(1 + 37 * i % 91,)], TYPES[i % 3], seed=i)
    want = _check_norm(grad_norm(grads), grads, 2.0)
    got = [g.clone() for g in grads]
    _check_norm(clip_grads_(got, 0.5 * want), grads, 2.0)
    _check_clipped(got, grads, want, 0.5 * want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start", range(1, 9))
def test_any_address(dtype, start):
    """Tensors that start anywhere, with the elements around them left alone."""
    buf = torch.full((40000,), 2.5, dtype=dtype, device="cuda")
    grads = [buf[start:start + 16391], buf[16400 + start:16400 + start + 5]]
    for i, g in enumerate(grads):
        g.copy_(_make([g.shape], dtype, seed=i)[0])
    was = [g.clone() for g in grads]
    want = _check_norm(grad_norm(grads), was, 2.0)
    clip_grads_(grads, 0.1 * want)
    _check_clipped(grads, was, want, 0.1 * want)
    outside = torch.ones_like(buf, dtype=torch.bool)
    outside[start:start + 16391] = False
    outside[16400 + start:16400 + start + 5] = False
    assert bool((buf[outside] == 2.5).all())
    out = torch.full((20000,), 1.5, dtype=torch.float32, device="cuda")
    clip_grads(was[:1], 0.1 * want, out=[out[start + 2:start + 2 + 16391]])
    assert bool((out[:start + 2] == 1.5).all()) and bool((out[start + 2 + 16391:] == 1.5).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Transposed, sliced, stepped and permuted gradients; broadcast ones for the norm alone."""
    base = _make([(64, 96), (33, 70), (500,), (6, 10, 14), (4, 6, 8, 10)], dtype)
    views = [base[0].t(), base[1][:, 3:41], base[2][::3], base[3].permute(2, 0, 1)[1:, :, 2:7],
             base[4][:, 1:4, :, 3:8]]
    was = [v.clone() for v in views]
    whole = [b.clone() for b in base]
    want = _check_norm(grad_norm(views), was, 2.0)
    _check_norm(clip_grads_(views, 0.5 * want), was, 2.0)
    _check_clipped(views, was, want, 0.5 * want)
    for b, w, v in zip(base, whole, views):  # elements outside the views keep their values
        v.zero_()
        mask = b != 0
        assert torch.equal(b[mask], w[mask])
    out = [torch.zeros(w.shape[::-1], dtype=dtype, device="cuda").permute(
        *reversed(range(w.dim()))) for w in was]
    clip_grads(was, 0.5 * want, out=out)
    _check_clipped(out, was, want, 0.5 * want)
    wide = _make([(40, 1)], dtype)[0].expand(40, 300)
    _check_norm(grad_norm([wide]), [wide], 2.0)


@pytest.mark.parametrize("scale", [1e25, 1e-25, 1e-40, 3e38])
def test_far_from_one(scale):
    """Squares beyond 32 bits' range on either side."""
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.rand(50001, device="cuda", dtype=torch.float64).add_(0.1).mul_(0.8)
        g[0] = 1e-3
        g = (g * scale).to(dtype)
        want = _norm64([g], 2.0)
        got = float(grad_norm([g]))
        if want > torch.finfo(torch.float32).max:
            assert got == math.inf
        else:
            assert abs(got - want) <= NORM_REL * want + 2.0 ** -149
    # a few large values among small ones, and zeros around them
    g = torch.zeros(100000, device="cuda")
    g[777] = scale if scale < 1e38 else 1.0
    g[99999] = 0.5
    _check_norm(grad_norm([g]), [g], 2.0)


@pytest.mark.parametrize("p", [1.0, 2.0, math.inf])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(bad, p):
    grads = _make([(100,), (20000,)], torch.float32)
    grads[1][12345] = bad
    norm = grad_norm(grads, p)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    got = [g.clone() for g in grads]
    clip_grads_(got, 1.0, p)
    if math.isnan(bad):
        assert all(bool(torch.isnan(g).all()) for g in got)
    else:
        assert math.isnan(float(got[1][12345])) and bool((got[0] == 0).all())
    params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
    for q, g in zip(params, grads):
        q.grad = g.clone()
    with pytest.raises(RuntimeError, match="not clipped"):
        clip_grad_norm_(params, 1.0, p, error_if_nonfinite=True)
    assert all(torch.equal(q.grad.nan_to_num(), g.nan_to_num()) for q, g in zip(params, grads))


def test_nothing_and_zeros():
    assert float(grad_norm([])) == 0.0
    assert float(clip_grads_([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    z = [torch.zeros(70000, device="cuda", dtype=torch.bfloat16)]
    assert float(clip_grads_(z, 1.0)) == 0.0 and not bool(z[0].any())
    g = _make([(1000,)], torch.float32)
    clip_grads_(g, 0.0)
    assert not bool(g[0].any())


def test_same_result_every_run_and_on_other_streams():
    grads = _make([(1 << 20,), (12345,), (300, 1001)], torch.bfloat16)
    first = grad_norm(grads)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [grad_norm(grads) for _ in range(20)]
    side.synchronize()
    assert all(torch.equal(first, a) for a in again)


def test_graph_capture():
    grads = _make([(4096, 33), (1001,)], torch.bfloat16)
    fresh = [g.clone() for g in grads]
    clip_grads_(grads, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip_grads_(grads, 1.0)
    for seed in range(3):
        new = _make([(4096, 33), (1001,)], torch.bfloat16, scale=10.0 ** (seed - 3), seed=seed)
        for g, f, n in zip(grads, fresh, new):
            g.copy_(n)
            f.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        want = clip_grads_(fresh, 1.0)
        assert torch.equal(norm, want)
        assert all(torch.equal(a, b) for a, b in zip(grads, fresh))


def test_after_the_loss():
    """The gradients that the fused loss gives, clipped as a training step does."""
    g = torch.Generator("cuda").manual_seed(3)
    hidden = torch.randn(300, 64, generator=g, device="cuda").bfloat16().requires_grad_(True)
    weight = torch.randn(1000, 64, generator=g, device="cuda").bfloat16().requires_grad_(True)
    targets = torch.randint(0, 1000, (300,), generator=g, device="cuda")
    fused_linear_cross_entropy(hidden, weight, targets).backward()
    was = [hidden.grad.clone(), weight.grad.clone()]
    spare = torch.nn.Parameter(torch.zeros(3, device="cuda"))  # has no gradient
    norm = clip_grad_norm_([hidden, weight, spare], 0.01)
    want = _check_norm(norm, was, 2.0)
    assert want > 0.01
    _check_clipped([hidden.grad, weight.grad], was, want, 0.01)
    assert abs(_norm64([hidden.grad, weight.grad], 2.0) - 0.01) < 0.01 * 2.0 ** -8


def test_autograd_sees_the_change():
    g = _make([(100,), (200,)], torch.float32)
    versions = [x._version for x in g]
    clip_grads_(g, 1.0)
    assert [x._version for x in g] == [v + 1 for v in versions]
    with torch.inference_mode():
        clip_grads_([torch.ones(100, device="cuda")], 1.0)


def test_refusals():
    a = torch.zeros(100, device="cuda")
    with pytest.raises(RuntimeError, match="overlap"):
        clip_grads_([a[:60], a[50:]], 1.0)
    with pytest.raises(RuntimeError, match="overlap"):
        clip_grads_([a, a], 1.0)
    with pytest.raises(RuntimeError, match="overlap"):
        clip_grads([a[:50]], 1.0, out=[a[1:51]])
    m = torch.zeros(10, 10, device="cuda")
    clip_grads_([m[:, :4], m[:, 4:7], m[:, 7:]], 1.0)  # side by side
    with pytest.raises(RuntimeError, match="overlap"):
        clip_grads_([m[:, :4], m[:, 3:7]], 1.0)
    with pytest.raises(RuntimeError):
        clip_grads_([torch.zeros(1, 1, device="cuda").expand(5, 5)], 1.0)
    with pytest.raises(ValueError):
        clip_grads([a], 1.0, out=[a[:5]])
    with pytest.raises(TypeError):
        clip_grads([a], 1.0, out=[torch.zeros(100, device="cuda", dtype=torch.float16)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_clips_in_a_row(dtype):
    """One launch reads the gradients for the norm and then writes them: clips in place of one
    piece of memory, one after the other, each of what the one before left or of new values."""
    buf = torch.empty(100003, dtype=dtype, device="cuda")
    grads = [buf[3:40000], buf[40000:40007], buf[40007:]]
    fresh = [_make([(100003,)], dtype, scale=10.0 ** (i % 5 - 2), seed=i)[0] for i in range(20)]
    was, got, norms, limits = [], [], [], []
    for x in fresh:
        buf.copy_(x)
        for limit in (3.0, 1.0, 0.25):
            was.append(buf[3:].clone())
            norms.append(clip_grads_(grads, limit))
            got.append(buf[3:].clone())
            limits.append(limit)
    for w, o, norm, limit in zip(was, got, norms, limits):
        want = _check_norm(norm, [w], 2.0)
        _check_clipped([o], [w], want, limit)


@pytest.mark.parametrize("p", [1.0, 2.0, math.inf])
def test_no_limit(p):
    """max_norm = inf: the norm is read and the gradients stay."""
    grads = _make([(100,), (20000,)], torch.bfloat16)
    params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
    for bad in (None, math.inf, math.nan):
        if bad is not None:
            grads[1][777] = bad
        for q, g in zip(params, grads):
            q.grad = g.clone()
        norm = clip_grad_norm_(params, math.inf, p)
        if bad is None:
            _check_norm(norm, grads, p)
        else:
            assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
            with pytest.raises(RuntimeError, match="not clipped"):
                clip_grad_norm_(params, math.inf, p, error_if_nonfinite=True)
        assert all(torch.equal(q.grad.view(torch.int16), g.view(torch.int16))
                   for q, g in zip(params, grads))
    for bad in (-1.0, math.nan, -math.inf):
        with pytest.raises(ValueError, match="max_norm"):
            clip_grad_norm_(params, bad, p)
    with pytest.raises(ValueError, match="eps"):
        clip_grad_norm_(params, math.inf, p, eps=-1.0)


@pytest.mark.parametrize("order", [(0, 1, 2), (1, 2, 0), (2, 1, 0)])
def test_autograd_sees_the_change_among_inference_tensors(order):
    """Lists that mix inference tensors, which have no version, with others, in any order; inside
    inference mode and outside."""
    with torch.inference_mode():
        plain = [torch.ones(50, device="cuda") for _ in range(2)]
    a = torch.ones(50, device="cuda")
    every = [plain[0], a, plain[1]]
    every = [every[i] for i in order]
    copies = [torch.empty(50, device="cuda") for _ in range(3)]
    for inside in (False, True):
        with torch.inference_mode(inside):
            was = a._version
            clip_grads_(every, 1.0)
            assert a._version == was + 1
            before = [c._version for c in copies]
            clip_grads(every, 1.0, out=copies)
            assert a._version == was + 1
            assert [c._version for c in copies] == [v + 1 for v in before]
            clip_grads(copies, 1.0, out=every)
            assert a._version == was + 2
    clip_grads_(plain, 1.0)
    clip_grads_([], 1.0)


@pytest.mark.parametrize("n", [5, 1 << 20])  # one launch, and two
@pytest.mark.parametrize("p", [1.0, 2.0, math.inf])
def test_zeros_without_eps(p, n):
    """Gradients of norm 0, eps 0 and max_norm 0: the quotient has no value, the gradients do."""
    zeros = [torch.zeros(n, device="cuda"), torch.zeros(3, dtype=torch.bfloat16, device="cuda")]
    out = [torch.full(z.shape, 7.0, device="cuda") for z in zeros]
    for limit in (0.0, 1.0):
        assert float(clip_grads(zeros, limit, p, out=out, eps=0.0)) == 0.0
        assert not any(bool(o.any()) for o in out)
        assert float(clip_grads_(zeros, limit, p, eps=0.0)) == 0.0
        assert not any(bool(z.any()) for z in zeros)
