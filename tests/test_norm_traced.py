"""The norm's operators where tensors have no data: fake tensors, tracing, torch.compile."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx
from torch.utils._python_dispatch import TorchDispatchMode

from linear_cross_entropy_vocab_gb300 import native_build, rms_norm, rms_norm_quantize

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(20,), (3, 16), (2, 3, 40), (2, 1, 4, 33)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    native_build.build()


def _inputs(shape, residual, make=torch.empty):
    x = make(shape, device="cuda", dtype=torch.bfloat16)
    r = None if residual is None else make(shape, device="cuda", dtype=residual)
    return x, make(shape[-1:], device="cuda", dtype=torch.float32), r


@pytest.mark.parametrize("shape", SHAPES)
def test_fake_tensors(shape):
    for residual in (None, torch.bfloat16, torch.float32):
        with FakeTensorMode():
            x, w, r = _inputs(shape, residual)
            got = rms_norm(x.requires_grad_(), w, residual=r)
            y, s = got if r is not None else (got, None)
            assert y.requires_grad and y.shape == shape and y.dtype == x.dtype and y.is_cuda and y.is_contiguous()
            assert s is None or (s.shape == shape and s.dtype == residual)
            with torch.no_grad():
                got = rms_norm(x, w, residual=r)
                assert (got if r is None else got[0]).shape == shape
                q, scale, *s = rms_norm_quantize(x, w, residual=r)
            pitch = (shape[-1] + 15) // 16 * 16
            assert q.shape == shape and q.dtype == torch.int8 and scale.shape == shape[:-1]
            assert scale.dtype == torch.float32 and q.stride(-1) == 1
            assert len(shape) == 1 or q.stride(-2) == pitch
            assert len(s) == (r is not None)


def _refusals(make):
    """Calls of the operators themselves whose shapes do not fit: nothing may be launched."""
    x, w, r = make(4, 40), make(40), make(4, 40)
    rstd = make(4)
    ops = torch.ops.flce
    for bad_w, bad_r in ((make(39), r), (make(1, 40), r), (w, make(40)), (w, make(3, 40)),
                         (w, make(4, 1))):
        for call in (ops.rms_norm_forward, ops.rms_norm_quantize,
                     lambda *a: ops.rms_norm(*a, False)):
            with pytest.raises(ValueError, match="weight must|residual must"):
                call(x, bad_w, 1e-6, bad_r)
    for call in (ops.rms_norm_forward, ops.rms_norm_quantize):
        with pytest.raises(ValueError, match="H of at least 1"):
            call(make(4, 0), None, 1e-6, None)
    good = dict(grad_y=x, grad_sum=r, total=x, weight=w, rstd=rstd, eps=1e-6, need_x=True,
                need_residual=False, need_weight=True)
    for bad in (dict(grad_y=make(4, 39)), dict(grad_sum=make(2, 40)), dict(weight=make(41)),
                dict(rstd=make(3)), dict(rstd=make(4, 1)), dict(rstd=make(8)[::2]),
                dict(rstd=make(4).half()), dict(total=make(5, 40)), dict(weight=None),
                dict(grad_sum=r.half())):
        with pytest.raises(ValueError):
            ops.rms_norm_backward(**{**good, **bad})


def test_refusals_of_the_operators():
    with FakeTensorMode():
        rms_norm(torch.empty(2, 8, device="cuda"))  # loads the library
        _refusals(lambda *shape: torch.empty(shape, device="cuda"))


@pytest.mark.gpu
def test_refusals_of_the_operators_on_a_gpu():
    rms_norm(torch.ones(1, 8, device="cuda"))
    _refusals(lambda *shape: torch.ones(shape, device="cuda"))
    x = torch.ones(4, 40, device="cuda")
    with pytest.raises(ValueError, match="device"):
        torch.ops.flce.rms_norm_forward(x, torch.ones(40), 1e-6, None)
    with pytest.raises(ValueError, match="each row"):
        torch.ops.flce.rms_norm_backward(x, None, x, None, torch.ones(4), 1e-6, True, False, False)


@pytest.mark.gpu  # autograd's threads ask for the device
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_of_fake_tensors(shape):
    for residual in (None, torch.bfloat16, torch.float32):
        with FakeTensorMode():
            x, w, r = _inputs(shape, residual)
            leaves = [t.requires_grad_() for t in (x, w, r) if t is not None]
            got = rms_norm(x, w, residual=r)
            outs = [got] if r is None else list(got)
            grads = torch.autograd.grad(outs, leaves, [torch.empty_like(t) for t in outs])
            for leaf, grad in zip(leaves, grads):
                assert grad.shape == leaf.shape and grad.dtype == leaf.dtype


@pytest.mark.gpu
def test_a_traced_training_step():
    """What a tracer sees: both directions as operators, with no data touched."""
    def step(x, w, r, dy, ds):
        y, s = rms_norm(x, w, residual=r)
        return torch.autograd.grad([y, s], [x, w, r], [dy, ds])

    with FakeTensorMode() as mode:
        x, w, r = (t.requires_grad_() for t in _inputs((4, 6, 40), torch.float32))
        dy, ds = torch.empty_like(x), torch.empty_like(r)
        with mode:
            graph = make_fx(step)(x, w, r, dy, ds)
    names = [str(n.target) for n in graph.graph.nodes if n.op == "call_function"]
    assert "flce.rms_norm_forward.default" in names
    assert "flce.rms_norm_backward.default" in names


@pytest.mark.gpu
@pytest.mark.parametrize("dynamic", [False, True])
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
def test_compiled(residual, dynamic):
    """The same bits as without compilation, in both directions and in 8 bits."""
    def step(x, w, r):
        got = rms_norm(x * 2, w, residual=r)
        y, s = got if r is not None else (got, x)
        return (y * y).sum() + s.float().sum() * 0.5, y

    def quantize(x, w, r):
        with torch.no_grad():
            return [t + 0 for t in rms_norm_quantize(x, w, residual=r)]

    rms_norm(torch.ones(1, 8, device="cuda"))  # loads the library
    torch._dynamo.reset()
    compiled = torch.compile(step, backend="aot_eager", fullgraph=True, dynamic=dynamic)
    compiled_q = torch.compile(quantize, backend="aot_eager", fullgraph=True, dynamic=dynamic)
    for shape in ((6, 64), (9, 64), (5, 33)):
        g = torch.Generator("cuda").manual_seed(len(shape) + shape[0])
        x, w, r = _inputs(shape, residual, lambda *a, **k: torch.randn(*a, generator=g, **k))
        leaves = [t.requires_grad_() for t in (x, w, r) if t is not None]
        results = []
        for f in (step, compiled):
            loss, y = f(x, w, r)
            results.append([y.detach(), *torch.autograd.grad(loss, leaves)])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        for a, b in zip(quantize(x, w, r), compiled_q(x, w, r)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_compiled_as_the_first_call():
    """Where the library is not loaded yet."""
    code = ("import torch\n"
            "from linear_cross_entropy_vocab_gb300 import rms_norm\n"
            "f = torch.compile(lambda x, w: rms_norm(x, w) * 2, backend='aot_eager')\n"
            "x = torch.randn(5, 64, device='cuda').requires_grad_()\n"
            "w = torch.rand(64, device='cuda').requires_grad_()\n"
            "y = f(x, w)\n"
            "got = [y, *torch.autograd.grad(y.sum(), (x, w))]\n"
            "z = rms_norm(x, w) * 2\n"
            "want = [z, *torch.autograd.grad(z.sum(), (x, w))]\n"
            "assert all(torch.equal(a, b) for a, b in zip(got, want))\n")
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=600)
    assert done.returncode == 0, done.stderr[-3000:]


class _Listener(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(str(func))
        return func(*args, **(kwargs or {}))


@pytest.mark.gpu
@pytest.mark.parametrize("forward", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_a_mode_that_listens_to_one_direction(forward, backward):
    g = torch.Generator("cuda").manual_seed(2)
    wide = torch.randn(6, 2, 70, generator=g, device="cuda")
    dy = torch.randn(6, 70, generator=g, device="cuda")
    for x in (wide[:, 0], wide[:, 1, ::2], wide.permute(1, 0, 2)[0]):
        leaf = x.detach().requires_grad_()
        w = torch.rand(x.shape[-1], generator=g, device="cuda").requires_grad_()
        up = dy[:, :x.shape[-1]]
        want = rms_norm(leaf, w)
        want = [want, *torch.autograd.grad(want, (leaf, w), up)]
        listener = _Listener()
        with listener if forward else contextlib.nullcontext():
            y = rms_norm(leaf, w)
        with listener if backward else contextlib.nullcontext():
            got = [y, *torch.autograd.grad(y, (leaf, w), up)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert ("flce.rms_norm_forward.default" in listener.seen) == forward
        assert ("flce.rms_norm_backward.default" in listener.seen) == backward


@pytest.mark.gpu
def test_operators_by_themselves():
    """Through the dispatcher they do what the call does, strided inputs included."""
    g = torch.Generator("cuda").manual_seed(1)
    for shape in SHAPES:
        for residual in (None, torch.bfloat16, torch.float32):
            x, w, r = _inputs(shape, residual,
                              lambda *a, **k: torch.randn(*a, generator=g, **k))
            x = torch.stack([x, x], -1)[..., 0]  # elements two apart
            rms_norm(x, w, residual=r)
            out = torch.ops.flce.rms_norm_forward(x, w, 1e-6, r)
            leaves = [t.detach().requires_grad_() for t in (x, w, r) if t is not None]
            got = rms_norm(leaves[0], leaves[1], residual=leaves[2] if r is not None else None)
            y, s = got if r is not None else (got, None)
            assert torch.equal(y, out[0]) and (s is None or torch.equal(s, out[2]))
            dy = torch.randn(shape, generator=g, device="cuda").bfloat16()
            want = torch.autograd.grad(y, leaves, dy)
            wide = residual == torch.float32
            back = torch.ops.flce.rms_norm_backward(dy, None, x if s is None else s.detach(), w,
                                                    out[1], 1e-6, True, wide, True)
            assert torch.equal(back[0], want[0]) and torch.equal(back[-1], want[1])
            assert not wide or torch.equal(back[1], want[2])
