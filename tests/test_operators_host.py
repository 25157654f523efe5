"""Refusals of the gradient, beam and 8-bit operators, which need no GPU: the C entry points
return their status before any CUDA call, and the Python layer raises before it calls them."""
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


def test_struct_layouts():
    assert ctypes.sizeof(abi.flce_grad) == 56
    assert ctypes.sizeof(abi.flce_beam_problem) == 80
    assert ctypes.sizeof(abi.flce_beam_state) == 88
    assert ctypes.sizeof(abi.flce_qproblem) == 80


# ------------------------------------------------------------- gradients
def _grad(**kw):
    args = dict(src=FAKE, dst=FAKE, rows=1, cols=100, src_pitch=100, dst_pitch=100, src_dtype=0,
                dst_dtype=0)
    args.update(kw)
    return abi.flce_grad(**args)


def _clip(*grads, norm=abi.FLCE_NORM_L2, max_norm=1.0, eps=0.0, norm_out=FAKE, workspace=FAKE,
          ws_bytes=1 << 40, call="clip", count=None):
    table = (abi.flce_grad * max(len(grads), 1))(*grads)
    n = len(grads) if count is None else count
    if call == "norm":
        return abi.flce_grad_norm(ctypes.addressof(table), n, norm, norm_out, workspace, ws_bytes,
                                  None, check=False)
    return abi.flce_grad_clip(ctypes.addressof(table), n, norm, max_norm, eps, norm_out,
                              workspace, ws_bytes, None, check=False)


def test_grad_refusals():
    for call in ("norm", "clip"):
        assert _clip(_grad(), call=call, norm=0) == INVALID
        assert _clip(_grad(), call=call, norm=4) == INVALID
        assert _clip(_grad(), call=call, norm_out=None) == INVALID
        assert _clip(_grad(), call=call, norm_out=FAKE + 2) == UNSUPPORTED
        assert _clip(_grad(src=None), call=call) == INVALID
        assert _clip(_grad(src_dtype=3), call=call) == INVALID
        assert _clip(_grad(rows=-1), call=call) == INVALID
        assert _clip(_grad(cols=-1), call=call) == INVALID
        assert _clip(_grad(rows=1 << 40, cols=1 << 40), call=call) == INVALID
        assert _clip(_grad(rows=1 << 30, src_pitch=1 << 40), call=call) == INVALID
        assert _clip(_grad(src=FAKE + 2), call=call) == UNSUPPORTED
        assert _clip(_grad(), call=call, count=-1) == INVALID
        assert _clip(_grad(), call=call, ws_bytes=8) == WORKSPACE
        assert _clip(_grad(), call=call, workspace=None) == WORKSPACE
        assert _clip(_grad(), call=call, workspace=FAKE + 8) == WORKSPACE
    assert _clip(_grad(dst=None)) == INVALID
    assert _clip(_grad(dst_dtype=abi.FLCE_BF16)) == INVALID  # fp32 gradients stay fp32
    assert _clip(_grad(rows=2, dst_pitch=50)) == INVALID
    for bad in (-1.0, math.nan, math.inf):
        assert _clip(_grad(), max_norm=bad) == INVALID
        assert _clip(_grad(), eps=bad) == INVALID


def test_grad_overlaps():
    far = 0x900000

    def status(*grads):
        st = _clip(*grads)
        return "overlap" in abi.flce_last_error() if st == INVALID else st

    # no overlap is refused further on, by the missing device at the latest
    assert status(_grad(), _grad(src=FAKE + 400, dst=FAKE + 400)) is not True
    assert status(_grad(), _grad(src=far, dst=FAKE + 396)) is True
    assert status(_grad(), _grad()) is True
    assert status(_grad(dst=FAKE + 4)) is True
    assert status(_grad(dst=far), _grad(dst=far + 400)) is not True  # one source, read twice
    assert status(_grad(dst=far), _grad(dst=far + 399 // 4 * 4)) is True
    half = dict(rows=9, cols=40, src_pitch=100, dst_pitch=100)
    assert status(_grad(**half), _grad(src=FAKE + 160, dst=FAKE + 160, **half)) is not True
    assert status(_grad(**half), _grad(src=FAKE + 156, dst=FAKE + 156, **half)) is True
    assert status(_grad(**half), _grad(src=FAKE + 244, dst=FAKE + 244, **half)) is True
    assert status(_grad(**half), _grad(src=FAKE + 160, dst=FAKE + 160, rows=9, cols=40,
                                       src_pitch=101, dst_pitch=101)) is True
    assert status(_grad(rows=0), _grad()) is not True


def test_grad_python_refusals():
    a = torch.zeros(4)
    for call in (lambda g: package.grad_norm(g), lambda g: package.clip_grads_(g, 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call([a])
        with pytest.raises(TypeError):
            call([a.double()])
    with pytest.raises(ValueError, match="norm_type"):
        package.grad_norm([a], 3)
    with pytest.raises(ValueError, match="norm_type"):
        package.grad_norm([a], "two")
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(ValueError, match="max_norm"):
            package.clip_grads_([a], bad)
        with pytest.raises(ValueError, match="eps"):
            package.clip_grads_([a], 1.0, eps=bad)
    with pytest.raises(ValueError):
        package.clip_grads([a], 1.0, out=[])


# ------------------------------------------------------------------ beams
def _select(ws_bytes=1 << 40, workspace=FAKE, **kw):
    prob = dict(batch=2, beams=3, v=1000, candidates=6, stride_batch=3000, stride_beam=1000,
                allowed_stride_batch=0, allowed_stride_beam=0, pad_token=0, dtype=0, reserved=0)
    ptr = dict(logits=FAKE, beam_scores=FAKE, finished=None, allowed=None, scores_out=FAKE,
               parents_out=FAKE, tokens_out=FAKE, err_word=None)
    for k in kw:
        (prob if k in prob else ptr)[k] = kw[k]
    p = abi.flce_beam_problem(**prob)
    return abi.flce_beam_select(p, *ptr.values(), workspace, ws_bytes, None, check=False)


def test_select_refusals():
    for bad in (dict(batch=-1), dict(v=0), dict(v=1 << 31), dict(pad_token=-1),
                dict(pad_token=1000), dict(dtype=3), dict(reserved=1), dict(stride_batch=-1),
                dict(allowed_stride_beam=-1), dict(logits=None), dict(beam_scores=None),
                dict(scores_out=None), dict(parents_out=None), dict(tokens_out=None)):
        assert _select(**bad) == INVALID, bad
    for bad in (dict(beams=0), dict(beams=1025), dict(candidates=0), dict(candidates=257),
                dict(logits=FAKE + 2), dict(tokens_out=FAKE + 4), dict(err_word=FAKE + 1)):
        assert _select(**bad) == UNSUPPORTED, bad
    assert _select(ws_bytes=100) == WORKSPACE
    assert _select(workspace=FAKE + 16) == WORKSPACE
    assert abi.flce_beam_select_workspace_size(abi.flce_beam_problem()) == 0


def _reorder(count=1, parents=FAKE, batch=2, beams=3, err_word=None, **kw):
    size, stride = kw.pop("size", (1, 1, 1, 1)), kw.pop("stride", (0, 0, 0, 0))
    s = dict(data=FAKE, beam_stride=1000, run_bytes=1000)
    s.update(kw)
    table = (abi.flce_beam_state * 1)(abi.flce_beam_state(
        s["data"], s["beam_stride"], (ctypes.c_int64 * 4)(*size), (ctypes.c_int64 * 4)(*stride),
        s["run_bytes"]))
    return abi.flce_beam_reorder(ctypes.addressof(table), count, parents, batch, beams, err_word,
                                 None, check=False)


def test_reorder_refusals():
    for bad in (dict(count=-1), dict(parents=None), dict(batch=-1), dict(data=None),
                dict(run_bytes=-1), dict(size=(-1, 1, 1, 1)), dict(beam_stride=999),
                dict(beam_stride=0), dict(beam_stride=-1000),
                dict(size=(1, 1, 1, 2), stride=(0, 0, 0, 500)),
                dict(size=(1, 1, 1, 2), stride=(0, 0, 0, 1000)),
                dict(size=(1, 1, 5, 2), stride=(0, 0, 6000, 6500), beam_stride=100000)):
        assert _reorder(**bad) == INVALID, bad
    for bad in (dict(beams=0), dict(beams=65), dict(parents=FAKE + 4), dict(err_word=FAKE + 2),
                dict(run_bytes=1 << 45, beam_stride=1 << 45), dict(size=(1 << 40, 1, 1, 1))):
        assert _reorder(**bad) == UNSUPPORTED, bad


def test_beam_python_refusals():
    z, s = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        package.beam_select(z, s)
    with pytest.raises(ValueError):
        package.beam_select(z[0], s)
    with pytest.raises(TypeError):
        package.beam_select(z.double(), s)
    p = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        package.beam_reorder_(z, p)
    with pytest.raises(TypeError):
        package.beam_reorder_(z, p.int())
    with pytest.raises(ValueError):
        package.beam_reorder_(z, p[0])


# ------------------------------------------------------------------ 8 bits
def _qlinear(ws_bytes=1 << 40, workspace=FAKE, **kw):
    prob = dict(n=5, h=64, v=100, x_pitch=64, weight_pitch=64, out_pitch=100, x_dtype=0,
                out_dtype=0, bias_dtype=0, has_bias=0, logit_scale=1.0, softcap=0.0, flags=0,
                reserved=0)
    ptr = dict(x=FAKE, x_scale=None, weight=FAKE, weight_scale=FAKE, bias=None, out=FAKE,
               err_word=None)
    for k in kw:
        (prob if k in prob else ptr)[k] = kw[k]
    return abi.flce_qlinear(abi.flce_qproblem(**prob), *ptr.values(), workspace, ws_bytes, None,
                            check=False)


def test_qlinear_refusals():
    for bad in (dict(n=-1), dict(v=-1), dict(x_dtype=4), dict(out_dtype=3), dict(has_bias=2),
                dict(has_bias=1), dict(has_bias=1, bias=FAKE, bias_dtype=3), dict(bias=FAKE),
                dict(x_pitch=63), dict(weight_pitch=63), dict(out_pitch=99),
                dict(logit_scale=math.nan), dict(softcap=math.inf), dict(x=None),
                dict(weight=None), dict(weight_scale=None), dict(out=None), dict(x_scale=FAKE),
                dict(x_dtype=abi.FLCE_Q_I8), dict(flags=2), dict(reserved=1)):
        assert _qlinear(**bad) == INVALID, bad
    for bad in (dict(h=0), dict(h=131072, x_pitch=131072, weight_pitch=131072),
                dict(x=FAKE + 2), dict(weight=FAKE + 8), dict(out=FAKE + 1), dict(weight_scale=FAKE + 2),
                dict(has_bias=1, bias=FAKE + 2)):
        assert _qlinear(**bad) == UNSUPPORTED, bad
    assert _qlinear(ws_bytes=16) == WORKSPACE
    assert _qlinear(workspace=FAKE + 1) == WORKSPACE
    assert abi.flce_qlinear_workspace_size(abi.flce_qproblem()) == 0


def test_quantize_refusals():
    def call(x=FAKE, dtype=0, n=3, h=10, x_pitch=10, q=FAKE, q_pitch=16, scale=FAKE):
        return abi.flce_quantize_rows(x, dtype, n, h, x_pitch, q, q_pitch, scale, None,
                                      check=False)

    for bad in (dict(x=None), dict(q=None), dict(scale=None), dict(dtype=3), dict(n=-1),
                dict(h=0), dict(x_pitch=9), dict(q_pitch=9)):
        assert call(**bad) == INVALID, bad
    assert call(x=FAKE + 1) == UNSUPPORTED
    assert call(scale=FAKE + 2) == UNSUPPORTED


def test_int8_python_refusals():
    x, w, s = torch.zeros(3, 8), torch.zeros(5, 8, dtype=torch.int8), torch.zeros(5)
    with pytest.raises(ValueError, match="CUDA"):
        package.int8_linear(x, w, s)
    with pytest.raises(ValueError, match="CUDA"):
        package.quantize_rows(x)
    with pytest.raises(TypeError):
        package.quantize_rows(x.double())
    with pytest.raises(TypeError):
        package.int8_linear(x.double(), w, s)
    with pytest.raises(TypeError):
        package.int8_linear(x, w, s, out_dtype=torch.float64)


@pytest.mark.parametrize("vectors", [0xffffff01, 0xfffffff0, 0xfffffff1, 1 << 32])
def test_reorder_refuses_more_vectors_than_its_blocks_can_count(vectors):
    """A beam's vectors, rounded up to whole blocks of 256, stay below 2^32."""
    for width in (1, 2, 4, 8, 16):
        stride = (vectors + 1) * width
        assert _reorder(batch=1, beams=2, run_bytes=vectors * width, beam_stride=stride,
                        data=FAKE + width) == UNSUPPORTED, width
        assert "too large" in abi.flce_last_error()
        # the same in pieces
        if vectors % 16 == 0:
            assert _reorder(batch=1, beams=2, run_bytes=16 * width, size=(1, 1, 1, vectors // 16),
                            stride=(0, 0, 0, 17 * width), beam_stride=2 * stride + width,
                            data=FAKE + width) == UNSUPPORTED, width


@pytest.mark.parametrize("v", [(1 << 31) - 8192, (1 << 31) - 4096, (1 << 31) - 4095, (1 << 31) - 1])
def test_select_refuses_rows_whose_tiles_leave_32_bits(v):
    """Rows that share their memory make such a vocabulary one tensor of 4 GB."""
    for dtype in (abi.FLCE_F32, abi.FLCE_BF16, abi.FLCE_F16):
        for batch, beams in ((1, 1), (64, 8), (600, 1)):
            at = dict(batch=batch, beams=beams, dtype=dtype, stride_batch=0, stride_beam=0)
            assert _select(v=v, **at) == INVALID, (batch, beams)
            last = abi.flce_beam_problem(batch=batch, beams=beams, candidates=6, dtype=dtype,
                                         v=(1 << 31) - 8193)
            assert abi.flce_beam_select_workspace_size(last) > 0


@pytest.mark.filterwarnings("ignore:.*torch.jit:DeprecationWarning")
def test_gradients_are_refused_not_dropped():
    """Operators that have no gradient raise for inputs that ask for one, in reverse or forward
    mode, and go on (here to the missing device) under no_grad."""
    x, w, s = torch.zeros(3, 8), torch.zeros(5, 8, dtype=torch.int8), torch.zeros(5)
    z, b = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    calls = [
        (package.quantize_rows, (x,), {}, (0,)),
        (package.int8_linear, (x, w, s, s.clone()), {}, (0, 2, 3)),
        (package.beam_select, (z, b), {}, (0, 1)),
    ]
    for call, args, kw, floats in calls:
        for i in floats:
            asking = list(args)
            asking[i] = args[i].clone().requires_grad_(True)
            with pytest.raises(RuntimeError, match="no gradient"):
                call(*asking, **kw)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(*asking, **kw)
            with torch.autograd.forward_ad.dual_level():
                asking[i] = torch.autograd.forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(RuntimeError, match="tangent"):
                    call(*asking, **kw)
                with torch.no_grad(), pytest.raises(RuntimeError, match="tangent"):
                    call(*asking, **kw)
                with pytest.raises(ValueError, match="CUDA"):
                    call(*args, **kw)
    q = torch.zeros(3, 8, dtype=torch.int8)
    with pytest.raises(RuntimeError, match="no gradient"):
        package.int8_linear(q, w, s, x_scale=torch.zeros(3, requires_grad=True))


def test_docstrings_name_the_limits():
    """What the C entry points refuse for its size, a user reads beforehand."""
    assert "at most 256" in package.beam_select.__doc__
    assert "K at most 1024" in package.beam_select.__doc__
    assert _select(candidates=257) == UNSUPPORTED and _select(beams=1025) == UNSUPPORTED
    assert "K is at most 64" in package.beam_reorder_.__doc__
    assert _reorder(beams=65) == UNSUPPORTED
    assert "H at\n    most 131071" in package.int8_linear.__doc__
    assert _qlinear(h=131072, x_pitch=131072, weight_pitch=131072) == UNSUPPORTED


def test_grad_overlaps_with_a_refusal_behind():
    """Which memory counts as shared: calls without any get as far as the next check, which
    refuses them for their max_norm, so that no made-up address reaches a device."""
    far = 0x900000

    def shared(*grads):
        assert _clip(*grads, max_norm=-1.0) == INVALID
        text = abi.flce_last_error()
        assert ("overlap" in text) != ("max_norm" in text), text
        return "overlap" in text

    rows = dict(rows=9, cols=40, src_pitch=100, dst_pitch=100)
    assert not shared(_grad(), _grad(src=FAKE + 400, dst=FAKE + 400))
    assert not shared(_grad(dst=far), _grad(dst=far + 400))  # one source, read twice
    assert not shared(_grad(**rows), _grad(src=FAKE + 160, dst=FAKE + 160, **rows))
    assert not shared(_grad(rows=0), _grad())
    assert shared(_grad(), _grad())
    assert shared(_grad(src=far, dst=FAKE + 396), _grad())
    assert shared(_grad(dst=FAKE + 4))
    assert shared(_grad(**rows), _grad(src=FAKE + 156, dst=FAKE + 156, **rows))
    assert shared(_grad(**rows), _grad(src=FAKE + 244, dst=FAKE + 244, **rows))


def test_softcap_without_a_reciprocal_is_refused():
    """The cap divides: one whose reciprocal overflows would make a logit of 0 NaN."""
    assert _qlinear(softcap=1e-39) == INVALID
    assert "softcap" in abi.flce_last_error()
    assert _qlinear(softcap=3e-39, ws_bytes=16) == WORKSPACE  # as far as the next check
    assert _qlinear(softcap=-1e-39, ws_bytes=16) == WORKSPACE  # no cap


@pytest.mark.parametrize("count", [2, 5, 64, 65, 300])
def test_reorder_refuses_a_state_that_is_listed_twice(count):
    """Two states of one address share its byte: moved twice, in no order, they would be garbage.
    Lists without such a pair get as far as the check of the last state, which is refused for
    its own sake, so that no made-up address reaches a device."""
    def call(addresses):
        states = [(a, 1000, 1000) for a in addresses] + [(FAKE, 999, 1000)]
        table = (abi.flce_beam_state * len(states))(*[
            abi.flce_beam_state(a, stride, (ctypes.c_int64 * 4)(1, 1, 1, 1),
                                (ctypes.c_int64 * 4)(0, 0, 0, 0), run)
            for a, stride, run in states])
        n = len(states) if addresses[0] != addresses[-1] else len(states) - 1
        assert abi.flce_beam_reorder(ctypes.addressof(table), n, FAKE, 2, 3, None, None,
                                     check=False) == INVALID
        return abi.flce_last_error()

    far = [0x100000 + 6000 * i for i in range(count)]
    assert "elements overlap" in call(far)
    assert "twice" in call(far[:-1] + far[:1])


def test_reorder_empty_states_share_nothing():
    """States without bytes may have any address; the last of these is refused for its own sake."""
    states = [(FAKE, 0), (FAKE, 0), (FAKE, -1)]
    table = (abi.flce_beam_state * 3)(*[
        abi.flce_beam_state(a, 1000, (ctypes.c_int64 * 4)(1, 1, 1, 1),
                            (ctypes.c_int64 * 4)(0, 0, 0, 0), run) for a, run in states])
    assert abi.flce_beam_reorder(ctypes.addressof(table), 3, FAKE, 2, 3, None, None,
                                 check=False) == INVALID
    assert "run_bytes" in abi.flce_last_error()
