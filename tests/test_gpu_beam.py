"""The beam choice and the reordering against 64-bit and indexed forms.

Tolerances. An exponential's argument is off by at most 2 * 2^-24 of itself (a difference and a
product; beyond 30 its weight is below e^-30) and the function by 2^-22: 30 * 2^-22 relative. The
sums add at most 25 roundings. So a beam's lse is within 8e-6, and a score within that and half a
step of its 32 bits. Two candidates of different beams may change places only where their scores
are closer than twice that; candidates of one beam never do.
"""
import math

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import abi, beam_reorder_, beam_select

pytestmark = pytest.mark.gpu

LSE_ABS = 8e-6


def _scores64(logits, scores, finished=None, allowed=None, pad=0):
    b, k, v = logits.shape
    z = logits.double()
    if allowed is not None:
        z = torch.where(allowed, z, -math.inf)
    lse = torch.logsumexp(z, 2, keepdim=True)
    s = torch.where(lse > -math.inf, z - lse, -math.inf) + scores.double().unsqueeze(2)
    if finished is not None:
        s[finished] = -math.inf
        s[:, :, pad] = torch.where(finished, scores.double(), s[:, :, pad])
    return s


def _check(got, s, m, pad=0):
    b, k, v = s.shape
    want, at = torch.sort(s.reshape(b, -1), dim=1, descending=True, stable=True)
    if k * v < m:
        want = torch.nn.functional.pad(want, (0, m - k * v), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, m - k * v))
    want, at = want[:, :m], at[:, :m]
    some = want > -math.inf
    assert got.scores.shape == got.parents.shape == got.tokens.shape == (b, m)
    assert torch.equal(got.scores > -math.inf, some)
    assert bool((got.parents[~some] == 0).all()) and bool((got.tokens[~some] == pad).all())
    flat = got.parents * v + got.tokens
    # the scores of what was chosen, and of what should have been
    mine = torch.gather(s.reshape(b, -1), 1, flat)
    err = (got.scores.double() - mine)[some].abs()
    assert bool((err <= LSE_ABS + 2.0 ** -24 * mine[some].abs()).all())
    assert bool(((mine - want)[some].abs() <= 2 * LSE_ABS).all())
    differ = (flat != at) & some
    for i in range(b):
        chosen = flat[i][some[i]].tolist()
        assert len(set(chosen)) == len(chosen)
        if bool(differ[i].any()):  # only near ties of different beams
            for j in torch.nonzero(differ[i]).flatten().tolist():
                assert int(got.parents[i, j]) != int(at[i, j]) // v, (i, j)


def _make(b, k, v, dtype, seed=0, std=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    logits = (torch.randn(b, k, v, generator=g, device="cuda") * std).to(dtype)
    return logits, torch.rand(b, k, generator=g, device="cuda") * -8.0, g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,k,v,m", [
    (1, 1, 1, 1), (1, 1, 3, 5), (2, 3, 7, 6), (1, 4, 2047, 8), (3, 2, 2048, 4), (2, 5, 2049, 10),
    (1, 4, 32000, 8), (5, 3, 9001, 33), (2, 16, 1000, 256), (1, 2, 128256, 64), (40, 8, 8193, 16),
    (1, 70, 300, 100), (64, 6, 8200, 1),
])
def test_select(b, k, v, m, dtype):
    logits, scores, _ = _make(b, k, v, dtype, seed=b + v)
    _check(beam_select(logits, scores, m), _scores64(logits, scores), m)


@pytest.mark.parametrize("shape", ["all", "batch", "beam"])
@pytest.mark.parametrize("v,share", [(500, 0.5), (9001, 0.02), (32001, 0.0003), (8192, 1.0)])
def test_masks(v, share, shape):
    b, k, m = 3, 4, 8
    logits, scores, g = _make(b, k, v, torch.bfloat16, seed=v)
    size = {"all": (v,), "batch": (b, 1, v), "beam": (b, k, v)}[shape]
    allowed = torch.rand(size, generator=g, device="cuda") < share
    if shape != "all":
        allowed[1, 0] = False  # nothing may come
    wide = allowed.expand(b, k, v)
    # masked places hold what they like
    junk = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min],
                        device="cuda")
    pick = torch.randint(0, 4, (b, k, v), generator=g, device="cuda")
    logits = torch.where(wide, logits.float(), junk[pick]).bfloat16()
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    got = beam_select(logits, scores, m, allowed=allowed, err_word=err)
    _check(got, _scores64(logits.nan_to_num(0.0), scores, allowed=wide), m)
    assert int(err) == 0


def test_finished_and_dead_beams():
    b, k, v, m = 4, 5, 3000, 10
    logits, scores, g = _make(b, k, v, torch.float16)
    finished = torch.rand(b, k, generator=g, device="cuda") < 0.5
    finished[3] = True
    scores[0, 1] = -math.inf
    scores[1] = -math.inf
    logits[finished] = math.nan  # not read
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    got = beam_select(logits, scores, m, finished=finished, pad_token=17, err_word=err)
    s = _scores64(logits.nan_to_num(0.0), scores, finished=finished, pad=17)
    _check(got, s, m, pad=17)
    assert int(err) == 0
    # each finished beam keeps its score as it was
    for j in range(k):
        assert float(got.scores[3, j]) in scores[3].tolist()
    assert bool((got.scores[1] == -math.inf).all())


def test_equal_scores_take_the_lowest_index():
    for dtype in (torch.float32, torch.bfloat16):
        for v in (100, 2500, 40000):
            logits = torch.zeros(2, 3, v, dtype=dtype, device="cuda")
            scores = torch.zeros(2, 3, device="cuda")
            got = beam_select(logits, scores, 6)
            assert got.tokens.tolist() == [[0, 1, 2, 3, 4, 5]] * 2
            assert got.parents.tolist() == [[0] * 6] * 2
            # +0 and -0 are one value
            logits[:, :, ::2] = -0.0
            assert beam_select(logits, scores, 6).tokens.tolist() == [[0, 1, 2, 3, 4, 5]] * 2
            # equal beams: the first one's tokens come first, then the second's
            logits[:, :, 50] = 3.0
            logits[:, :, 7] = 3.0
            got = beam_select(logits, scores, 6)
            assert got.tokens.tolist() == [[7, 50] * 3] * 2
            assert got.parents.tolist() == [[0, 0, 1, 1, 2, 2]] * 2
    # whole numbers: many ties within and across beams
    g = torch.Generator("cuda").manual_seed(1)
    row = torch.randint(-3, 4, (1, 1, 5000), generator=g, device="cuda").float()
    logits = row.expand(2, 4, 5000).contiguous()
    scores = torch.zeros(2, 4, device="cuda")
    got = beam_select(logits, scores, 250)
    order = torch.sort(logits.reshape(2, -1), dim=1, descending=True, stable=True).indices[:, :250]
    assert torch.equal(got.parents * 5000 + got.tokens, order)


@pytest.mark.parametrize("v", [40000, 40001, 40006])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_slices(dtype, v):
    """Slices of several tiles: equal logits that overflow the list of candidates, logits that only
    rise and only fall, a mask that opens late, and ordinary ones."""
    b, k, m = 64, 8, 16
    logits, scores, g = _make(b, k, v, dtype)
    _check(beam_select(logits, scores, m), _scores64(logits, scores), m)
    # a row's scores do not depend on where it lies
    part = logits[5:9, :, 3:].contiguous()
    assert all(torch.equal(x, y) for x, y in zip(beam_select(logits[5:9, :, 3:], scores[5:9], m),
                                                 beam_select(part, scores[5:9], m)))
    late = torch.arange(v, device="cuda") >= v - 3000
    _check(beam_select(logits, scores, m, allowed=late),
           _scores64(logits, scores, allowed=late.expand(b, k, v)), m)
    few = torch.arange(v, device="cuda") % 4099 == 7
    _check(beam_select(logits, scores, m, allowed=few),
           _scores64(logits, scores, allowed=few.expand(b, k, v)), m)
    scores = scores - 100.0 * torch.arange(k, device="cuda")  # the first beam alone counts
    logits[:, :2] = 1.5
    got = beam_select(logits, scores, m)
    assert got.tokens.tolist() == [list(range(m))] * b and not bool(got.parents.any())
    _check(got, _scores64(logits, scores), m)
    logits[:, 0] = torch.linspace(-9, 9, v, device="cuda").to(dtype)
    _check(beam_select(logits, scores, m), _scores64(logits, scores), m)
    logits[:, 0] = logits[:, 0].flip(1)
    _check(beam_select(logits, scores, m), _scores64(logits, scores), m)
    logits[:, 0] = -math.inf
    logits[:, 0, -1] = 0.25
    got = beam_select(logits, scores, m)
    assert got.tokens[:, 0].tolist() == [v - 1] * b
    _check(got, _scores64(logits, scores), m)


def test_strided_logits():
    """The last position of a longer output, a padded vocabulary, rows at odd addresses."""
    g = torch.Generator("cuda").manual_seed(5)
    whole = torch.randn(2, 3, 4, 5003, generator=g, device="cuda").bfloat16()
    scores = torch.rand(2, 3, generator=g, device="cuda")
    for view in (whole[:, :, -1], whole[:, :, 1, :5001], whole[:, :, 2, 1:], whole[:, :, 0, 3:4003],
                 whole.permute(0, 1, 3, 2)[..., 1]):
        _check(beam_select(view, scores, 6), _scores64(view, scores), 6)
        assert all(torch.equal(x, y) for x, y in zip(beam_select(view, scores, 6),
                                                     beam_select(view.contiguous(), scores, 6)))
    one = whole[:, :1, 0].expand(2, 3, 5003)
    _check(beam_select(one, scores, 6), _scores64(one, scores), 6)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_not_finite(bad):
    logits, scores, _ = _make(2, 3, 4000, torch.float32)
    logits[0, 1, 3999] = bad
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    got = beam_select(logits, scores, 6, err_word=err)
    assert int(err) == abi.FLCE_DEVERR_NOT_FINITE
    assert 1 not in got.parents[0].tolist()
    rest = scores.clone()
    rest[0, 1] = -math.inf
    logits[0, 1, 3999] = 0.0
    _check(got, _scores64(logits, rest), 6)
    err.zero_()
    scores[1, 0] = bad
    got = beam_select(logits, scores, 6, err_word=err)
    assert int(err) == abi.FLCE_DEVERR_NOT_FINITE and 0 not in got.parents[1].tolist()


def test_extreme_logits():
    """The type's lowest and highest finite values, and all but one at -inf."""
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        lo, hi = torch.finfo(dtype).min, torch.finfo(dtype).max
        logits = torch.full((1, 3, 3001), lo, dtype=dtype, device="cuda")
        logits[0, 1, 5] = hi
        logits[0, 2] = -math.inf
        logits[0, 2, 2999] = lo
        scores = torch.tensor([[-1.0, -2.0, -3.0]], device="cuda")
        got = beam_select(logits, scores, 4)
        assert got.tokens[0, :3].tolist() == [5, 2999, 0]
        assert got.parents[0, :3].tolist() == [1, 2, 0]
        assert abs(float(got.scores[0, 0]) + 2.0) <= LSE_ABS
        assert abs(float(got.scores[0, 1]) + 3.0) <= LSE_ABS
        assert abs(float(got.scores[0, 2]) + 1.0 + math.log(3001)) <= LSE_ABS + 1e-6


def test_select_streams_and_graph():
    logits, scores, _ = _make(3, 4, 20000, torch.bfloat16)
    first = beam_select(logits, scores, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [beam_select(logits, scores, 8) for _ in range(10)]
    side.synchronize()
    assert all(torch.equal(x, y) for a in again for x, y in zip(a, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = beam_select(logits, scores, 8)
    for seed in range(3):
        logits.copy_(_make(3, 4, 20000, torch.bfloat16, seed=seed + 9)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, beam_select(logits, scores, 8)))


def test_empty_batch():
    got = beam_select(torch.zeros(0, 2, 5, device="cuda"), torch.zeros(0, 2, device="cuda"), 3)
    assert got.scores.shape == (0, 3) and got.tokens.shape == (0, 3)


# --------------------------------------------------------------- reordering
def _rows(parents):
    b, k = parents.shape
    return (parents + torch.arange(b, device="cuda").unsqueeze(1) * k).reshape(-1)


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 13, 16, 31, 32, 33, 64])
def test_reorder_beams(k):
    g = torch.Generator("cuda").manual_seed(k)
    for b in (1, 3):
        parents = torch.randint(0, k, (b, k), generator=g, device="cuda")
        states = [torch.randn(b * k, 4, 17, 64, generator=g, device="cuda").bfloat16(),
                  torch.randint(0, 1 << 40, (b * k, 37), generator=g, device="cuda"),
                  torch.rand(b * k, generator=g, device="cuda"),
                  torch.rand(b * k, 3, generator=g, device="cuda") < 0.5]
        want = [s[_rows(parents)] for s in states]
        assert beam_reorder_(states, parents) is None
        assert all(torch.equal(s, w) for s, w in zip(states, want))


def test_reorder_swaps_and_cycles():
    state = torch.arange(6, device="cuda").repeat_interleave(1000).view(6, 1000).clone()
    beam_reorder_(state, torch.tensor([[5, 0, 1, 2, 3, 4]], device="cuda"))
    assert state[:, 0].tolist() == [5, 0, 1, 2, 3, 4] and bool((state == state[:, :1]).all())
    beam_reorder_(state, torch.tensor([[1, 0, 2], [2, 2, 2]], device="cuda"))
    assert state[:, 999].tolist() == [0, 5, 1, 4, 4, 4]


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float32, torch.complex64])
def test_reorder_layouts(dtype):
    """The beam axis anywhere, filled parts of caches, odd sizes and addresses; what lies outside
    the view stays."""
    g = torch.Generator("cuda").manual_seed(2)
    b, k = 2, 3
    parents = torch.tensor([[1, 1, 0], [0, 2, 1]], device="cuda")

    def make(*shape):
        return torch.randint(0, 100, shape, generator=g, device="cuda").to(dtype)

    cases = [
        (make(5, 6, 4, 32, 16), lambda x: x[:, :, :, :7], 1),
        (make(5, 6, 4, 32, 16), lambda x: x[1:, :, 1:, 3:4, 2:9], 1),
        (make(6, 1001), lambda x: x[:, 1:], 0),
        (make(6, 1001), lambda x: x[:, ::7], 0),
        (make(3, 5, 6), lambda x: x, -1),
        (make(7, 6, 2, 3, 5, 8), lambda x: x[:, :, :, :2, :3], 1),
        (make(6, 0, 4), lambda x: x, 0),
    ]
    for whole, view, dim in cases:
        was = whole.clone()
        x = view(whole)
        d = dim % x.dim()
        want = x.index_select(d, _rows(parents))
        beam_reorder_([x], parents, dim=dim)
        assert torch.equal(x, want)
        y = view(was)
        y.copy_(want)
        assert torch.equal(whole, was)


def test_reorder_many_states_of_all_widths():
    g = torch.Generator("cuda").manual_seed(8)
    parents = torch.randint(0, 4, (3, 4), generator=g, device="cuda")
    states = [torch.randint(0, 255, (12, 1 + 5 * i % 64), generator=g, device="cuda").to(
        [torch.uint8, torch.int16, torch.int32, torch.int64][i % 4]) for i in range(200)]
    want = [s[_rows(parents)] for s in states]
    beam_reorder_(states, parents)
    assert all(torch.equal(s, w) for s, w in zip(states, want))


def test_reorder_parent_out_of_range():
    state = torch.arange(8, device="cuda").view(8, 1).repeat(1, 100).contiguous()
    err = torch.zeros((), dtype=torch.int32, device="cuda")
    beam_reorder_(state, torch.tensor([[1, 4, -1, 0], [0, 1, 2, 3]], device="cuda"), err_word=err)
    assert int(err) == abi.FLCE_DEVERR_PARENT_RANGE
    assert state[:, 0].tolist() == [1, 1, 2, 0, 4, 5, 6, 7]


def test_reorder_beyond_32_bit_offsets():
    """A cache whose last beam starts more than 2^32 bytes from its first."""
    state = torch.empty(3, 1 << 31, dtype=torch.uint8, device="cuda")
    for j in range(3):
        state[j].fill_(j + 1)
    part = state[:, -70001:]
    beam_reorder_(part, torch.tensor([[2, 0, 1]], device="cuda"))
    assert [int(x) for x in state[:, -70001]] == [3, 1, 2]
    assert [int(x) for x in state[:, -1]] == [3, 1, 2]
    assert [int(x) for x in state[:, -70002]] == [1, 2, 3]


def test_reorder_graph():
    state = torch.arange(4, device="cuda").view(4, 1).repeat(1, 50).contiguous()
    parents = torch.zeros(1, 4, dtype=torch.int64, device="cuda")
    beam_reorder_(state.clone(), parents)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        beam_reorder_(state, parents)
    state.copy_(torch.arange(4, device="cuda").view(4, 1))
    parents.copy_(torch.tensor([[3, 2, 1, 0]]))
    graph.replay()
    assert state[:, 49].tolist() == [3, 2, 1, 0]


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_reorder_autograd_sees_the_change(order):
    """States that mix inference tensors, which have no version, with others."""
    with torch.inference_mode():
        plain = torch.arange(4, device="cuda")
    a = torch.arange(4, device="cuda")
    both = [(plain, a)[i] for i in order]
    parents = torch.tensor([[1, 0], [1, 0]], device="cuda")
    for inside in (False, True):
        with torch.inference_mode(inside):
            was = a._version
            beam_reorder_(both, parents)
            assert a._version == was + 1
            beam_reorder_(plain, parents)
    assert a.tolist() == [0, 1, 2, 3] and plain.tolist() == [0, 1, 2, 3]
    beam_reorder_([], parents)


def test_reorder_states_that_interleave():
    """Keys and values side by side in one buffer are two states; one of them twice is refused."""
    g = torch.Generator("cuda").manual_seed(4)
    both = torch.randn(6, 2, 4, 33, generator=g, device="cuda")
    parents = torch.tensor([[1, 2, 0], [0, 0, 2]], device="cuda")
    want = both[_rows(parents)]
    was = both.clone()
    with pytest.raises(RuntimeError, match="twice"):
        beam_reorder_([both[:, 0], both[:, 1], both[:, 0]], parents)
    assert torch.equal(both, was)
    beam_reorder_([both[:, 0], both[:, 1]], parents)
    assert torch.equal(both, want)
    one = torch.arange(3, device="cuda")  # a single beam never moves
    beam_reorder_([one, one], torch.zeros(3, 1, dtype=torch.int64, device="cuda"))
    assert one.tolist() == [0, 1, 2]
