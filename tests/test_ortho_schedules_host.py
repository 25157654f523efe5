"""Which schedules of coefficients the orthogonalising operator takes (no GPU: the C entry point
answers before any CUDA call)."""
import ctypes

import pytest

from linear_cross_entropy_vocab_gb300 import abi, native_build

# published five-step schedule, each step tuned to the interval that the one before leaves
TUNED = ((8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518),
         (3.3184, -2.4885, 0.5100), (2.3007, -1.6690, 0.4188))
TUNED8 = TUNED + ((1.8913, -1.2680, 0.3768), (1.875, -1.25, 0.375), (1.875, -1.25, 0.375))
# another one, whose steps differ less
STEPWISE = ((4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037),
            (2.8769, -3.1427, 1.2046), (2.8366, -3.0525, 1.2012))
FAKE = 0x10000  # never dereferenced


def safe(schedule, factor=1.01):
    return tuple((a / factor, b / factor ** 3, c / factor ** 5) for a, b, c in schedule)


@pytest.fixture(scope="module", autouse=True)
def lib():
    native_build.build()
    return abi.load()


def _call(triples):
    table = (ctypes.c_float * (3 * len(triples)))(*[v for t in triples for v in t])
    p = abi.flce_ortho_problem(batch=1, rows=300, cols=500, batch_stride=0, row_pitch=500,
                               dtype=abi.FLCE_F32, out_dtype=abi.FLCE_BF16, steps=len(triples),
                               eps=1e-7, coefficients=ctypes.addressof(table), reserved=0)
    size = abi.flce_orthogonalize_workspace_size(p)
    st = abi.flce_orthogonalize(p, FAKE, FAKE, None, FAKE, 8, None, check=False)
    assert (size > 0) == (st == abi.FLCE_ERR_WORKSPACE)
    return st, abi.load().flce_last_error().decode()


def test_schedules_with_a_safety_factor_are_taken():
    for triples in (safe(TUNED), safe(TUNED[:-1]) + TUNED[-1:], safe(TUNED8),
                    safe(TUNED8[:-1]) + TUNED8[-1:], safe(TUNED, 1.02)):
        assert _call(triples)[0] == abi.FLCE_ERR_WORKSPACE, triples


def test_schedules_that_magnify_roundings_are_refused():
    """Just above 1 the first polynomial rises twelve times as fast as its value (24 / 1.99), and
    so do the next ones above where it ends: a value that a rounding takes 2^-11 past 1 is 12^4
    times as far off after four steps."""
    for triples in (TUNED, TUNED8, TUNED[:3]):
        st, why = _call(triples)
        assert st == abi.FLCE_ERR_UNSUPPORTED and "safety factor" in why, (triples, why)


def test_schedules_that_settle_are_taken():
    for triples in (((3.4445, -4.7750, 2.0315),) * 5, ((3.4445, -4.7750, 2.0315),) * 64,
                    ((1.5, -0.5, 0.0),) * 64, ((1.875, -1.25, 0.375),) * 64, ((1.0, 0.0, 0.0),) * 64,
                    ((2.0, -1.5, 0.5),) * 6, TUNED[:1], TUNED[:2], STEPWISE,
                    # the largest value at the top of each interval, 1 and 1.5 in turn
                    ((1.0, 0.5, 0.0), (0.3, 0.163, 0.0)) * 3):
        assert _call(triples)[0] == abi.FLCE_ERR_WORKSPACE, triples
