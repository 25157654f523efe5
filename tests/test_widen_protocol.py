"""The stage ring between the weight's copies and the widening warps of the 8-bit linear kernel, on
the CPU: copies land in any order, groups of warps take stages in turn, and every wait is for the
parity of a phase. For the ring sizes that the launcher picks, no group may pass a wait before its
stage has landed; sizes that its rule leaves out are shown to fail."""
import random

import pytest

GROUPS, SLOTS, STAGE, BUDGET = 3, 4, 16384, 224 * 1024


def _allowed(w):
    return w % GROUPS == 0 or w >= GROUPS + SLOTS


def _rings():
    """(weight stages, x stages) of every tile, by the launcher's rule."""
    found = set()
    for cg, nts in ((1, range(16, 129, 16)), (2, range(32, 257, 32))):
        for nt in nts:
            box = 2 * (nt // cg * 128)
            w = 12
            while w > GROUPS and (not _allowed(w) or BUDGET - w * STAGE < 4 * box):
                w -= 1
            x = min(12, (BUDGET - w * STAGE) // box)
            assert x >= 4 and w * STAGE + x * box <= BUDGET and _allowed(w)
            found.add((w, x))
    return sorted(found)


class Phase:
    """An mbarrier as a waiter sees it: phases completed, and a wait on a parity."""

    def __init__(self):
        self.done = 0

    def passed(self, parity):
        # true where the phase under way has the other parity
        return self.done % 2 != parity


def _run(w, seed, stages=200):
    """False when a group passed a wait before its stage had landed."""
    rng = random.Random(seed)
    full, empty = [Phase() for _ in range(w)], [Phase() for _ in range(w)]
    a_full, a_empty = [Phase() for _ in range(SLOTS)], [Phase() for _ in range(SLOTS)]
    landed, flying, issued, mma = set(), [], 0, 0
    groups = [{"i": g, "loaded": False} for g in range(GROUPS)]
    idle = 0
    while mma < stages:
        assert idle < 2000, "the ring stands still"
        idle += 1
        actor = rng.randrange(4)
        if actor == 0 and issued < stages and empty[issued % w].passed(issued // w % 2 ^ 1):
            flying.append(issued)
            issued, idle = issued + 1, 0
        elif actor == 1 and flying and rng.random() < 0.3:
            j = flying.pop(rng.randrange(len(flying)))
            landed.add(j)
            full[j % w].done += 1
            idle = 0
        elif actor == 2:
            g = rng.choice(groups)
            i = g["i"]
            if i >= stages:
                continue
            if not g["loaded"] and full[i % w].passed(i // w % 2):
                if i not in landed:
                    return False
                g["loaded"], idle = True, 0
            elif g["loaded"] and a_empty[i % SLOTS].passed(i // SLOTS % 2 ^ 1):
                empty[i % w].done += 1
                a_full[i % SLOTS].done += 1
                g["i"], g["loaded"], idle = i + GROUPS, False, 0
        elif actor == 3 and a_full[mma % SLOTS].passed(mma // SLOTS % 2):
            assert all(g["i"] > mma for g in groups if g["i"] % GROUPS == mma % GROUPS)
            a_empty[mma % SLOTS].done += 1
            mma, idle = mma + 1, 0
    return True


@pytest.mark.parametrize("w,x", _rings())
def test_ring_is_safe(w, x):
    assert all(_run(w, seed) for seed in range(60))


@pytest.mark.parametrize("w", [4, 5])
def test_other_sizes_are_not(w):
    assert not _allowed(w) and not all(_run(w, seed) for seed in range(60))
