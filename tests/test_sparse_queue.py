"""The queue by which the dk/dv kernel's producers collect the positions that listed a key block, restated step by step:
the two shares of a block together take each position once, in order."""

import numpy as np
import pytest

UNIT, WINDOW = 32, 1024                 # positions a step takes; positions whose masks are read at a time
QUEUE = UNIT + WINDOW


def share_positions(listed, first, steps):
    """Positions that a CTA takes which begins at step `first` of the block and makes `steps` steps.  `listed`: bool per
    position from the block's first on."""
    queue = np.full(QUEUE, -1)
    window = used = queued = 0
    skip = first * UNIT
    taken = []
    for _ in range(steps):
        while queued - used < UNIT and window * WINDOW < len(listed):
            rest = queued - used
            assert rest == 0 or skip == 0
            queue[:rest] = queue[used:used + rest].copy()
            used, queued = 0, rest
            new = window * WINDOW + np.flatnonzero(listed[window * WINDOW:(window + 1) * WINDOW])
            window += 1
            if len(new) <= skip:
                skip -= len(new)
                continue
            queue[rest:rest + len(new)] = new
            used, skip, queued = skip, 0, rest + len(new)
        n = min(UNIT, queued - used)
        taken += list(queue[used:used + n])
        used += n
    return taken


def check(listed):
    rows = int(listed.sum())
    steps = -(-rows // UNIT)
    got = share_positions(listed, 0, steps // 2), share_positions(listed, steps // 2, steps - steps // 2)
    assert got[0] + got[1] == list(np.flatnonzero(listed))
    assert len(got[0]) == steps // 2 * UNIT
    assert share_positions(listed, 0, steps) == list(np.flatnonzero(listed))


@pytest.mark.parametrize("counts", [(1024, 1014, 25, 0, 1024, 1010), (1024, 1023, 3, 0, 1023, 1024), (1000, 1000, 40, 30, 1024),
                                    (1024,) * 6, (1024, 1024, 1024, 1003, 0, 0), (0, 0, 1024, 0, 1, 0, 31, 0, 1024, 33, 0, 1024, 1024)])
def test_shares_partition_the_rows(counts):
    listed = np.zeros(WINDOW * len(counts), bool)
    for w, c in enumerate(counts):
        listed[w * WINDOW:w * WINDOW + c] = True
    check(listed)


def test_shares_partition_random_rows():
    rng = np.random.default_rng(5)
    for _ in range(300):
        windows = int(rng.integers(1, 12))
        counts = np.where(rng.random(windows) < 0.4, rng.integers(0, 64, windows), rng.integers(0, WINDOW + 1, windows))
        counts[rng.random(windows) < 0.3] = 0
        listed = np.zeros(windows * WINDOW - int(rng.integers(0, WINDOW)), bool)
        for w, c in enumerate(counts):
            at = rng.permutation(WINDOW)[:c] + w * WINDOW
            listed[at[at < len(listed)]] = True
        check(listed)
