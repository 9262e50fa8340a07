"""Block selection with boxes that no call has made: infinities, NaN, any bit patterns.  Every row still gets a full list of
distinct blocks of its own, and nothing is written outside the lists."""

import numpy as np
import pytest

from tests.test_gpu_append import kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD = 4096                        # list entries kept free on either side


def garbage(kind, blocks):
    import torch

    g = torch.Generator(device="cuda").manual_seed(blocks)
    b = torch.randn(1, 8, blocks, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    if kind == "one +inf":
        b[0, :, blocks // 3, 0] = float("inf")
    elif kind == "one -inf":
        b[0, :, blocks // 3] = float("-inf")
    elif kind == "mostly nan":
        b[0, :, 3:] = float("nan")
    elif kind == "all nan":
        b[:] = float("nan")
    elif kind == "infinities":
        b[torch.rand(b.shape, generator=g, device="cuda") < 0.5] = float("inf")
        b[torch.rand(b.shape, generator=g, device="cuda") < 0.3] = float("-inf")
    else:
        b = torch.randint(-32768, 32768, b.shape, generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    return b


@pytest.mark.parametrize("kind", ["one +inf", "one -inf", "mostly nan", "all nan", "infinities", "any bits"])
@pytest.mark.parametrize("L,blocks,n", [(1, 40, 16), (1, 700, 128), (3, 300, 5), (200, 40, 16), (130, 250, 128), (200, 700, 16),
                                        (130, 700, 34), (17, 600, 60)])
def test_lists_are_full_and_nothing_else_is_written(kb, kind, L, blocks, n):
    import torch

    boxes = garbage(kind, blocks)
    start = blocks * 128 - L
    q = randn(70 + L, 1, 32, L, 128)
    wide = torch.full((2 * GUARD + 8 * L * n,), -77, dtype=torch.int32, device="cuda")
    out = wide[GUARD:GUARD + 8 * L * n].view(1, 8, L, n)
    kb.select_blocks(q, boxes, start, n, keep_first=2, keep_last=1, out=out, check=True)
    assert bool((wide[:GUARD] == -77).all()) and bool((wide[GUARD + 8 * L * n:] == -77).all())
    got = out.cpu().numpy()[0]
    last = (start + np.arange(L)) // 128
    for i in range(L):
        rows = got[:, i]
        full = min(n, last[i] + 1)
        assert np.all(np.diff(rows[:, :full], axis=-1) > 0) and np.all(rows[:, 0] == 0) and np.all(rows[:, 1] == 1), (i, rows)
        assert np.all(rows[:, full - 1] == last[i]) and np.all(rows[:, full:] == -1), (i, rows)
