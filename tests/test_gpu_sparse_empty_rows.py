"""Rows that list nothing, and tiles that a row did not list, whose scores are not finite: padded rows that hold NaN or infinities,
and keys so large that a neighbour's scores overflow.  They count for nothing, bit for bit."""

import numpy as np
import pytest

from tests.test_gpu_append import kb, randn  # noqa: F401
from tests.test_gpu_sparse import random_lists

pytestmark = pytest.mark.gpu


def same(a, b):
    import torch

    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("S,n", [(40, 1), (300, 2), (900, 4)])
def test_padded_rows_may_hold_anything(kb, value, S, n):
    """Rows that list nothing between rows that do: their own results are zero and nobody else's change."""
    import torch

    q, k, v, dout = (randn(5000 + i, 2, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = random_lists(5004, 2, S, 0, n)
    empty = torch.from_numpy(np.random.default_rng(5).random(S) < 0.4).cuda()
    empty[-5:] = True
    lists[:, :, empty] = -1
    q[:, :, empty] = 0
    dout[:, :, empty] = 0
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    want = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)
    padded_q, padded_dout = q.clone(), dout.clone()
    padded_q[:, :, empty] = value
    padded_dout[:, :, empty] = value
    got_o, got_lse = kb.sparse_prefill_lse(padded_q, k, v, lists)
    assert bool((got_o[:, :, empty] == 0).all()) and bool((got_lse[:, :, empty] == float("-inf")).all())
    assert same(got_o, o) and same(got_lse, lse)
    got = kb.sparse_backward(padded_q, k, v, got_o, padded_dout, got_lse, lists, check=True)
    assert bool((got[0][:, :, empty] == 0).all())
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x, y)
    chunk = kb.sparse_chunk(padded_q, k, v, 0, lists, check=True)
    assert same(chunk, o)


@pytest.mark.parametrize("value", [3e38, float("inf"), float("nan")])
def test_keys_of_a_block_that_only_neighbours_list(kb, value):
    """Every other row lists a block of keys whose scores overflow; the rows between have the bits they have as tokens."""
    import torch

    L, cap = 200, 1024
    start = cap - L
    q, k, v = randn(5100, 1, 32, L, 128), randn(5101, 1, 8, cap, 128), randn(5102, 1, 8, cap, 128)
    k[:, :, 128:256] = value
    lists = torch.tensor([0, 2, 4, -1], dtype=torch.int32, device="cuda").expand(1, 8, L, 4).clone()
    lists[:, :, ::2, 3] = 1
    o = kb.sparse_chunk(q, k, v, start, lists, check=True)
    assert bool(torch.isfinite(o[:, :, 1::2]).all())
    for i in (1, 17, 33, 199):
        token = kb.sparse_decode(q[:, :, i:i + 1].contiguous(), k, v, start + i + 1, lists[:, :, i:i + 1].contiguous(), check=True)
        assert same(token[:, :, 0], o[:, :, i])
