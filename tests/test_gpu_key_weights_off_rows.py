"""A row whose log-sum-exp is infinite gives no key anything, whatever stands in its query and in the keys, in every tile of
keys: the weights have the bits of a call in which nothing of it is odd."""

import pytest

from tests.test_gpu_append import kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu

S = 1000
SHAPES = [(1, 1), (1, 3), (2, 20), (1, 32), (1, 33), (2, 130), (1, 300), (1, 700)]


def off_rows(B, L):
    """[B, 32, L]: the first, the last and some rows between, all of one head, none of a group."""
    import torch

    off = torch.zeros(B, 32, L, dtype=torch.bool, device="cuda")
    off[:, ::3, 0] = True
    off[:, 1::5, L - 1] = True
    off[:, 2, ::7] = True
    off[:, 6] = True
    off[:, 28:] = False
    return off


@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("B,L", SHAPES)
def test_queries_of_rows_that_are_off(kb, B, L, odd, inf):
    import torch

    q, k = randn(1, B, 32, L, 128), randn(2, B, 8, S, 128)
    off = off_rows(B, L)
    lse = torch.where(off, inf, 5.0)
    want = torch.rand(B, 8, S, device="cuda")
    got = want.clone()
    kb.key_weights(q, k, lse, want, S - L, check=True)
    assert bool(torch.isfinite(want).all())
    q[off] = odd
    kb.key_weights(q, k, lse, got, S - L, check=True)
    assert torch.equal(got, want)


@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
@pytest.mark.parametrize("B,L", SHAPES)
def test_infinite_keys_of_rows_that_are_off(kb, B, L, inf):
    """Keys whose scores are +inf with the rows that are off, -inf with the others."""
    import torch

    q, k = randn(3, B, 32, L, 128), randn(4, B, 8, S, 128)
    off = off_rows(B, L)
    q[..., 5] = torch.where(off, 1.0, -1.0).bfloat16()
    lse = torch.where(off, inf, 5.0)
    want = torch.rand(B, 8, S, device="cuda")
    got, before = want.clone(), want.clone()
    kb.key_weights(q, k, lse, want, S - L, check=True)
    at = [0, 130, S - L - 1]
    k[:, :, at, 5] = float("inf")
    kb.key_weights(q, k, lse, got, S - L, check=True)
    assert torch.equal(got[:, :, at], before[:, :, at])
    got[:, :, at] = want[:, :, at]
    assert torch.equal(got, want)


def test_ragged_and_paged(kb):
    import torch

    B, L, page = 3, 150, 128
    q, pool = randn(5, B, 32, L, 128), randn(6, 26, 8, page, 128)
    pages = torch.randperm(26, generator=torch.Generator().manual_seed(7))[:24].view(3, 8).int().cuda()
    off = off_rows(B, L)
    lse = torch.where(off, float("inf"), 5.0)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ((800, 0, 300), (150, 150, 77)))
    want = torch.zeros(B, 8, 1024, device="cuda")
    got = want.clone()
    kb.key_weights_varlen(q, pool, lse, want, starts, lens, block_table=pages, check=True)
    q[off] = float("nan")
    kb.key_weights_varlen(q, pool, lse, got, starts, lens, block_table=pages, check=True)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())
