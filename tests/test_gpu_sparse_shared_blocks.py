"""dk and dv of key blocks that two CTAs share, over patterns of the rows that list them: full, sparse and empty stretches, gaps,
tails that list nothing, and a first half that ends inside a stretch."""

import numpy as np
import pytest

from tests.test_gpu_append import f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu

# rows that list the block in each 1024 positions from the block's first on, per KV head (4065 rows or more are shared)
PATTERNS = [(1024, 1014, 25, 0, 1024, 1010), (1024, 1024, 1, 0, 1024, 1000), (1024,) * 6, (700, 690, 680, 670, 700, 705),
            (1024, 1024, 1024, 1003, 0, 0), (1000, 1000, 40, 30, 1024, 1024), (1024, 1023, 3, 0, 1023, 1024),
            (1024, 1024, 0, 0, 1008, 1008)]


def block_gradients(q, k, v, dout, pos, first):
    """dk, dv [128, 128] of the keys k, v [128, 128] at positions first .. first + 127, from rows q, dout [4, R, 128] at
    positions pos [R] that list this block and no other."""
    s = np.where(np.arange(128) + first <= pos[:, None], q @ k.T / np.sqrt(128.0), -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    dp = dout @ v.T
    ds = p * (dp - (p * dp).sum(-1, keepdims=True)) / np.sqrt(128.0)
    return np.einsum("grs,grd->sd", ds, q), np.einsum("grs,grd->sd", p, dout)


@pytest.mark.parametrize("block", [0, 3])
def test_patterns_of_listing_rows(kb, block):
    """Three or four independent roundings to bf16 (P or dS, the result, the output behind delta), each at most 2^-8 / sqrt 3
    of a value root mean square, make 0.0045; one lost position of 4097 is 0.0156, one counted twice as much."""
    import torch

    first = 128 * block
    S = first + 1024 * len(PATTERNS[0])
    rng = np.random.default_rng(40 + block)
    lists = np.broadcast_to((np.arange(S) // 128)[:, None], (1, 8, S, 1)).astype(np.int32).copy()
    rows = []
    for g, counts in enumerate(PATTERNS):
        at = np.concatenate([first + 1024 * w + (np.arange(c) if g % 2 == 0 else np.sort(rng.permutation(1024)[:c]))
                             for w, c in enumerate(counts)])
        lists[0, g, first:first + 128] = -1                            # the block's own rows list it by the pattern alone
        lists[0, g, at] = block
        rows.append(at)
    lists = torch.from_numpy(lists).cuda()
    q, k, v, dout = (randn(4000 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    _, dk, dv, _ = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)
    q, dout = f64(q)[0], f64(dout)[0]
    k, v, dk, dv = (f64(x)[0, :, first:first + 128] for x in (k, v, dk, dv))
    for g, at in enumerate(rows):
        h = slice(4 * g, 4 * g + 4)
        want = block_gradients(q[h][:, at], k[g], v[g], dout[h][:, at], at, first)
        for name, x, y in zip(("dk", "dv"), (dk[g], dv[g]), want):
            err = np.sqrt(((x - y) ** 2).mean() / (y ** 2).mean())
            assert err <= 0.0045, (name, PATTERNS[g], err)
