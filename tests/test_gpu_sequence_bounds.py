"""Starts beyond any cache, up to the largest 32-bit number, are reported by every call that takes them, and the next call
is as ever."""

import pytest

from tests.test_gpu_append import bits, kb, randn  # noqa: F401
from tests.test_gpu_cache8 import bf16_of, filled

pytestmark = pytest.mark.gpu


def i32(*x):
    import torch

    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("L", [1, 2, 3, 32, 33, 130, 512])
def test_far_starts_are_reported(kb, page, L):
    import torch

    cap = 1024
    cache, pages, seq = filled(kb, 2, cap, page, seed=3)
    k, v = bf16_of(kb, cache, pages, seq, 2)
    pools = [kb.cache_values(c, e) for c, e in zip(cache[:2], cache[2:])]
    q, lse, w = randn(4, 2, 32, L, 128), torch.zeros(2, 32, L, device="cuda"), torch.zeros(2, 8, cap, device="cuda")
    lens = i32(L, L)
    calls = [lambda st: kb.chunk_varlen(q, *pools, st, lens, block_table=pages, check=True),
             lambda st: kb.chunk_lse_varlen(q, *pools, st, lens, block_table=pages, check=True)[0],
             lambda st: kb.chunk_8bit_varlen(q, *cache, st, lens, block_table=pages, check=True)]
    want = kb.chunk(q, k, v, cap - L, check=True)
    for call in calls:
        for far in (cap - L + 1, 2 ** 31 - L - 1, 2 ** 31 - L, 2 ** 31 - 1):
            for st in (i32(far, 0), i32(0, far)):
                with pytest.raises(kb.KBError):
                    call(st)
        assert torch.equal(bits(call(i32(cap - L, cap - L))), bits(want))
    for far in (cap - L + 1, 2 ** 31 - L, 2 ** 31 - 1):
        with pytest.raises(kb.KBError):
            kb.key_weights_varlen(q, pools[0], lse, w, i32(far, far), lens, block_table=pages, check=True)
        with pytest.raises(kb.KBError):
            kb.append_8bit_varlen(None, randn(5, 2, 8, L, 128), randn(6, 2, 8, L, 128), *cache, None, i32(far, far), lens,
                                  block_table=pages, check=True)
    assert bool((w == 0).all())
    assert torch.equal(bits(calls[2](i32(cap - L, cap - L))), bits(want))
