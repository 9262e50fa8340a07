"""Tokens over an 8-bit cache of two to eight segments, whose CTAs meet in a cluster: sequences of different lengths, without a
row, out of range, on two streams, captured; and what a block that holds a NaN does to the rows that see it."""

import numpy as np
import pytest

from tests.test_gpu_append import bits, kb, randn  # noqa: F401
from tests.test_gpu_cache8 import bf16_of, empty8, filled

pytestmark = pytest.mark.gpu


def i32(*x):
    import torch

    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("cap,lens", [(2048, (1, 1024, 1025, 2048, 129)), (4096, (1, 1025, 4096)), (4096, (3073, 2049, 1024)), (8192, (8192,)),
                                      (7168, (5000, 7168)), (7168, (5000,)), (5120, (128, 5120)), (4864, (4097,)), (6144, (6143, 1))])
def test_contexts_of_any_length(kb, page, cap, lens):
    import torch

    B = len(lens)
    ns = -(-cap // 1024)
    in_clusters = B * 8 * ns <= (120 if ns <= 4 else 96)
    assert (kb.kb_attn_chunk_8bit_workspace_bytes(B, 8, 1, cap) == 0) == in_clusters     # (they need no workspace)
    cache, pages, seq = filled(kb, B, cap, page, seed=11)
    k, v = bf16_of(kb, cache, pages, seq, B)
    q = randn(12, B, 32, 1, 128)
    n = i32(*lens)
    want = torch.cat([kb.decode(q[b:b + 1], k[b:b + 1], v[b:b + 1], lens[b]) for b in range(B)])
    call = lambda n, on, out=None: kb.chunk_8bit_varlen(q, *cache, n - 1, on, block_table=pages, out=out, check=True)  # noqa: E731
    one = torch.ones_like(n)
    assert torch.equal(bits(call(n, one)), bits(want))
    if page:
        assert torch.equal(bits(kb.decode_8bit_paged(q, *cache, pages, n, check=True)), bits(want))
    else:
        got = [kb.decode_8bit(q, *cache, lens[b], check=True)[b:b + 1] for b in range(B)]
        assert torch.equal(bits(torch.cat(got)), bits(want))
    # every other sequence without a row, the first among them
    on = (torch.arange(B, device="cuda") % 2).int()
    out = torch.full_like(q, 7.0)
    call(n, on, out)
    assert torch.equal(bits(out[on == 1]), bits(want[on == 1])) and bool((out[on == 0] == 7.0).all())
    # a context beyond the cache, one far beyond it, a negative one: reported, and the next call is as ever
    for bad in (cap + 1, 2 ** 31 - 1, -5):
        broken = n.clone()
        broken[B - 1] = bad
        with pytest.raises(kb.KBError):
            call(broken, one)
        if page:
            with pytest.raises(kb.KBError):
                kb.decode_8bit_paged(q, *cache, pages, broken, check=True)
        assert torch.equal(bits(call(n, one)), bits(want))
    if page:
        broken = pages.clone()
        broken[0, (lens[0] - 1) // page] = -1
        with pytest.raises(kb.KBError):
            kb.decode_8bit_paged(q, *cache, broken, n, check=True)
        assert torch.equal(bits(kb.decode_8bit_paged(q, *cache, pages, n, check=True)), bits(want))


def test_on_two_streams_and_captured(kb):
    import torch

    B, cap = 2, 4096
    cache, _, seq = filled(kb, B, cap, seed=21)
    q, one = randn(22, B, 32, 1, 128), torch.ones(B, dtype=torch.int32, device="cuda")
    pos, out = i32(0, 0), torch.empty_like(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=streams[0]):
        kb.chunk_8bit_varlen(q, *cache, pos, one, out=out)
    for at in ((0, 4095), (1024, 1023), (2500, 3071), (4095, 4095)):
        pos.copy_(i32(*at))
        g.replay()
        want = kb.chunk_8bit_varlen(q, *cache, i32(*at), one, check=True)
        assert torch.equal(bits(out), bits(want))
    got = [kb.chunk_8bit_varlen(q, *cache, pos, one, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    kb.check_device_status()
    assert all(torch.equal(bits(x), bits(want)) for x in got)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("L", [1, 2, 5, 32, 40, 300])
def test_rows_that_see_a_marked_block(kb, L, bad):
    """A value that is not finite marks its block's keys (values): NaN in every row that sees one of them, in no other."""
    import torch

    S, at = 700, 400                                            # position 400 lies in block 3: keys 384..511
    for which in (0, 1):
        kv = [randn(31 + i, 1, 8, S, 128) for i in range(2)]
        kv[which][0, 5, at, 17] = bad
        cache = empty8(1, S)[:4]
        kb.append_8bit(None, *kv, *cache, None, 0, check=True)
        q = randn(33, 1, 32, L, 128)
        for start in (384 - L, 384, min(512 - min(L, 100), S - L), S - L):
            o = kb.chunk_8bit(q, *cache, start, check=True)
            nan = torch.isnan(o[0]).all(-1).cpu().numpy()       # [32, L]
            some = torch.isnan(o[0]).any(-1).cpu().numpy()
            want = np.zeros((32, L), bool)
            want[20:24] = np.arange(start, start + L) >= 384
            assert np.array_equal(nan, want) and np.array_equal(some, want), (which, start)


def test_refused_rotations_leave_their_arguments_alone(kb):
    import torch

    table, x, pos = kb.rope_table(50), randn(41, 1, 8, 9, 128), torch.zeros(1, 1, 9, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 3.0)
    kept = [t.clone() for t in (table, x, pos, out)]
    for planes, p in (([1] * 64, pos), ([0] * 63, pos), ([0] * 64, pos[:, :, :8].contiguous()), ([-1] + [0] * 63, pos)):
        with pytest.raises(ValueError):
            kb.rope_axes(x, table, p, planes, out=out)
    kb.check_device_status()
    assert all(torch.equal(t, k) for t, k in zip((table, x, pos, out), kept))
