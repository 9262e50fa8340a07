"""Block selection on the GPU: the chosen blocks equal the definition's, whole
number for whole number, at every split, cache and size."""

import numpy as np
import pytest

from tests import sparse_plain as plain
from tests.test_gpu_append import caches, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def check_rows(got, q, bx, pos, n, rows, **keep):
    """got [8, L, n], q [32, L, 128], bx [8, blocks, 2, 128], pos [L]; the rows listed."""
    for g in range(8):
        for i in rows:
            want = plain.choose(q[4 * g:4 * g + 4, i], bx[g], int(pos[i]), n, **keep)
            assert np.array_equal(got[g, i], want), (g, i, got[g, i], want)


@pytest.mark.parametrize("ctx,n,keep", [(1, 1, {"keep_first": 0}), (128, 2, {}), (129, 2, {}), (700, 3, {}), (2000, 16, {}),
                                        (5000, 5, {"keep_first": 2, "keep_last": 3}), (5000, 2, {"keep_first": 0}),
                                        (40_000, 24, {}), (140_001, 16, {}), (140_001, 128, {"keep_first": 0})])
def test_one_token(kb, ctx, n, keep):
    B = 2
    k = randn(100 + ctx, B, 8, ctx, 128)
    bx = kb.block_boxes(k)
    q = randn(101 + ctx, B, 32, 1, 128)
    got = kb.select_blocks(q, bx, ctx - 1, n, check=True, **keep).cpu().numpy()
    for b in range(B):
        check_rows(got[b], f64(q)[b], f64(bx)[b], [ctx - 1], n, [0], **keep)


@pytest.mark.parametrize("start,L,n", [(0, 1000, 4), (1000, 333, 6), (127, 2, 1), (3000, 17, 24), (0, 4000, 16)])
def test_chunk_rows_equal_one_token_calls(kb, start, L, n):
    import torch

    S = start + L
    k = randn(200 + S, 1, 8, S, 128)
    bx = kb.block_boxes(k)
    q = randn(201 + S, 1, 32, L, 128)
    keep = {"keep_first": 1 if n > 1 else 0}
    got = kb.select_blocks(q, bx, start, n, check=True, **keep)
    rows = sorted(set([0, L - 1, L // 2, L // 3, min(L - 1, 128), min(L - 1, 129)]))
    check_rows(got[0].cpu().numpy(), f64(q)[0], f64(bx)[0], np.arange(start, S), n, rows, **keep)
    for i in rows:
        one = kb.select_blocks(q[:, :, i:i + 1].contiguous(), bx, start + i, n, **keep)
        assert torch.equal(one[:, :, 0], got[:, :, i])


@pytest.mark.parametrize("start,L,n,keep", [(39_000, 300, 16, {}), (39_000, 40, 40, {}), (20_000, 200, 128, {"keep_first": 0}),
                                            (3000, 200, 2, {}), (70_000, 129, 34, {}), (33_000, 17, 5, {"keep_last": 4}),
                                            (32_760, 30, 12, {"keep_first": 9})])
def test_long_chunks_over_many_blocks(kb, start, L, n, keep):
    """Around 256 blocks the scores of a chunk's rows take more than one pass."""
    import torch

    S = start + L
    bx = kb.block_boxes(randn(250 + S, 1, 8, S, 128))
    q = randn(251 + S, 1, 32, L, 128)
    got = kb.select_blocks(q, bx, start, n, check=True, **keep)
    rows = [0, L // 2, L - 1]
    check_rows(got[0].cpu().numpy(), f64(q)[0], f64(bx)[0], np.arange(start, S), n, rows, **keep)
    for i in range(0, L, 7):
        one = kb.select_blocks(q[:, :, i:i + 1].contiguous(), bx, start + i, n, **keep)
        assert torch.equal(one[:, :, 0], got[:, :, i])


def test_ties_over_several_passes(kb):
    import torch

    bx = torch.ones(1, 8, 700, 2, 128, dtype=torch.bfloat16, device="cuda")
    bx[:, :, 300] = 2.0
    bx[:, :, 650] = 2.0
    q = torch.ones(1, 32, 100, 128, dtype=torch.bfloat16, device="cuda")
    got = kb.select_blocks(q, bx, 699 * 128, 8, check=True)
    want = torch.tensor([0, 1, 2, 3, 4, 300, 650, 699], dtype=torch.int32)
    assert bool((got.cpu() == want).all())


def test_ties_go_to_the_lowest_block(kb):
    import torch

    bx = torch.ones(1, 8, 60, 2, 128, dtype=torch.bfloat16, device="cuda")
    bx[:, :, 40:45] = 2.0
    q = torch.ones(1, 32, 200, 128, dtype=torch.bfloat16, device="cuda")
    got = kb.select_blocks(q, bx, 59 * 128 - 100, 9, check=True)
    assert torch.equal(got[0, 0, 150].cpu(), torch.tensor([0, 1, 2, 40, 41, 42, 43, 44, 59], dtype=torch.int32))
    assert torch.equal(got[0, 5, 0].cpu(), torch.tensor([0, 1, 2, 40, 41, 42, 43, 44, 58], dtype=torch.int32))
    q.zero_()                                                    # every score is zero
    got = kb.select_blocks(q, bx, 59 * 128 - 100, 4, check=True)
    assert torch.equal(got[0, 3, 150].cpu(), torch.tensor([0, 1, 2, 59], dtype=torch.int32))


def test_scores_near_each_other(kb):
    """Boxes that differ by one step in one channel, queries of very different magnitudes."""
    import torch

    bx = torch.zeros(1, 8, 300, 2, 128, dtype=torch.bfloat16, device="cuda")
    bx[0, :, :, 0] = 64.0 / 64
    bx[0, :, :, 1] = -64.0 / 64
    for j in range(300):
        bx[0, :, j, 0, j % 128] += ((j * 7) % 3) / 64.0
    q = randn(300, 1, 32, 130, 128) * torch.logspace(-6, 6, 130, device="cuda").to(torch.bfloat16)[None, None, :, None]
    got = kb.select_blocks(q, bx, 299 * 128 - 60, 20, check=True)
    check_rows(got[0].cpu().numpy(), f64(q)[0], f64(bx)[0], np.arange(130) + 299 * 128 - 60, 20, [0, 59, 60, 129])


@pytest.mark.parametrize("page", [128, 512])
@pytest.mark.parametrize("L", [1, 40, 300])
def test_paged_and_ragged(kb, page, L):
    import torch

    B, cap, n = 3, 4096, 6
    k_cache, v_cache, bx, table, seq = caches(B, cap, page, seed=400)
    kb.block_boxes(k_cache, block_table=table, boxes=bx, check=True)
    starts = torch.tensor([0, 3777, 1500], dtype=torch.int32, device="cuda")
    lens = torch.tensor([L, L if L == 1 else L - 1, 0], dtype=torch.int32, device="cuda")
    q = randn(401, B, 32, L, 128)
    out = torch.full((B, 8, L, n), -7, dtype=torch.int32, device="cuda")
    kb.select_blocks_varlen(q, bx, starts, n, lens=lens, block_table=table, out=out, check=True)
    for b in range(B):
        m, s = int(lens[b]), int(starts[b])
        assert bool((out[b, :, m:] == -7).all())
        if m:
            flat = seq(bx, b).contiguous()
            want = kb.select_blocks(q[b:b + 1, :, :m].contiguous(), flat[None], s, n)
            assert torch.equal(out[b, :, :m], want[0])
            check_rows(out[b].cpu().numpy(), f64(q)[b], f64(flat), np.arange(s, s + L), n, [0, m - 1])


def test_bad_device_arguments(kb):
    import torch

    bx = torch.ones(4, 8, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = randn(500, 1, 32, 2, 128)
    for table, start, length in (([0, 4], 500, 2), ([0, 1], 511, 2), ([0, 1], -1, 2), ([0, 1], 5, 3)):
        out = torch.full((1, 8, 2, 1), -7, dtype=torch.int32, device="cuda")
        kb.select_blocks_varlen(q, bx, torch.tensor([start], dtype=torch.int32, device="cuda"), 1, keep_first=0,
                                lens=torch.tensor([length], dtype=torch.int32, device="cuda"),
                                block_table=torch.tensor([table], dtype=torch.int32, device="cuda"), out=out)
        with pytest.raises(kb.KBError):
            kb.check_device_status()
        if table[1] != 4:
            assert bool((out == -7).all())
    out = kb.select_blocks_varlen(q, bx, torch.tensor([500], dtype=torch.int32, device="cuda"), 3,
                                  block_table=torch.tensor([[0, 4]], dtype=torch.int32, device="cuda"))
    with pytest.raises(kb.KBError):
        kb.check_device_status()
    kb.check_device_status()


@pytest.mark.parametrize("L", [1, 200])
def test_on_two_streams_and_replayed(kb, L):
    """Two calls at once have their own lists, and a captured one reads what its tensors hold at the replay."""
    import torch

    start, n = 2000, 5
    q = [randn(670 + i, 1, 32, L, 128) for i in range(3)]
    bx = kb.block_boxes(randn(675, 1, 8, start + L, 128), check=True)
    want = [kb.select_blocks(x, bx, start, n, check=True) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = [kb.select_blocks(x, bx, start, n, stream=s) for _ in range(4) for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    kb.check_device_status()
    assert all(torch.equal(x, want[i % 3]) for i, x in enumerate(got))
    held, out = q[0].clone(), torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kb.select_blocks(held, bx, start, n, out=out)
    for x, y in zip(q, want):
        held.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
