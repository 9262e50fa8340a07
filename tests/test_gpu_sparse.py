"""Block-sparse attention on the GPU: against the 64-bit definition, and bit
for bit against the dense entry points, other splits and other caches."""

import numpy as np
import pytest

from bitwise_aligned_causal_gb300 import inputs
from tests import sparse_plain as plain
from tests.gpu_util import to_dev
from tests.test_gpu_append import bits, caches, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def random_lists(seed, B, L, start, n, none=0.0, order=False):
    """int32 [B, 8, L, n]: per row up to n of its own blocks, in random order or ascending, -1 elsewhere; a share `none`
    of the rows lists nothing."""
    import torch

    rng = np.random.default_rng(seed)
    out = np.full((B, 8, L, n), -1, dtype=np.int32)
    for b in range(B):
        for g in range(8):
            for i in range(L):
                if rng.random() < none:
                    continue
                nb = (start + i) // 128 + 1
                m = min(n, nb, int(rng.integers(1, n + 1)))
                got = rng.choice(nb, size=m, replace=False)
                out[b, g, i, :m] = got if order else np.sort(got)
    return torch.from_numpy(out).cuda()


def all_blocks(B, L, start):
    import torch

    n = (start + L - 1) // 128 + 1
    return torch.arange(n, dtype=torch.int32, device="cuda").expand(B, 8, L, n).contiguous()


def check_rows(o, q, k, v, blocks, pos, what="", lse=None):
    """o, q [32, L, 128], k, v [8, S, 128], blocks [8, L, n], positions [L] of one sequence, all rows."""
    for g in range(8):
        h = slice(4 * g, 4 * g + 4)
        want, p, z = plain.attention(q[h], k[g], v[g], blocks[g], pos)
        mag = p @ np.abs(v[g])
        # P and the output are rounded to bf16 (2^-8 each, relative to p|v|); fp32 scores, exponentials and sums
        # stay far below 2^-10 of it for these magnitudes
        tol = (2 * 2.0 ** -8 + 2.0 ** -10) * mag
        err = np.abs(o[h] - want)
        assert np.all(err <= tol), (what, g, err.max(), tol[err > tol].min())
        if lse is not None:
            fin = np.isfinite(z)
            assert np.array_equal(np.isneginf(lse[h]), ~fin)
            # fp32 scores (|s| up to a few hundred before scaling), fp32 sum of at most 2^14 weights
            assert np.all(np.abs(lse[h][fin] - z[fin]) <= 1e-4 * np.maximum(1.0, np.abs(z[fin])))


@pytest.mark.parametrize("B,S,n,none", [(1, 1, 1, 0.0), (2, 33, 1, 0.3), (1, 128, 1, 0.0), (1, 129, 2, 0.1),
                                        (2, 500, 3, 0.05), (1, 1500, 5, 0.0), (1, 2200, 16, 0.9)])
def test_prefill_matches_the_definition(kb, B, S, n, none):
    q, k, v = randn(1000 + S, B, 32, S, 128), randn(1001 + S, B, 8, S, 128), randn(1002 + S, B, 8, S, 128)
    lists = random_lists(1003 + S, B, S, 0, n, none)
    o, lse = kb.sparse_prefill_lse(q, k, v, lists, check=True)
    for b in range(B):
        check_rows(f64(o)[b], f64(q)[b], f64(k)[b], f64(v)[b], lists[b].cpu().numpy(), np.arange(S), f"b{b}", f64(lse)[b])


@pytest.mark.parametrize("S", [1, 100, 128, 1024, 1025, 2500])
def test_every_block_listed_gives_the_dense_bits(kb, S):
    import torch

    q, k, v = randn(1100, 1, 32, S, 128), randn(1101, 1, 8, S, 128), randn(1102, 1, 8, S, 128)
    o, lse = kb.prefill_lse(q, k, v)
    so, slse = kb.sparse_prefill_lse(q, k, v, all_blocks(1, S, 0), check=True)
    assert torch.equal(bits(o), bits(so)) and torch.equal(lse, slse)
    d = kb.sparse_decode(q[:, :, S - 1:].contiguous(), k, v, S, all_blocks(1, S, 0)[:, :, S - 1:].contiguous(), check=True)
    assert torch.equal(bits(d), bits(o[:, :, S - 1:]))


def test_peaked_scores_give_the_dense_bits(kb):
    """Inputs whose reference max moves often."""
    import torch

    x = inputs.make_stress_qkv(1, 2300, seed=1200)
    q, k, v = to_dev(x.q), to_dev(x.k), to_dev(x.v)
    o = kb.prefill(q, k, v)
    assert torch.equal(bits(kb.sparse_chunk(q, k, v, 0, all_blocks(1, 2300, 0), check=True)), bits(o))
    lists = random_lists(1201, 1, 2300, 0, 6, 0.02)
    whole = kb.sparse_chunk(q, k, v, 0, lists, check=True)
    for p in (0, 127, 700, 1500, 2299):
        one = kb.sparse_decode(q[:, :, p:p + 1].contiguous(), k, v, p + 1, lists[:, :, p:p + 1].contiguous(), check=True)
        assert torch.equal(bits(one), bits(whole[:, :, p:p + 1])), p


@pytest.mark.parametrize("splits", [(1, 30, 1, 95, 1, 128, 300, 2, 642), (600, 600)])
def test_splits_give_the_same_bits(kb, splits):
    import torch

    S, n = sum(splits), 4
    q, k, v = randn(1300, 2, 32, S, 128), randn(1301, 2, 8, S, 128), randn(1302, 2, 8, S, 128)
    lists = random_lists(1303, 2, S, 0, n, 0.05)
    want = kb.sparse_chunk(q, k, v, 0, lists, check=True)
    at = 0
    for L in splits:
        rows = slice(at, at + L)
        got = kb.sparse_chunk(q[:, :, rows].contiguous(), k, v, at, lists[:, :, rows].contiguous(), check=True)
        assert torch.equal(bits(got), bits(want[:, :, rows])), (at, L)
        if L == 1:
            got = kb.sparse_decode(q[:, :, rows].contiguous(), k, v, at + 1, lists[:, :, rows].contiguous(), check=True)
            assert torch.equal(bits(got), bits(want[:, :, rows])), at
        at += L


@pytest.mark.parametrize("ctx,n,B", [(1, 1, 1), (127, 1, 1), (4097, 16, 1), (130_000, 128, 1), (130_000, 40, 2),
                                     (20_000, 16, 20), (5000, 7, 3)])
def test_one_token_equals_its_row_of_a_chunk(kb, ctx, n, B):
    """Every way the segments' partials travel: one CTA, a cluster that pushes, gathers or is read."""
    import torch

    q, k, v = randn(1400, B, 32, 1, 128), randn(1401, B, 8, ctx, 128), randn(1402, B, 8, ctx, 128)
    lists = random_lists(1403 + ctx, B, 1, ctx - 1, n)
    if n > 30:                                                   # as many blocks as the list holds
        rng = np.random.default_rng(5)
        lists = torch.from_numpy(np.stack([np.sort(rng.choice(ctx // 128, n, replace=False)) for _ in range(B * 8)])
                                 .reshape(B, 8, 1, n).astype(np.int32)).cuda()
    got = kb.sparse_decode(q, k, v, ctx, lists, check=True)
    want = kb.sparse_chunk(q, k, v, ctx - 1, lists, check=True)
    assert torch.equal(bits(got), bits(want))
    check_rows(f64(got)[0], f64(q)[0], f64(k)[0], f64(v)[0], lists[0].cpu().numpy(), [ctx - 1])


@pytest.mark.parametrize("page", [0, 128])
def test_many_tokens_with_ragged_contexts(kb, page):
    """More (sequence, KV head) units than SMs, contexts of their own, cache rows past them NaN, a row without blocks."""
    import torch

    B, cap, n = 24, 1280, 4
    k_cache, v_cache, _, table, seq = caches(B, cap, page, seed=1450)
    rng = np.random.default_rng(1451)
    ctx = rng.integers(1, cap + 1, size=B)
    ctx[:4] = (1, 128, 129, cap)
    lists = torch.cat([random_lists(1452 + b, 1, 1, int(ctx[b]) - 1, n) for b in range(B)])
    lists[5] = -1
    for b in range(B):
        for c in (k_cache, v_cache):
            if not page:
                c[b, :, ctx[b]:] = float("nan")
            else:
                for j in range(cap // page):
                    c[table[b, j], :, max(0, min(page, ctx[b] - j * page)):] = float("nan")
    q = randn(1453, B, 32, 1, 128)
    lens = torch.from_numpy(ctx.astype(np.int32)).cuda()
    if page:
        got = kb.sparse_decode_paged(q, k_cache, v_cache, table, lens, lists, check=True)
    else:
        got = kb.sparse_chunk_varlen(q, k_cache, v_cache, lens - 1, lists, check=True)
    assert bool((got[5] == 0).all())
    for b in range(B):
        kc, vc = (seq(x, b)[:, :ctx[b]].contiguous()[None] for x in (k_cache, v_cache))
        want = kb.sparse_decode(q[b:b + 1], kc, vc, int(ctx[b]), lists[b:b + 1], check=True)
        assert torch.equal(bits(got[b:b + 1]), bits(want)), b


@pytest.mark.parametrize("L", [1, 70])
def test_order_repeats_and_later_blocks_change_nothing(kb, L):
    import torch

    start, cap = 1500, 2500
    q, k, v = randn(1500, 1, 32, L, 128), randn(1501, 1, 8, cap, 128), randn(1502, 1, 8, cap, 128)
    lists = random_lists(1503, 1, L, start, 6, 0.1)
    want = kb.sparse_chunk(q, k, v, start, lists, check=True)
    more = torch.cat([lists.flip(-1), torch.full_like(lists[..., :2], 19), lists[..., 1:4]], -1).contiguous()
    assert torch.equal(bits(kb.sparse_chunk(q, k, v, start, more, check=True)), bits(want))
    if L == 1:
        for some in (lists, more):
            assert torch.equal(bits(kb.sparse_decode(q, k, v, start + 1, some, check=True)), bits(want))


def test_rows_that_list_nothing_are_zero(kb):
    import torch

    S = 300
    q, k, v = randn(1600, 1, 32, S, 128), randn(1601, 1, 8, S, 128), randn(1602, 1, 8, S, 128)
    lists = torch.full((1, 8, S, 3), -1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    o, lse = kb.sparse_prefill_lse(q, k, v, lists, out=out, check=True)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    out = torch.full_like(q[:, :, :1], 9.0)
    for ctx in (1, 200, S):
        d = kb.sparse_decode(q[:, :, :1].contiguous(), k, v, ctx, lists[:, :, :1].contiguous(), out=out, check=True)
        assert bool((d == 0).all())
    # later blocks only: nothing visible
    lists[..., 0] = 2
    o, lse = kb.sparse_prefill_lse(q, k, v, lists, check=True)
    assert bool((o[:, :, :256] == 0).all()) and not bool((o[:, :, 256:] == 0).all())


@pytest.mark.parametrize("page", [0, 128, 512])
@pytest.mark.parametrize("L", [1, 45, 200])
def test_ragged_and_paged_equal_each_sequence_alone(kb, page, L):
    import torch

    B, cap, n = 4, 2048, 5
    k_cache, v_cache, _, table, seq = caches(B, cap, page, seed=1700)
    starts = np.array([0, 1000, 1777, 333])
    lens = np.array([L, L, max(1, L - 7), 0])
    for b in range(B):                                            # rows past each sequence hold anything
        if page:
            continue
        k_cache[b, :, starts[b] + lens[b]:] = float("nan")
        v_cache[b, :, starts[b] + lens[b]:] = float("nan")
    q = randn(1701, B, 32, L, 128)
    lists = torch.cat([random_lists(1702 + b, 1, L, int(starts[b]), n, 0.05) for b in range(B)])
    st, ln = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (starts, lens))
    out = torch.full_like(q, 3.0)
    kb.sparse_chunk_varlen(q, k_cache, v_cache, st, lists, lens=ln, block_table=table, out=out, check=True)
    for b in range(B):
        m, s = int(lens[b]), int(starts[b])
        assert bool((out[b, :, m:] == 3.0).all())
        if not m:
            continue
        kc, vc = (seq(x, b).contiguous()[None] for x in (k_cache, v_cache))
        want = kb.sparse_chunk(q[b:b + 1, :, :m].contiguous(), kc, vc, s, lists[b:b + 1, :, :m].contiguous(), check=True)
        assert torch.equal(bits(out[b:b + 1, :, :m]), bits(want))
    if page and L == 1:
        got = kb.sparse_decode_paged(q, k_cache, v_cache, table, st + 1, lists, check=True)
        for b in range(B):
            kc, vc = (seq(x, b).contiguous()[None] for x in (k_cache, v_cache))
            want = kb.sparse_chunk(q[b:b + 1], kc, vc, int(starts[b]), lists[b:b + 1], check=True)
            assert torch.equal(bits(got[b:b + 1]), bits(want))


def test_bad_device_arguments_are_recorded(kb):
    import torch

    q, k, v = randn(1800, 2, 32, 1, 128), randn(1801, 9, 8, 256, 128), randn(1802, 9, 8, 256, 128)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lists = torch.tensor([0, 3], dtype=torch.int32, device="cuda").expand(2, 8, 1, 2).contiguous()
    ctx = torch.tensor([500, 1024], dtype=torch.int32, device="cuda")
    kb.sparse_decode_paged(q, k, v, table, ctx, lists, check=True)
    kb.sparse_chunk_varlen(q, k, v, ctx - 1, lists, block_table=table, check=True)

    def both(table, ctx, lists):
        out = torch.full_like(q, 4.0)
        kb.sparse_decode_paged(q, k, v, table, ctx, lists, out=out)
        with pytest.raises(kb.KBError):
            kb.check_device_status()
        kb.sparse_chunk_varlen(q, k, v, ctx - 1, lists, block_table=table)
        with pytest.raises(kb.KBError):
            kb.check_device_status()
        return out

    for wrong in (8, -2, 1 << 30):                                # blocks
        bad = lists.clone()
        bad[1, 2, 0, 1] = wrong
        both(table, ctx, bad)
    for wrong in (9, -1):                                         # pages
        bad = table.clone()
        bad[0, 1] = wrong
        both(bad, ctx, lists)
    for wrong in (0, 1025):                                       # contexts
        bad = ctx.clone()
        bad[1] = wrong
        assert bool((both(table, bad, lists)[1] == 4.0).all())


def test_two_streams_and_a_replayed_graph(kb):
    import torch

    S, n = 700, 3
    q, k, v = randn(1900, 1, 32, S, 128), randn(1901, 1, 8, S, 128), randn(1902, 1, 8, S, 128)
    lists = random_lists(1903, 1, S, 0, n)
    want = kb.sparse_chunk(q, k, v, 0, lists, check=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [kb.sparse_chunk(q, k, v, 0, lists, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(bits(o), bits(want)) for o in outs)
    ws = torch.empty(kb.kb_attn_sparse_workspace_bytes(1, 8, S, n, S), dtype=torch.uint8, device="cuda")
    out, changing = torch.empty_like(q), lists.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kb.sparse_chunk(q, k, v, 0, changing, out=out, workspace=ws)
    for seed in (0, 1):
        changing.copy_(random_lists(1904 + seed, 1, S, 0, n, 0.1))
        graph.replay()
        assert torch.equal(bits(out), bits(kb.sparse_chunk(q, k, v, 0, changing, check=True)))
    with pytest.raises(kb.KBError):
        kb.sparse_chunk(q, k, v, 0, lists, workspace=ws[:-512])


@pytest.mark.parametrize("page", [128, 256])
def test_serving_run_equals_the_training_forward(kb, page):
    """The operators together: a prompt in two chunks and then token by token through append, selection and sparse
    attention over a paged cache gives the rows of the whole sequence's rotation, boxes, selection and training forward,
    bit for bit."""
    import torch

    S, n, cap = 1000, 4, 1024
    q, k, v = randn(2000, 1, 32, S, 128), randn(2001, 1, 8, S, 128), randn(2002, 1, 8, S, 128)
    rope = kb.rope_table(cap)
    tq, tk = kb.rope(q, rope), kb.rope(k, rope)
    boxes = kb.block_boxes(tk)
    lists = kb.select_blocks(tq, boxes, 0, n)
    # a whole sequence's boxes hold later keys of a row's own block, which is always taken: the choice is the same
    want, _ = kb.sparse_prefill_lse(tq, tk, v, lists, check=True)
    k_cache, v_cache, bx, table, _ = caches(1, cap, page, seed=2003)
    at = 0
    for L in (700, 290) + (1,) * 10:
        st = torch.tensor([at], dtype=torch.int32, device="cuda")
        cut = slice(at, at + L)
        rows = kb.append_varlen(q[:, :, cut], k[:, :, cut], v[:, :, cut], k_cache, v_cache, rope, st, block_table=table,
                                boxes=bx)
        chosen = kb.select_blocks_varlen(rows, bx, st, n, block_table=table)
        assert torch.equal(chosen, lists[:, :, cut])
        if L == 1:
            got = kb.sparse_decode_paged(rows, k_cache, v_cache, table, st + 1, chosen)
        else:
            got = kb.sparse_chunk_varlen(rows, k_cache, v_cache, st, chosen, block_table=table)
        kb.check_device_status()
        assert torch.equal(bits(got), bits(want[:, :, cut])), at
        at += L


@pytest.mark.parametrize("S", [4860, 4864])
def test_ctas_that_go_from_unit_to_unit(kb, S):
    """8 KV heads x 152 position tiles are a whole number of units for every SM of this GPU, so a CTA takes several; cut
    into chunks of 500 rows, one each.  Same bits, with rows and whole units that list nothing among them."""
    import torch

    q, k, v = randn(150, 1, 32, S, 128), randn(151, 1, 8, S, 128), randn(152, 1, 8, S, 128)
    blocks = random_lists(153, 1, S, 0, 3, none=0.2)
    blocks[:, :, 640:800] = -1
    o, lse = kb.sparse_prefill_lse(q, k, v, blocks, check=True)
    for a in range(0, S, 500):
        z = min(a + 500, S)
        part = kb.sparse_chunk(q[:, :, a:z].contiguous(), k, v, a, blocks[:, :, a:z].contiguous(), check=True)
        assert torch.equal(bits(part), bits(o[:, :, a:z]))
    empty = (blocks < 0).all(-1).repeat_interleave(4, 1)
    assert torch.equal(torch.isneginf(lse), empty) and not o[empty].any()
