"""Log-sum-exps of chunks and tokens, and the attention weight that each cached
key gets, against their 64-bit definitions."""

import numpy as np
import pytest

from tests import cache_plain as plain
from tests.test_gpu_append import bits, caches, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(*x):
    import torch

    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,S,L", [(1, 1, 1), (2, 128, 1), (1, 1300, 1), (2, 1300, 2), (1, 1300, 20), (1, 700, 33), (1, 1300, 1300),
                                   (1, 20000, 1), (20, 300, 1)])
def test_chunk_lse_has_the_bits_of_the_whole_sequence(kb, B, S, L):
    import torch

    q, k, v = randn(1, B, 32, S, 128), randn(2, B, 8, S, 128), randn(3, B, 8, S, 128)
    o, lse = kb.prefill_lse(q, k, v, check=True)
    part = q[:, :, S - L:].contiguous()
    got, got_lse = kb.chunk_lse(part, k, v, S - L, check=True)
    assert torch.equal(bits(got), bits(o[:, :, S - L:])) and torch.equal(got_lse, lse[:, :, S - L:])
    assert torch.equal(bits(got), bits(kb.chunk(part, k, v, S - L, check=True)))
    st = torch.full((B,), S - L, dtype=torch.int32, device="cuda")
    vo, vlse = kb.chunk_lse_varlen(part, k, v, st, torch.full_like(st, L), check=True)
    assert torch.equal(bits(vo), bits(got)) and torch.equal(vlse, got_lse)


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("L", [1, 6, 40])
def test_chunk_lse_paged_and_ragged(kb, page, L):
    import torch

    B, cap = 3, 1024
    k, v, _, pages, seq = caches(B, cap, page, seed=10)
    q = randn(11, B, 32, L, 128)
    starts, lens = (0, 1000 - L, 500), (L, max(L - 2, 1), 0)
    out, lse = torch.full_like(q, 7.0), torch.full((B, 32, L), 9.0, device="cuda")
    kb.chunk_lse_varlen(q, k, v, i32(*starts), i32(*lens), block_table=pages, out=out, lse=lse, check=True)
    for b in range(B):
        n = lens[b]
        assert bool((out[b, :, n:] == 7.0).all()) and bool((lse[b, :, n:] == 9.0).all())
        if n:
            o1, l1 = kb.chunk_lse(q[b:b + 1, :, :n].contiguous(), seq(k, b)[None].contiguous(), seq(v, b)[None].contiguous(), starts[b], check=True)
            assert torch.equal(bits(out[b, :, :n]), bits(o1[0])) and torch.equal(lse[b, :, :n], l1[0])


def check_weights(got, before, q, k, lse, starts, lens):
    """got, before [B,8,cap] float32; q [B,32,L,128], lse [B,32,L]; k: sequence b's keys [8, cap, 128]."""
    for b in range(q.shape[0]):
        n = lens[b]
        end = starts[b] + n if n else 0
        assert np.array_equal(got[b, :, end:], before[b, :, end:])
        for g in range(8):
            if not n:
                continue
            heads = slice(4 * g, 4 * g + 4)
            w, tol = plain.key_weights(q[b, heads, :n], k(b)[g, :end], lse[b, heads, :n], np.arange(starts[b], end))
            want = before[b, g, :end].astype(np.float64) + w
            assert np.all(np.abs(got[b, g, :end] - want) <= tol + 2.0 ** -24 * np.abs(want) + 1e-37), (b, g)


@pytest.mark.parametrize("B,L,start", [(1, 1, 0), (2, 1, 127), (1, 1, 128), (3, 1, 1500), (1, 2, 127), (2, 5, 600), (1, 32, 0),
                                       (1, 31, 2000), (1, 33, 0), (2, 100, 29), (1, 128, 128), (1, 257, 300), (1, 700, 0), (1, 129, 1)])
def test_weights_match_the_definition(kb, B, L, start):
    import torch

    cap = start + L + 7
    q, k, v = randn(20, B, 32, L, 128), randn(21, B, 8, cap, 128), randn(22, B, 8, cap, 128)
    k[:, :, start + L:] = float("nan")                           # rows that no call wrote
    v[:, :, start + L:] = float("nan")
    _, lse = kb.chunk_lse(q, k, v, start, check=True)
    w = torch.rand(B, 8, cap, device="cuda")
    before = w.cpu().numpy()
    assert kb.key_weights(q, k, lse, w, start, check=True) is w
    check_weights(w.cpu().numpy(), before, f64(q), lambda b: f64(k[b]), lse.double().cpu().numpy(), [start] * B, [L] * B)
    # every row gives the group's four heads' worth, and nothing else comes in
    got = (w.double() - torch.from_numpy(before).cuda().double()).sum(-1)
    assert torch.all((got - 4 * L).abs() <= 2.0 ** -24 * cap + 4 * L * 2.0 ** -12)
    # again on the same numbers: the same bits
    again = torch.from_numpy(before).cuda()
    kb.key_weights(q, k, lse, again, start, check=True)
    assert torch.equal(again, w)


@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("L,starts,lens", [(1, (0, 900, 40), (1, 1, 0)), (9, (120, 0, 700), (9, 4, 0)), (30, (100, 0, 994), (30, 1, 30)),
                                           (300, (0, 100, 724), (300, 0, 131))])
def test_ragged_and_paged(kb, page, L, starts, lens):
    import torch

    B, cap = 3, 1024
    k, v, _, pages, seq = caches(B, cap, page, seed=30)
    q = randn(31, B, 32, L, 128)
    for b in range(B):
        q[b, :, lens[b]:] = float("nan")                          # rows of no sequence
    lse = torch.full((B, 32, L), float("nan"), device="cuda")
    kb.chunk_lse_varlen(q, k, v, i32(*starts), i32(*lens), block_table=pages, lse=lse, check=True)
    w = torch.rand(B, 8, cap, device="cuda")
    before = w.cpu().numpy()
    kb.key_weights_varlen(q, k, lse, w, i32(*starts), i32(*lens), block_table=pages, check=True)
    check_weights(w.cpu().numpy(), before, f64(q), lambda b: f64(seq(k, b)), lse.double().cpu().numpy(), starts, lens)


@pytest.mark.parametrize("L", [3, 40])
def test_rows_that_saw_nothing_and_strong_rows(kb, L):
    """An lse of -inf gives no weight; a sink key takes all of a row's weight; garbage lse (NaN) shows."""
    import torch

    S = 400
    q, k, v = randn(40, 1, 32, L, 128), randn(41, 1, 8, S, 128), randn(42, 1, 8, S, 128)
    k[:, :, 0] = q.view(1, 8, 4, L, 128)[:, :, 0, 0] * 30
    _, lse = kb.chunk_lse(q, k, v, S - L, check=True)
    lse[0, 5, 1] = float("-inf")
    lse[0, 6, :] = float("inf")
    w = torch.zeros(1, 8, S, device="cuda")
    kb.key_weights(q, k, lse, w, S - L, check=True)
    l64 = lse.double().cpu().numpy()
    check_weights(w.cpu().numpy(), np.zeros((1, 8, S), np.float32), f64(q), lambda b: f64(k[b]), l64, [S - L], [L])
    lse[0, 9, 0] = float("nan")
    kb.key_weights(q, k, lse, w, S - L, check=True)
    assert bool(torch.isnan(w[0, 2, :S - L]).all()) and bool(torch.isfinite(w[0, 3]).all())


def test_bad_device_arguments_are_reported(kb):
    import torch

    B, cap, L = 2, 512, 5
    k, v, _, pages, _ = caches(B, cap, 128, seed=50)
    q, lse = randn(51, B, 32, L, 128), torch.zeros(B, 32, L, device="cuda")
    w = torch.zeros(B, 8, cap, device="cuda")
    for st, ln in ((i32(-1, 0), i32(1, 1)), (i32(508, 0), i32(5, 1)), (i32(0, 0), i32(6, 1)), (i32(0, 0), i32(1, -1))):
        with pytest.raises(kb.KBError):
            kb.key_weights_varlen(q, k, lse, w, st, ln, block_table=pages, check=True)
    for bad in (-1, 10, 2 ** 31 - 1):
        broken = pages.clone()
        broken[0, 1] = bad
        w.zero_()
        with pytest.raises(kb.KBError):
            kb.key_weights_varlen(q, k, lse, w, i32(300, 300), i32(5, 5), block_table=broken, check=True)
        assert bool((w[0, :, 128:256] == 0).all())


def test_refusals(kb):
    import torch

    q, k = randn(60, 1, 32, 5, 128), randn(61, 1, 8, 50, 128)
    lse, w = torch.zeros(1, 32, 5, device="cuda"), torch.zeros(1, 8, 50, device="cuda")
    for args in ((q, k, lse.double(), w, 0), (q, k, lse, w.half(), 0), (q.float(), k, lse, w, 0), (q, k, lse, w.cpu(), 0)):
        with pytest.raises(TypeError):
            kb.key_weights(*args)
    for args in ((q, k, lse[:, :, :4].contiguous(), w, 0), (q, k, lse, w, 46), (q, k, lse, w, -1), (q, k, lse, w[:, :, :49].contiguous(), 0)):
        with pytest.raises(ValueError):
            kb.key_weights(*args)
    with pytest.raises(TypeError):
        kb.key_weights_varlen(q, k, lse, w, i32(0), None)
    with pytest.raises(TypeError):
        kb.chunk_lse_varlen(q, k, k, None, i32(5))


def test_captured_and_on_two_streams(kb):
    import torch

    S, L = 900, 300
    q, k, v = randn(70, 1, 32, L, 128), randn(71, 1, 8, S, 128), randn(72, 1, 8, S, 128)
    _, lse = kb.chunk_lse(q, k, v, S - L, check=True)
    want = torch.zeros(1, 8, S, device="cuda")
    kb.key_weights(q, k, lse, want, S - L, check=True)
    got = [torch.zeros(1, 8, S, device="cuda") for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, w in zip(streams, got):
        st.wait_stream(torch.cuda.current_stream())
        kb.key_weights(q, k, lse, w, S - L, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kb.key_weights(q, k, lse, got[2], S - L)
    g.replay()
    torch.cuda.synchronize()
    kb.check_device_status()
    for w in got:
        assert torch.equal(w, want)


def test_far_rows(kb):
    """A cache and queries beyond 2^31 elements: the last rows' weights."""
    import torch

    cap, L = 2_200_000, 3
    k = torch.zeros(1, 8, cap, 128, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 31
    k[:, :, -70:] = randn(80, 1, 8, 70, 128)
    q = randn(81, 1, 32, L, 128)
    _, lse = kb.chunk_lse(q, k, k, cap - L, check=True)
    w = torch.zeros(1, 8, cap, device="cuda")
    kb.key_weights(q, k, lse, w, cap - L, check=True)
    l64 = lse.double().cpu().numpy()
    for g in (0, 7):
        want, tol = plain.key_weights(f64(q)[0, 4 * g:4 * g + 4], f64(k[0, g, -100:]), l64[0, 4 * g:4 * g + 4], np.arange(100 - L, 100))
        assert np.all(np.abs(w[0, g, -100:].cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("L", [1, 3, 20, 33, 130])
def test_infinite_keys_that_weigh_nothing(kb, L):
    """A key of -inf scores adds exactly nothing, and the others' weights keep their bits, however many rows there are."""
    import torch

    S, j = 700, 301
    q, k = randn(90, 1, 32, L, 128), randn(91, 1, 8, S, 128)
    q[..., 5] = -q[..., 5].abs() - 1
    lse = torch.full((1, 32, L), 5.0, device="cuda")
    want = torch.rand(1, 8, S, device="cuda")
    got, before = want.clone(), want.clone()
    kb.key_weights(q, k, lse, want, S - L, check=True)
    k[:, :, j, 5] = float("inf")
    kb.key_weights(q, k, lse, got, S - L, check=True)
    assert torch.equal(got[:, :, j], before[:, :, j])
    got[:, :, j] = want[:, :, j]
    assert torch.equal(got, want)
