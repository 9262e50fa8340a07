"""Gradient of block-sparse attention on the GPU: against the 64-bit formulas,
against differences, and bit for bit across calls."""

import numpy as np
import pytest

from tests import sparse_plain as plain
from tests.test_gpu_append import bits, f64, kb, randn  # noqa: F401
from tests.test_gpu_sparse import all_blocks, random_lists

pytestmark = pytest.mark.gpu

U = 2.0 ** -8                      # half a bf16 step, relative to the value


def tolerances(q, k, v, dout, blocks):
    """Elementwise bounds on the kernels' roundings for one KV head: P, dS and the outputs rounded to bf16, delta from
    the rounded output, the fp32 steps together below 2^-11 of the magnitudes."""
    n = q.shape[1]
    o, p, _ = plain.attention(q, k, v, blocks, np.arange(n))
    mag_o = p @ np.abs(v)
    # |dP - delta| and the error of delta (o is off by 2U of p|v|: P's and its own rounding)
    dp = dout @ v.T
    d_delta = (np.abs(dout) * (2 * U + 2.0 ** -10) * mag_o).sum(-1, keepdims=True)
    ds = p * np.abs(dp - (dout * o).sum(-1, keepdims=True))
    fp32 = 2.0 ** -11 * p * (np.abs(dout) @ np.abs(v).T)
    e_ds = U * ds + p * d_delta + fp32
    e_p = (U + 2.0 ** -11) * p
    s = 1 / np.sqrt(128.0)
    t = 1.25                       # products of two of these roundings
    return (t * (e_ds + U * ds) @ np.abs(k) * s,
            t * np.einsum("grs,grd->sd", e_ds + U * ds, np.abs(q)) * s,
            t * np.einsum("grs,grd->sd", e_p + U * p, np.abs(dout)))


@pytest.mark.parametrize("B,S,n,none", [(1, 1, 1, 0.0), (1, 31, 1, 0.0), (2, 130, 1, 0.2), (1, 129, 2, 0.0),
                                        (1, 700, 3, 0.05), (2, 300, 2, 0.95), (1, 1300, 5, 0.0)])
def test_matches_the_definition(kb, B, S, n, none):
    q, k, v = randn(3000 + S, B, 32, S, 128), randn(3001 + S, B, 8, S, 128), randn(3002 + S, B, 8, S, 128)
    dout = randn(3003 + S, B, 32, S, 128)
    lists = random_lists(3004 + S, B, S, 0, n, none)
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    got = [f64(x) for x in kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)]
    q, k, v, dout, lists = f64(q), f64(k), f64(v), f64(dout), lists.cpu().numpy()
    for b in range(B):
        for g in range(8):
            h = slice(4 * g, 4 * g + 4)
            args = q[b, h], k[b, g], v[b, g], dout[b, h], lists[b, g]
            want, tol = plain.gradients(*args), tolerances(*args)
            for name, x, y, t in zip(("dq", "dk", "dv"), (got[0][b, h], got[1][b, g], got[2][b, g]), want, tol):
                err = np.abs(x - y)
                assert np.all(err <= t + 1e-7), (name, b, g, err.max(), (err - t).max())


@pytest.mark.parametrize("S", [100, 128, 1025])
def test_every_block_listed_is_the_dense_gradient(kb, S):
    """The same formula with the sums taken in units of 32 positions: equal up to the roundings of both."""
    q, k, v, dout = (randn(3100 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    o, lse = kb.prefill_lse(q, k, v)
    dense = kb.backward(q, k, v, o, dout, lse, check=True)
    lists = all_blocks(1, S, 0)
    sparse = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)
    import torch

    assert torch.equal(sparse[3], dense[3])
    for g in range(8):
        h = slice(4 * g, 4 * g + 4)
        tol = tolerances(f64(q)[0, h], f64(k)[0, g], f64(v)[0, g], f64(dout)[0, h], lists[0, g].cpu().numpy())
        for i, (x, y) in enumerate(((sparse[0][0, h], dense[0][0, h]), (sparse[1][0, g], dense[1][0, g]),
                                    (sparse[2][0, g], dense[2][0, g]))):
            assert np.all(np.abs(f64(x) - f64(y)) <= 2 * tol[i] + 1e-7)


def test_against_differences(kb):
    """The directional derivative of sum(dout * o) from the gradients against a central difference of the definition."""
    S, n, h = 300, 2, 1e-4
    q, k, v, dout = (randn(3200 + i, 1, heads, S, 128) for i, heads in enumerate((32, 8, 8, 32)))
    lists = random_lists(3204, 1, S, 0, n, 0.1)
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    grads = [f64(x)[0] for x in kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)[:3]]
    q, k, v, dout = (f64(x)[0] for x in (q, k, v, dout))
    rng = np.random.default_rng(1)
    d = [rng.standard_normal(x.shape) for x in (q, k, v)]

    def loss(t, g):
        r = slice(4 * g, 4 * g + 4)
        o = plain.attention(q[r] + t * d[0][r], k[g] + t * d[1][g], v[g] + t * d[2][g], lists[0, g].cpu().numpy(),
                            np.arange(S))[0]
        return (dout[r] * o).sum()

    for g in range(8):
        r = slice(4 * g, 4 * g + 4)
        diff = (loss(h, g) - loss(-h, g)) / (2 * h)
        slopes = (grads[0][r] * d[0][r]).sum() + (grads[1][g] * d[1][g]).sum() + (grads[2][g] * d[2][g]).sum()
        tol = tolerances(q[r], k[g], v[g], dout[r], lists[0, g].cpu().numpy())
        bound = (tol[0] * np.abs(d[0][r])).sum() + (tol[1] * np.abs(d[1][g])).sum() + (tol[2] * np.abs(d[2][g])).sum()
        assert abs(slopes - diff) <= bound + 1e-3, (slopes, diff, bound)


def test_unlisted_blocks_and_rows_have_zero_gradients(kb):
    import torch

    S = 520
    q, k, v, dout = (randn(3300 + i, 2, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = torch.full((2, 8, S, 2), -1, dtype=torch.int32, device="cuda")
    lists[0, :, 200:] = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    outs = [torch.full_like(x, 7.0) for x in (q, k, v)]
    dq, dk, dv, _ = kb.sparse_backward(q, k, v, o, dout, lse, lists, dq=outs[0], dk=outs[1], dv=outs[2], check=True)
    assert bool((dq[:, :, :200] == 0).all()) and bool((dq[1] == 0).all()) and not bool((dq[0, :, 200:] == 0).all())
    for x in (dk, dv):
        assert bool((x[1] == 0).all()) and bool((x[0, :, 128:384] == 0).all()) and bool((x[0, :, 512:] == 0).all())
        assert not bool((x[0, :, :128] == 0).all()) and not bool((x[0, :, 384:512] == 0).all())
    assert all(bool(torch.isfinite(x).all()) for x in (dq, dk, dv))


def test_repeats_order_and_streams_give_the_same_bits(kb):
    import torch

    S, n = 900, 4
    q, k, v, dout = (randn(3400 + i, 2, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = random_lists(3404, 2, S, 0, n, 0.05)
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    want = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)
    other = torch.cat([lists.flip(-1), lists[..., :2]], -1).contiguous()
    torch.cuda.synchronize()
    runs = [kb.sparse_backward(q, k, v, o, dout, lse, l, stream=s) for l in (lists, other)
            for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    kb.check_device_status()
    for run in runs:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(run, want))
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(kb.kb_attn_sparse_backward_workspace_bytes(2, 8, S, n), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x) for x in want]
    with torch.cuda.graph(graph):
        kb.sparse_backward(q, k, v, o, dout, lse, lists, delta=outs[3], dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))


def test_long_blocks_shared_by_two_ctas(kb):
    """Rows enough for a block's gradient to be summed in two halves: every row keeps the first block, and the batch and the
    lists' width change no bit."""
    import torch

    S, n = 4500, 3
    q, k, v, dout = (randn(3700 + i, 2, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = random_lists(3704, 1, S, 0, n).repeat(2, 1, 1, 1)
    lists[..., 2] = 0
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    got = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)
    one = [x[1:].contiguous() for x in (q, k, v, o, dout, lse, lists)]
    wide = torch.cat([one[6], torch.full_like(one[6], -1)], -1).contiguous()
    alone = kb.sparse_backward(*one[:6], wide, check=True)
    for x, y in zip(got, alone):
        assert torch.equal(x[1:].contiguous().view(torch.uint8), y.view(torch.uint8))
    for g in (0, 7):
        h = slice(4 * g, 4 * g + 4)
        args = f64(q)[1, h], f64(k)[1, g], f64(v)[1, g], f64(dout)[1, h], lists[1, g].cpu().numpy()
        want, tol = plain.gradients(*args), tolerances(*args)
        for x, y, t in zip((got[0][1, h], got[1][1, g], got[2][1, g]), want, tol):
            assert np.all(np.abs(f64(x) - y) <= t + 1e-7)


def test_a_training_step(kb):
    """Rotation, boxes, selection, forward, backward and the rotation's gradient together."""
    import torch

    S, n = 640, 3
    q, k, v, dout = (randn(3500 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    rope = kb.rope_table(S)
    tq, tk = kb.rope(q, rope), kb.rope(k, rope)
    lists = kb.select_blocks(tq, kb.block_boxes(tk), 0, n)
    o, lse = kb.sparse_prefill_lse(tq, tk, v, lists)
    dq, dk, dv, _ = kb.sparse_backward(tq, tk, v, o, dout, lse, lists)
    gq, gk = kb.rope(dq, rope, inverse=True), kb.rope(dk, rope, inverse=True, check=True)
    pos = np.arange(S)
    for g in (0, 5):
        h = slice(4 * g, 4 * g + 4)
        args = f64(tq)[0, h], f64(tk)[0, g], f64(v)[0, g], f64(dout)[0, h], lists[0, g].cpu().numpy()
        want, tol = plain.gradients(*args), tolerances(*args)
        for got, i in ((gq[0, h], 0), (gk[0, g], 1)):
            y = plain.rotate(want[i], pos, inverse=True)
            # a rotation mixes two elements and rounds once more
            pair = tol[i][..., :64] + tol[i][..., 64:]
            t = np.concatenate([pair, pair], -1) + U * np.abs(y)
            assert np.all(np.abs(f64(got) - y) <= t + 1e-7)
        assert np.all(np.abs(f64(dv)[0, g] - want[2]) <= tol[2] + 1e-7)


def test_refusals(kb):
    import torch

    S = 64
    q, k, v, dout = (randn(3600 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = torch.zeros(1, 8, S, 1, dtype=torch.int32, device="cuda")
    o, lse = kb.sparse_prefill_lse(q, k, v, lists, check=True)
    for bad in (lambda: kb.sparse_backward(q, k, v, o, dout[:, :, :-1].contiguous(), lse, lists),
                lambda: kb.sparse_backward(q, k, v, o, dout, lse[..., :-1].contiguous(), lists),
                lambda: kb.sparse_backward(q, k, v, o, dout, lse, lists[:, :4].contiguous()),
                lambda: kb.sparse_backward(q, k, v, o, dout, lse, lists, dk=torch.empty_like(q)),
                lambda: kb.sparse_prefill_lse(q, k[:, :, :-1].contiguous(), v[:, :, :-1].contiguous(), lists)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kb.sparse_backward(q, k, v, o, dout, lse, lists.long())
    with pytest.raises(kb.KBError):
        kb.sparse_backward(q, k, v, o, dout, lse, lists, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    lists[0, 3, 10, 0] = 1                                        # no such block in the sequence
    kb.sparse_backward(q, k, v, o, dout, lse, lists)
    with pytest.raises(kb.KBError):
        kb.check_device_status()


def test_ctas_that_go_from_unit_to_unit(kb):
    """8 KV heads x 152 position tiles are a whole number of units for every SM of this GPU, so a CTA takes several; a
    shorter sequence's are not, and it has the same rows' dq, bit for bit."""
    import torch

    S, short, n = 4864, 2000, 3
    q, k, v, dout = (randn(3800 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = random_lists(3804, 1, S, 0, n, none=0.2)
    lists[:, :, 640:800] = -1
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    whole = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)[0]
    cut = [x[:, :, :short].contiguous() for x in (q, k, v, o, dout, lse, lists)]
    dq = kb.sparse_backward(*cut, check=True)[0]
    assert torch.equal(whole[:, :, :short].contiguous().view(torch.uint8), dq.view(torch.uint8))
    assert not whole[:, :, 640:800].any()
