"""Rotation, cache append and key-block boxes on the GPU against their 64-bit
definitions, and bit for bit across splits, layouts and caches."""

import numpy as np
import pytest

from tests import sparse_plain as plain

pytestmark = pytest.mark.gpu

BF16_HALF_STEP = 2.0 ** -8        # a rounding to bf16 is off by at most this, relative to the value


@pytest.fixture(scope="module")
def kb():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bitwise_aligned_causal_gb300 import build

    build.build()
    from bitwise_aligned_causal_gb300 import kb_attn

    yield kb_attn
    assert kb_attn.kb_attn_check_device_status(None) == kb_attn.KB_OK


def randn(seed, *shape):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    import torch

    return t.contiguous().view(torch.int16)


def assert_rotated(got, x, want):
    # two fp32 products, an fp32 sum and the table's rounding: at most 4 roundings of 2^-24 of the pair's magnitudes
    tol = BF16_HALF_STEP * np.abs(want) + 4 * 2.0 ** -24 * 2 * np.abs(x).max()
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()


@pytest.mark.parametrize("rot_dim,interleaved", [(128, False), (128, True), (64, False), (16, True), (80, False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_definition(kb, rot_dim, interleaved, inverse):
    table = kb.rope_table(200, rot_dim)
    x = randn(1, 2, 37, 7, 128).transpose(1, 2)                  # rows as a projection leaves them, 7 heads
    y = kb.rope(x, table, start=150, inverse=inverse, interleaved=interleaved, check=True)
    want = plain.rotate(f64(x), np.arange(150, 187), rot_dim, interleaved=interleaved, inverse=inverse)
    assert y.is_contiguous() and tuple(y.shape) == (2, 7, 37, 128)
    assert_rotated(f64(y), f64(x), want)


def test_rope_far_positions_and_own_frequencies(kb):
    import torch

    inv = torch.linspace(1.0, 0.01, 8, dtype=torch.float64)
    table = kb.rope_table(2_000_003, 16, inv_freq=inv)
    pos = np.array([0, 1, 1_999_999, 2_000_002])
    got = table[torch.from_numpy(pos).cuda()].double().cpu().numpy()
    ang = pos[:, None] * inv.numpy()
    want = np.stack([np.cos(ang), np.sin(ang)], -1)
    # rounded to fp32 once; the 64-bit angle itself is off by at most 2^-53 of 2e6
    assert np.all(np.abs(got - want) <= 2.0 ** -25 + 2e6 * 2.0 ** -52)
    x = randn(2, 1, 3, 3, 128)
    y = kb.rope(x, table, start=2_000_000)
    for i in range(3):
        a, b = f64(x)[0, :, i, :8], f64(x)[0, :, i, 8:16]
        an = (2_000_000 + i) * inv.numpy()
        assert_rotated(f64(y)[0, :, i, :8], f64(x), a * np.cos(an) - b * np.sin(an))
    assert torch.equal(bits(y[..., 16:]), bits(x[..., 16:]))


def test_rope_in_place_and_one_row(kb):
    import torch

    table = kb.rope_table(64)
    x = randn(3, 3, 5, 33, 128)
    want = kb.rope(x, table, start=7)
    y = x.clone()
    kb.rope(y, table, start=7, out=y)
    assert torch.equal(bits(y), bits(want))
    one = kb.rope(x[:, :, 20:21], table, start=27)
    assert torch.equal(bits(one), bits(want[:, :, 20:21]))


def test_rope_gradient_is_the_adjoint(kb):
    """sum(dout * rope(x)) differentiated along dx equals sum(inverse(dout) * dx): checked by a difference, which is
    exact for a linear map up to the roundings of both sides."""
    table = kb.rope_table(500)
    x, dx, dout = randn(4, 1, 8, 400, 128), randn(5, 1, 8, 400, 128), randn(6, 1, 8, 400, 128)
    grad = f64(kb.rope(dout, table, inverse=True, check=True))
    pos = np.arange(400)
    h = 1.0 / 1024
    diff = (f64(dout) * (plain.rotate(f64(x) + h * f64(dx), pos) - plain.rotate(f64(x) - h * f64(dx), pos))).sum() / (2 * h)
    # every element of the gradient is off by half a bf16 step at most
    assert abs((grad * f64(dx)).sum() - diff) <= BF16_HALF_STEP * np.abs(grad * f64(dx)).sum() + 1e-6
    want = plain.rotate(f64(dout), pos, inverse=True)
    assert_rotated(grad, f64(dout), want)


def caches(B, cap, page=0, extra=2, seed=0):
    """Zero-free caches, page table and a function that reads sequence b as [8, cap, 128]."""
    import torch

    if not page:
        k, v = randn(seed, B, 8, cap, 128), randn(seed + 1, B, 8, cap, 128)
        bx = torch.zeros(B, 8, -(-cap // 128), 2, 128, dtype=torch.bfloat16, device="cuda")
        return k, v, bx, None, lambda t, b: t[b]
    per = cap // page
    n = B * per + extra
    g = torch.Generator().manual_seed(seed + 5)
    table = torch.randperm(n, generator=g)[:B * per].view(B, per).to(torch.int32).cuda()
    k, v = randn(seed, n, 8, page, 128), randn(seed + 1, n, 8, page, 128)
    bx = torch.zeros(n, 8, page // 128, 2, 128, dtype=torch.bfloat16, device="cuda")
    return k, v, bx, table, lambda t, b: t[table[b].long()].transpose(0, 1).reshape(8, -1, *t.shape[3:])


@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("starts,lens,L", [((0, 0, 0), (300, 1, 0), 300), ((127, 128, 255), (1, 1, 1), 1),
                                           ((100, 5, 384), (257, 130, 128), 257), ((0, 511, 64), (1, 1, 1), 1)])
def test_append_writes_the_new_rows_and_their_boxes(kb, page, starts, lens, L):
    import torch

    B, cap = 3, 768
    k_cache, v_cache, bx, table_pages, seq = caches(B, cap, page, seed=10)
    k0, v0 = k_cache.clone(), v_cache.clone()
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if max(starts):
        kb.block_boxes(k_cache, kv_len=cap, kv_lens=st, block_table=table_pages, boxes=bx, check=True)
    rope = kb.rope_table(cap)
    fused = randn(20, B, L, 48, 128).transpose(1, 2)              # q | k | v of one projection
    q, k, v = fused[:, :32], fused[:, 32:40], fused[:, 40:]
    out = torch.full((B, 32, L, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = kb.append_varlen(q, k, v, k_cache, v_cache, rope, st, ln, block_table=table_pages, boxes=bx, out=out,
                           check=True)
    assert got is out
    touched_k, touched_v = torch.zeros_like(k0, dtype=torch.bool), torch.zeros_like(k0, dtype=torch.bool)
    for b in range(B):
        s, n = starts[b], lens[b]
        assert bool((out[b, :, n:] == 7.0).all())
        if n == 0:
            continue
        want_q = kb.rope(q[b:b + 1, :, :n], rope, start=s)
        want_k = kb.rope(k[b:b + 1, :, :n], rope, start=s)
        assert torch.equal(bits(out[b, :, :n]), bits(want_q[0]))
        assert torch.equal(bits(seq(k_cache, b)[:, s:s + n]), bits(want_k[0]))
        assert torch.equal(bits(seq(v_cache, b)[:, s:s + n]), bits(v[b, :, :n]))
        want_box = plain.boxes(f64(seq(k_cache, b)[:, :s + n]))
        first = s // 128
        assert np.array_equal(f64(seq(bx, b))[:, first:want_box.shape[1]], want_box[:, first:])
        # the rows around are as they were
        assert torch.equal(bits(seq(k_cache, b)[:, :s]), bits(seq(k0, b)[:, :s]))
        assert torch.equal(bits(seq(k_cache, b)[:, s + n:]), bits(seq(k0, b)[:, s + n:]))
        assert torch.equal(bits(seq(v_cache, b)[:, s + n:]), bits(seq(v0, b)[:, s + n:]))
    if page:                                                      # pages of no sequence
        free = sorted(set(range(k0.shape[0])) - set(table_pages.view(-1).tolist()))
        assert torch.equal(bits(k_cache[free]), bits(k0[free]))


@pytest.mark.parametrize("splits", [(1,) * 40 + (90, 200, 1, 128, 141), (300, 300), (599, 1)])
def test_any_split_gives_the_same_bits(kb, splits):
    import torch

    S = 600
    assert sum(splits) == S
    q, k, v = randn(30, 1, 32, S, 128), randn(31, 1, 8, S, 128) * 3, randn(32, 1, 8, S, 128)
    k[:, :, 200] *= 64                                            # one key widens its block's grid late
    rope = kb.rope_table(S)
    kw, vw, bw, _, _ = caches(1, S, seed=40)
    qw = kb.append(q, k, v, kw, vw, rope, 0, boxes=bw)
    ks, vs, bs, _, _ = caches(1, S, seed=41)
    bs.fill_(float("nan"))
    at, rows = 0, []
    for n in splits:
        rows.append(kb.append(q[:, :, at:at + n], k[:, :, at:at + n], v[:, :, at:at + n], ks, vs, rope, at, boxes=bs))
        at += n
    kb.check_device_status()
    for a, b in ((torch.cat(rows, 2), qw), (ks, kw), (vs, vw)):
        assert torch.equal(bits(a), bits(b))
    assert torch.equal(bs, bw) and torch.equal(bw, kb.block_boxes(kw, check=True))
    assert np.array_equal(f64(bw)[0], plain.boxes(f64(kw)[0]))


def test_append_without_queries_table_or_boxes(kb):
    import torch

    k_cache, v_cache, _, _, _ = caches(2, 200, seed=50)
    k, v = randn(51, 2, 8, 70, 128), randn(52, 2, 8, 70, 128)
    assert kb.append(None, k, v, k_cache, v_cache, None, 130, check=True) is None
    assert torch.equal(bits(k_cache[:, :, 130:]), bits(k)) and torch.equal(bits(v_cache[:, :, 130:]), bits(v))


@pytest.mark.parametrize("scale", [0.0, 1e-38, 2.0 ** -107, 1.0, 1.984375, 3e38])
def test_boxes_over_the_whole_range(kb, scale):
    """Zero, tiny, ordinary and the largest keys; 127/128 of a power of two sits on the grid's border."""
    import torch

    k = torch.clamp(randn(60, 1, 8, 300, 128).float(), -1, 1) * scale
    k[:, :, :, 0] = -scale
    k = k.to(torch.bfloat16)
    bx = f64(kb.block_boxes(k, check=True))[0]
    assert np.array_equal(bx, plain.boxes(f64(k)[0]))


def test_non_finite_keys_keep_boxes_finite(kb):
    import torch

    k = randn(61, 1, 8, 128, 128)
    k[0, 0, 5, 3], k[0, 1, 6, 4], k[0, 2, :, 7] = float("inf"), float("nan"), float("nan")
    assert bool(torch.isfinite(kb.block_boxes(k, check=True)).all())


def test_bad_device_arguments_are_recorded_and_nothing_is_written(kb):
    import torch

    rope = kb.rope_table(512)
    q, k, v = randn(70, 2, 32, 4, 128), randn(71, 2, 8, 4, 128), randn(72, 2, 8, 4, 128)
    for starts, lens, pages in (((0, -1), (4, 4), None), ((0, 509), (4, 4), None), ((0, 0), (4, 5), None),
                                ((0, 0), (4, -1), None), ((0, 0), (4, 4), 6), ((0, 0), (4, 4), -1)):
        k_cache, v_cache, bx, table, seq = caches(2, 512, 256, seed=73)
        if pages is not None:
            table[1, 0] = pages
        k0 = k_cache.clone()
        out = torch.full_like(q, 5.0)
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kb.append_varlen(q, k, v, k_cache, v_cache, rope, st, ln, block_table=table, boxes=bx, out=out)
        with pytest.raises(kb.KBError):
            kb.check_device_status()
        assert bool((out[1] == 5.0).all())
        rest = [p for p in range(k0.shape[0]) if p not in table[0].tolist()]
        assert torch.equal(bits(k_cache[rest]), bits(k0[rest]))


def test_append_on_another_stream_and_replayed(kb):
    """A captured append replays with the positions its device arrays hold then."""
    import torch

    rope = kb.rope_table(512)
    q, k, v = randn(80, 2, 32, 1, 128), randn(81, 2, 8, 1, 128), randn(82, 2, 8, 1, 128)
    k_cache, v_cache, bx, table, seq = caches(2, 512, 256, seed=83)
    st = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    kb.append_varlen(q, k, v, k_cache, v_cache, rope, st, block_table=table, boxes=bx, out=out, check=True)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            kb.append_varlen(q, k, v, k_cache, v_cache, rope, st, block_table=table, boxes=bx, out=out)
            st.add_(1)
    for step in range(3):
        graph.replay()
    torch.cuda.synchronize()
    kb.check_device_status()
    for b, first in ((0, 3), (1, 4)):
        for step in range(3):
            want = kb.rope(k[b:b + 1], rope, start=first + step)
            assert torch.equal(bits(seq(k_cache, b)[:, first + step]), bits(want[0, :, 0]))
    assert torch.equal(bits(out[:1]), bits(kb.rope(q[:1], rope, start=5)))
