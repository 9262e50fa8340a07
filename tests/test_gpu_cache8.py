"""A KV cache held in 8 bits: what appends write, byte for byte, and the
attention over it, bit for bit against the attention over the bf16 cache that
holds the same values."""

import numpy as np
import pytest

from tests import cache_plain as plain
from tests.test_gpu_append import bits, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def empty8(B, cap, page=0, extra=2, seed=0, fill=0x35, exp=3):
    """Caches of arbitrary bytes, exponents, page table, and a function that reads sequence b as [8, cap, ...]."""
    import torch

    if page:
        per = cap // page
        g = torch.Generator().manual_seed(seed + 5)
        table = torch.randperm(B * per + extra, generator=g)[:B * per].view(B, per).to(torch.int32).cuda()
        shape = (B * per + extra, 8, page)
    else:
        table, shape = None, (B, 8, cap)
    c = [torch.full((*shape, 128), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    e = [torch.full((*shape[:2], -(-shape[2] // 128)), exp, dtype=torch.int8, device="cuda") for _ in range(2)]

    def seq(t, b):
        if t.dtype == torch.float8_e4m3fn:
            t = t.view(torch.uint8)
        return t[b] if table is None else t[table[b].long()].transpose(0, 1).reshape(8, -1, *t.shape[3:])

    return *c, *e, table, seq


def held(t, e):
    """64-bit values of a uint8 [8, rows, 128] with exponents [8, blocks]."""
    import torch

    x = t.contiguous().view(torch.float8_e4m3fn).double().cpu().numpy()
    return x * np.repeat(2.0 ** e.double().cpu().numpy(), 128, axis=1)[:, :x.shape[1], None]


def table_rows(table, a, n):
    return table[a:a + n].cpu().numpy()


@pytest.mark.parametrize("page", [0, 128, 256])
@pytest.mark.parametrize("starts,lens,L", [((0, 0, 0), (300, 1, 0), 300), ((100, 5, 384), (257, 130, 128), 257),
                                           ((0, 511, 64), (1, 1, 1), 1), ((0, 0, 128), (3, 128, 97), 130)])
def test_append_writes_the_defined_bytes(kb, page, starts, lens, L):
    import torch

    B, cap = 3, 768
    k8, v8, ke, ve, pages, seq = empty8(B, cap, page, seed=10)
    rope = kb.rope_table(cap)
    st, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (starts, lens))
    # what lies before the new rows: loud and quiet keys, from the start of the sequence
    old = [randn(30 + i, B, 8, max(max(starts), 1), 128) * (0.1 if i else 4.0) for i in range(2)]
    if max(starts):
        kb.append_8bit_varlen(None, *old, k8, v8, ke, ve, None, torch.zeros_like(st), st, block_table=pages, check=True)
    before = [t.view(torch.uint8).clone() for t in (k8, v8)]
    exps = [t.clone() for t in (ke, ve)]
    fused = randn(20, B, L, 48, 128).transpose(1, 2)              # q | k | v of one projection
    q, k, v = fused[:, :32], fused[:, 32:40], fused[:, 40:]
    out = torch.full((B, 32, L, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kb.append_8bit_varlen(q, k, v, k8, v8, ke, ve, rope, st, ln, block_table=pages, out=out, check=True) is out
    for b in range(B):
        s, n = starts[b], lens[b]
        assert bool((out[b, :, n:] == 7.0).all())
        if n == 0:
            for t, e, t0, e0 in ((k8, ke, before[0], exps[0]), (v8, ve, before[1], exps[1])):
                assert torch.equal(seq(t, b), seq(t0, b)) and torch.equal(seq(e, b), seq(e0, b))
            continue
        assert torch.equal(bits(out[b, :, :n]), bits(kb.rope(q[b:b + 1, :, :n], rope, start=s)[0]))
        new_k = plain.rotate32(k[b, :, :n].float().cpu().numpy(), table_rows(rope, s, n))
        for t, e, o, new in ((k8, ke, old[0], new_k), (v8, ve, old[1], f64(v[b, :, :n]))):
            want, want_e = plain.blocks8(np.concatenate([f64(o[b, :, :s]), new], 1))
            first = s // 128
            got, got_e = seq(t, b), seq(e, b)
            assert np.array_equal(got_e.cpu().numpy()[:, :want_e.shape[1]], want_e)
            assert np.array_equal(held(got[:, :s + n], got_e), want)
        # rows behind, and pages of no sequence, are as they were
        for t, t0 in ((k8, before[0]), (v8, before[1])):
            assert torch.equal(seq(t, b)[:, s + n:], seq(t0, b)[:, s + n:])
    if page:
        free = sorted(set(range(k8.shape[0])) - set(pages.view(-1).tolist()))
        assert bool((k8.view(torch.uint8)[free] == 0x35).all()) and bool((ke[free] == 3).all())


@pytest.mark.parametrize("splits", [(1,) * 40 + (90, 200, 1, 128, 141), (300, 300), (599, 1), (127, 2, 471)])
def test_any_split_gives_the_same_bytes(kb, splits):
    import torch

    S = 600
    assert sum(splits) == S
    q, k, v = randn(30, 1, 32, S, 128), randn(31, 1, 8, S, 128) * 3, randn(32, 1, 8, S, 128)
    loud = torch.tensor([1e-6, 1e-3, 1.0, 40.0, 1e4], device="cuda")[torch.arange(S, device="cuda") * 7 // 128 % 5]
    k, v = k * loud[None, None, :, None].bfloat16(), v * loud.flip(0)[None, None, :, None].bfloat16()
    rope = kb.rope_table(S)
    whole, parts = empty8(1, S), empty8(1, S, fill=0x77, exp=-9)
    qw = kb.append_8bit(q, k, v, *whole[:4], rope, 0)
    at, rows = 0, []
    for n in splits:
        rows.append(kb.append_8bit(q[:, :, at:at + n], k[:, :, at:at + n], v[:, :, at:at + n], *parts[:4], rope, at))
        at += n
    kb.check_device_status()
    assert torch.equal(bits(torch.cat(rows, 2)), bits(qw))
    for a, b in zip(parts[:4], whole[:4]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("rot_dim,interleaved", [(128, True), (64, False), (16, True)])
def test_other_rotations(kb, rot_dim, interleaved):
    S = 200
    k, v = randn(40, 1, 8, S, 128), randn(41, 1, 8, S, 128)
    rope = kb.rope_table(S, rot_dim)
    k8, v8, ke, ve, _, seq = empty8(1, S)
    assert kb.append_8bit(None, k, v, k8, v8, ke, ve, rope, 0, interleaved=interleaved, check=True) is None
    want, want_e = plain.blocks8(plain.rotate32(k[0].float().cpu().numpy(), table_rows(rope, 0, S), interleaved))
    assert np.array_equal(ke[0].cpu().numpy(), want_e) and np.array_equal(held(seq(k8, 0), ke[0]), want)


@pytest.mark.parametrize("scale", [0.0, 1e-38, 2.0 ** -107, 448 * 2.0 ** -12, 3e38])
def test_the_whole_range(kb, scale):
    """Zero, tiny, the border of an exponent, and the largest values; fp32 holds what rotation leaves."""
    import torch

    S = 130
    x = torch.clamp(randn(50, 1, 8, S, 128).float(), -1, 1)
    x[:, :, 3] = 1.0                                              # the largest magnitude is `scale`
    x = (x * scale).bfloat16()
    k8, v8, ke, ve, _, seq = empty8(1, S)
    kb.append_8bit(None, x, -x, k8, v8, ke, ve, None, 0, check=True)
    want, want_e = plain.blocks8(f64(x[0]))
    assert np.array_equal(ke[0].cpu().numpy(), want_e) and torch.equal(ke, ve)
    got = held(seq(k8, 0), ke[0])
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
    assert np.array_equal(held(seq(v8, 0), ve[0]), -want)
    values = kb.cache_values(k8, ke, check=True)
    assert np.array_equal(f64(values)[0], want)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite_mark_their_block(kb, bad):
    import torch

    S = 300
    k, v = randn(60, 1, 8, S, 128), randn(61, 1, 8, S, 128)
    k[0, 2, 140, 5] = bad
    v[0, 3, 299, 127] = bad
    whole, parts = empty8(1, S), empty8(1, S, fill=1, exp=5)
    kb.append_8bit(None, k, v, *whole[:4], None, 0, check=True)
    for at, n in ((0, 130), (130, 30), (160, 40), (200, 100)):
        kb.append_8bit(None, k[:, :, at:at + n], v[:, :, at:at + n], *parts[:4], None, at, check=True)
    for a, b in zip(parts[:4], whole[:4]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    k8, v8, ke, ve = whole[:4]
    assert (ke == 127).nonzero().tolist() == [[0, 2, 1]] and (ve == 127).nonzero().tolist() == [[0, 3, 2]]
    for c, e, x in ((k8, ke, k), (v8, ve, v)):
        y = kb.cache_values(c, e)
        nan = torch.isnan(y)
        assert int(nan.sum()) in (128 * 128, 44 * 128)
        want, _ = plain.blocks8(f64(x[0]))
        assert np.array_equal(f64(y)[0], want, equal_nan=True)
    # the rows that see the marked keys are NaN, the others are not
    q = randn(62, 1, 32, S, 128)
    o = kb.chunk_8bit(q, *whole[:4], 0, check=True)
    assert bool(torch.isnan(o[0, 8:12, 128:]).any(-1).all()) or bad != bad
    assert bool(torch.isfinite(o[0, 8:12, :128]).all()) and bool(torch.isfinite(o[0, :8]).all())
    d = kb.decode_8bit(q[:, :, 255:256].contiguous(), *whole[:4], 256, check=True)
    assert bool(torch.isnan(d[0, 8:12]).all()) and bool(torch.isfinite(d[0, 12:]).all())
    # the first row anew: the block's mark is gone
    kb.append_8bit(None, randn(63, 1, 8, 1, 128), randn(64, 1, 8, 1, 128), *whole[:4], None, 128, check=True)
    assert bool((ke[0, :, 1] < 100).all())


@pytest.mark.parametrize("planes,Hkv,rows", [(1, 1, 1), (3, 8, 127), (2, 8, 129), (5, 3, 640)])
def test_every_byte_reads_as_its_value(kb, planes, Hkv, rows):
    """All 256 bytes, e4m3's own subnormals included, at every exponent."""
    import torch

    c = (torch.arange(planes * Hkv * rows * 128, device="cuda") % 256).to(torch.uint8).view(planes, Hkv, rows, 128)
    c[(c & 0x7F) == 0x7F] = 0
    blocks = -(-rows // 128)
    e = (torch.arange(planes * Hkv * blocks, device="cuda") * 17 % 201 - 100).to(torch.int8).view(planes, Hkv, blocks)
    e.view(-1)[0] = -100
    got = f64(kb.cache_values(c.view(torch.float8_e4m3fn), e, check=True))
    for p in range(planes):
        assert np.array_equal(got[p], held(c[p], e[p]))
    edge = torch.tensor([-128, -101, 101, 126], dtype=torch.int8, device="cuda")     # read as the nearest in range
    near = torch.tensor([-100, -100, 100, 100], dtype=torch.int8, device="cuda")
    x = c.view(-1)[:128].view(1, 1, 1, 128).expand(4, 1, 1, 128).contiguous().view(torch.float8_e4m3fn)
    assert torch.equal(bits(kb.cache_values(x, edge.view(4, 1, 1))), bits(kb.cache_values(x, near.view(4, 1, 1))))


# ------------------------------------------------------------------ attention

def filled(kb, B, cap, page=0, seed=70, n=None):
    """An 8-bit cache of n keys per sequence whose blocks differ in loudness, behind them bytes of NaN."""
    import torch

    n = cap if n is None else n
    k8, v8, ke, ve, pages, seq = empty8(B, cap, page, seed=seed, fill=0x7F, exp=127)
    k, v = randn(seed, B, 8, n, 128), randn(seed + 1, B, 8, n, 128)
    loud = torch.exp(torch.randn(n // 128 + 1, generator=torch.Generator().manual_seed(seed)) * 0.3).cuda()
    k = k * loud[torch.arange(n, device="cuda") // 128][None, None, :, None].bfloat16()
    v = v * (loud * loud)[torch.arange(n, device="cuda") // 128][None, None, :, None].bfloat16()
    starts = torch.zeros(B, dtype=torch.int32, device="cuda")
    kb.append_8bit_varlen(None, k, v, k8, v8, ke, ve, None, starts, block_table=pages, check=True)
    return (k8, v8, ke, ve), pages, seq


def bf16_of(kb, cache, pages, seq, B):
    """Contiguous bf16 caches [B, 8, cap, 128] of the same values."""
    import torch

    return [torch.stack([seq(kb.cache_values(c, e), b) for b in range(B)]) for c, e in zip(cache[:2], cache[2:])]


@pytest.mark.parametrize("page", [0, 128, 384])
@pytest.mark.parametrize("B,ctx", [(1, 1), (2, 127), (1, 128), (3, 129), (1, 1025), (2, 5000), (1, 20000), (20, 700)])
def test_decode_has_the_bits_of_the_bf16_cache(kb, page, B, ctx):
    import torch

    cap = -(-(ctx + 3) // (page or 1)) * (page or 1)
    cache, pages, seq = filled(kb, B, cap, page, n=ctx)
    q = randn(80, B, 32, 1, 128)
    k, v = (t[:, :, :ctx].contiguous() for t in bf16_of(kb, cache, pages, seq, B))
    want = kb.decode(q, k, v, ctx, check=True)
    assert bool(torch.isfinite(want).all())
    if page:
        lens = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
        got = kb.decode_8bit_paged(q, *cache, pages, lens, check=True)
    else:
        got = kb.decode_8bit(q, *cache, ctx, check=True)
    assert torch.equal(bits(got), bits(want))
    pos = torch.full((B,), ctx - 1, dtype=torch.int32, device="cuda")
    again = kb.chunk_8bit_varlen(q, *cache, pos, torch.ones_like(pos), block_table=pages, check=True)
    assert torch.equal(bits(again), bits(want))


@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("lens", [(9000,) * 20, (1, 9000, 1024, 1025, 127, 128, 5000, 129, 8999, 3, 7168, 2049, 6000, 6001, 800, 9000, 2048, 4097, 1, 8193),
                                  tuple(200 * i + 1 for i in range(37))])
def test_tokens_of_many_contexts(kb, page, lens):
    """Batches that fill the SMs unevenly: runs of segments cut across sequences and heads."""
    import torch

    B, cap = len(lens), -(-max(lens) // 128) * 128
    cache, pages, seq = filled(kb, B, cap, page, seed=7)
    k, v = bf16_of(kb, cache, pages, seq, B)
    q = randn(89, B, 32, 1, 128)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = torch.cat([kb.decode(q[b:b + 1], k[b:b + 1], v[b:b + 1], lens[b]) for b in range(B)])
    got = kb.decode_8bit_paged(q, *cache, pages, n, check=True) if page else kb.chunk_8bit_varlen(q, *cache, n - 1, torch.ones_like(n), check=True)
    assert torch.equal(bits(got), bits(want))
    if not page and len(set(lens)) == 1:
        assert torch.equal(bits(kb.decode_8bit(q, *cache, lens[0], check=True)), bits(want))
    # some of them without a row
    on = torch.arange(B, device="cuda") % 3 != 1
    out = torch.full_like(q, 7.0)
    kb.chunk_8bit_varlen(q, *cache, n - 1, on.int(), block_table=pages, out=out, check=True)
    assert torch.equal(bits(out[on]), bits(want[on])) and bool((out[~on] == 7.0).all())
    # a length out of range is reported, and the next call is as ever
    n[5] = cap + 1
    with pytest.raises(kb.KBError):
        kb.chunk_8bit_varlen(q, *cache, n - 1, torch.ones_like(n), block_table=pages, check=True)
    n[5] = lens[5]
    assert torch.equal(bits(kb.chunk_8bit_varlen(q, *cache, n - 1, torch.ones_like(n), block_table=pages, check=True)), bits(want))


@pytest.mark.parametrize("page", [0, 256])
@pytest.mark.parametrize("B,L,start", [(1, 2, 126), (2, 2, 127), (1, 3, 0), (2, 7, 1500), (1, 32, 1000), (3, 32, 112), (1, 33, 500),
                                       (2, 130, 60), (1, 700, 0), (1, 257, 2047), (1, 5, 9000), (2, 32, 4090), (1, 2, 20479)])
def test_chunks_have_the_bits_of_the_bf16_cache(kb, page, B, L, start):
    import torch

    cap = -(-(start + L + 5) // (page or 1)) * (page or 1)
    cache, pages, seq = filled(kb, B, cap, page, n=start + L)
    q = randn(81, B, 32, L, 128)
    k, v = (t[:, :, :start + L].contiguous() for t in bf16_of(kb, cache, pages, seq, B))
    want = kb.chunk(q, k, v, start, check=True)
    assert bool(torch.isfinite(want).all())
    if page == 0:
        got = kb.chunk_8bit(q, *cache, start, check=True)
        assert torch.equal(bits(got), bits(want))
    st = torch.full((B,), start, dtype=torch.int32, device="cuda")
    got = kb.chunk_8bit_varlen(q, *cache, st, torch.full_like(st, L), block_table=pages, check=True)
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("L,starts,lens", [(1, (0, 299, 40), (1, 1, 0)), (9, (120, 0, 700), (9, 4, 0)), (32, (0, 127, 900), (32, 1, 20)),
                                           (300, (0, 100, 724), (300, 0, 299))])
def test_ragged_chunks(kb, page, L, starts, lens):
    import torch

    B, cap = 3, 1024
    cache, pages, seq = filled(kb, B, cap, page)
    q = randn(82, B, 32, L, 128)
    q[1, :, lens[1]:] = float("nan")                              # rows of no sequence
    st, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (starts, lens))
    out = torch.full((B, 32, L, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kb.chunk_8bit_varlen(q, *cache, st, ln, block_table=pages, out=out, check=True) is out
    k, v = bf16_of(kb, cache, pages, seq, B)
    want = kb.chunk_varlen(q, k, v, st, ln, out=torch.full_like(out, 7.0), check=True)
    assert torch.equal(bits(out), bits(want))
    for b in range(B):
        assert bool((out[b, :, lens[b]:] == 7.0).all())


@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("B,L,start", [(1, 33, 9000), (1, 64, 20448), (2, 100, 12001), (1, 200, 24577), (3, 65, 8100), (1, 300, 9000)])
def test_longer_chunks_late_in_a_context(kb, page, B, L, start):
    """Few query rows for many keys: the ways that fill the SMs, against the packed kernel's rows over bf16."""
    import torch

    cap = -(-(start + L + 5) // (page or 1)) * (page or 1)
    cache, pages, seq = filled(kb, B, cap, page, n=start + L)
    q = randn(83, B, 32, L, 128)
    k, v = (t[:, :, :start + L].contiguous() for t in bf16_of(kb, cache, pages, seq, B))
    want = torch.cat([kb.chunk(q[:, :, i:i + 32].contiguous(), k, v, start + i, check=True) for i in range(0, L, 32)], 2)
    assert bool(torch.isfinite(want).all())
    assert torch.equal(bits(kb.chunk(q, k, v, start, check=True)), bits(want))
    if page == 0:
        assert torch.equal(bits(kb.chunk_8bit(q, *cache, start, check=True)), bits(want))
    # sequences of their own: the last one row short, the one before empty
    lens = [L] * B
    lens[-1] = L - 1
    if B > 1:
        lens[-2] = 0
    st, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([start] * B, lens))
    out = torch.full_like(q, 7.0)
    kb.chunk_8bit_varlen(q, *cache, st, ln, block_table=pages, out=out, check=True)
    for b in range(B):
        assert torch.equal(bits(out[b, :, :lens[b]]), bits(want[b, :, :lens[b]])) and bool((out[b, :, lens[b]:] == 7.0).all())


@pytest.mark.parametrize("kind", ["grows", "falls", "jumps"])
@pytest.mark.parametrize("L", [1, 2, 6, 40])
def test_rows_whose_maximum_moves(kb, kind, L):
    """Keys along the queries, louder or quieter tile by tile: rows that are scaled again and again, and never."""
    import torch

    S = 3000
    at = torch.arange(S, device="cuda")
    scale = {"grows": 0.2 + at / S * 6, "falls": 6.2 - at / S * 6, "jumps": 0.3 + 5.0 * ((at // 128) % 3)}[kind]
    q = randn(84, 1, 32, L, 128)
    k = (randn(85, 1, 8, S, 128) + q.view(1, 8, 4 * L, 128).mean(2, keepdim=True)) * scale[None, None, :, None].bfloat16()
    v = randn(87, 1, 8, S, 128)
    k8, v8, ke, ve = empty8(1, S)[:4]
    kb.append_8bit(None, k, v, k8, v8, ke, ve, None, 0, check=True)
    kk, vv = kb.cache_values(k8, ke), kb.cache_values(v8, ve)
    want = kb.chunk(q, kk, vv, S - L, check=True)
    assert torch.equal(bits(kb.chunk_8bit(q, k8, v8, ke, ve, S - L, check=True)), bits(want))


def test_longer_chunks_captured_and_on_two_streams(kb):
    import torch

    L, start = 70, 12000
    cache, _, _ = filled(kb, 1, start + L)
    q = randn(88, 1, 32, L, 128)
    want = kb.chunk_8bit(q, *cache, start, check=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [kb.chunk_8bit(q, *cache, start, stream=st) for st in streams for _ in range(3)]
    torch.cuda.synchronize()
    g, o = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(g):
        kb.chunk_8bit(q, *cache, start, out=o)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(want))
    kb.check_device_status()
    assert all(torch.equal(bits(x), bits(want)) for x in got)


@pytest.mark.parametrize("B,L,start", [(1, 1, 9000), (2, 1, 70000), (1, 20, 9000)])
def test_without_a_workspace_and_with_one_of_its_own(kb, B, L, start):
    """Long contexts of small batches: CTAs that share a KV head's keys through the workspace, and the way without."""
    import torch

    ctx = start + L
    cache, _, _ = filled(kb, B, ctx)
    q = randn(86, B, 32, L, 128)
    want = kb.chunk_8bit(q, *cache, start, check=True)
    nbytes = kb.kb_attn_chunk_8bit_workspace_bytes(B, 8, L, ctx)
    assert nbytes > 0
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(bits(kb.chunk_8bit(q, *cache, start, workspace=ws, check=True)), bits(want))
    with pytest.raises(kb.KBError):
        kb.chunk_8bit(q, *cache, start, workspace=ws[:-256])
    ptrs = [t.data_ptr() for t in (q, *cache)]
    o = torch.zeros_like(q)
    s = torch.cuda.current_stream().cuda_stream
    assert kb.kb_attn_chunk_8bit(*ptrs, o.data_ptr(), B, 32, 8, L, start, None, None, ctx, None, 0, 0, 0, None, 0, s) == kb.KB_OK
    kb.check_device_status()
    assert torch.equal(bits(o), bits(want))
    if L == 1:
        assert kb.kb_attn_decode_8bit(*ptrs, o.zero_().data_ptr(), B, 32, 8, ctx, None, ctx, None, 0, 0, 0, None, 0, s) == kb.KB_OK
        kb.check_device_status()
        assert torch.equal(bits(o), bits(want))


def test_against_64_bits(kb):
    """Weights and outputs are rounded to bf16 (half a step each); scores and sums are fp32."""
    cache, pages, seq = filled(kb, 1, 1500)
    k, v = (f64(kb.cache_values(c, e))[0] for c, e in zip(cache[:2], cache[2:]))
    q = randn(83, 1, 32, 20, 128)
    o = f64(kb.chunk_8bit(q, *cache, 1480, check=True))[0]
    for g in range(8):
        want, _, mag = plain.attend(f64(q)[0, 4 * g:4 * g + 4], k[g], v[g], np.arange(1480, 1500))
        assert np.all(np.abs(o[4 * g:4 * g + 4] - want) <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * np.abs(want))


def test_bad_device_arguments_are_reported(kb):
    import torch

    cache, pages, seq = filled(kb, 2, 512, 128)
    q = randn(84, 2, 32, 1, 128)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for lens in (i32(0, 5), i32(5, 513)):
        with pytest.raises(kb.KBError):
            kb.decode_8bit_paged(q, *cache, pages, lens, check=True)
    for bad in (-1, 10, 2 ** 31 - 1):
        broken = pages.clone()
        broken[1, 0] = bad
        with pytest.raises(kb.KBError):
            kb.decode_8bit_paged(q, *cache, broken, i32(5, 5), check=True)
        with pytest.raises(kb.KBError):
            kb.chunk_8bit_varlen(randn(85, 2, 32, 40, 128), *cache, i32(0, 0), i32(40, 40), block_table=broken, check=True)
        with pytest.raises(kb.KBError):
            kb.append_8bit_varlen(None, randn(86, 2, 8, 3, 128), randn(87, 2, 8, 3, 128), *cache, None, i32(0, 0), block_table=broken,
                                  check=True)
    for st, ln in ((i32(-1, 0), i32(1, 1)), (i32(512, 0), i32(1, 1)), (i32(0, 0), i32(2, 1)), (i32(0, 0), i32(-1, 1))):
        with pytest.raises(kb.KBError):
            kb.chunk_8bit_varlen(q, *cache, st, ln, block_table=pages, check=True)
    assert bool(torch.isfinite(kb.decode_8bit_paged(q, *cache, pages, i32(5, 512), check=True)).all())


def test_refusals(kb):
    import torch

    cache, _, _ = filled(kb, 1, 300)
    k8, v8, ke, ve = cache
    q, k = randn(88, 1, 32, 1, 128), randn(89, 1, 8, 1, 128)
    for args in ((q, k8.view(torch.uint8), v8, ke, ve, 5), (q, k8, v8, ke.int(), ve, 5), (q.float(), k8, v8, ke, ve, 5), (q, k8.cpu(), v8, ke, ve, 5)):
        with pytest.raises(TypeError):
            kb.decode_8bit(*args)
    for args in ((q, k8, v8, ke, ve, 0), (q, k8, v8, ke, ve, 301), (q, k8, v8, ke[:, :, :2].contiguous(), ve, 5)):
        with pytest.raises(ValueError):
            kb.decode_8bit(*args)
    with pytest.raises(ValueError):
        kb.append_8bit(None, k, k, k8, v8, ke, ve, None, 300)
    with pytest.raises(ValueError):
        kb.append_8bit(None, k, k, k8, v8, ke, ve, kb.rope_table(10), 10)
    with pytest.raises(TypeError):
        kb.append_8bit(None, k, k, k8.to(torch.bfloat16), v8, ke, ve, None, 0)
    with pytest.raises(TypeError):
        kb.chunk_8bit_varlen(q, *cache, None, None)
    with pytest.raises(kb.KBError):
        kb.chunk_8bit(randn(90, 1, 32, 40, 128), *cache, 0, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_two_streams_and_a_captured_step(kb):
    """A decode step captured with its append, replayed as the cache grows; and two calls at once on two streams."""
    import torch

    S = 400
    q, k, v = randn(91, 1, 32, S, 128), randn(92, 1, 8, S, 128), randn(93, 1, 8, S, 128)
    rope = kb.rope_table(S)
    a, b = empty8(1, S), empty8(1, S)
    for c in (a, b):
        kb.append_8bit(None, k[:, :, :380], v[:, :, :380], *c[:4], rope, 0, check=True)
    qs, ks, vs = (torch.empty(1, h, 1, 128, dtype=torch.bfloat16, device="cuda") for h in (32, 8, 8))
    turned, o = torch.empty_like(qs), torch.empty_like(qs)
    pos, one = torch.full((1,), 380, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        kb.append_8bit_varlen(qs, ks, vs, *a[:4], rope, pos, one, out=turned)
        kb.chunk_8bit_varlen(turned, *a[:4], pos, one, out=o)
    for p in range(380, S):
        qs.copy_(q[:, :, p:p + 1]), ks.copy_(k[:, :, p:p + 1]), vs.copy_(v[:, :, p:p + 1]), pos.fill_(p)
        g.replay()
        t = kb.append_8bit(q[:, :, p:p + 1], k[:, :, p:p + 1], v[:, :, p:p + 1], *b[:4], rope, p)
        assert torch.equal(bits(o), bits(kb.decode_8bit(t, *b[:4], p + 1)))
    kb.check_device_status()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [kb.chunk_8bit(q, *b[:4], 0, stream=st) for st in streams for _ in range(4)]
    torch.cuda.synchronize()
    want = kb.chunk_8bit(q, *b[:4], 0, check=True)
    assert all(torch.equal(bits(x), bits(want)) for x in got)


def test_far_rows(kb):
    """Caches beyond 2^32 bytes: the last rows of the last head, appended and attended."""
    import torch

    cap = 1 << 22
    k8, v8 = (torch.zeros(2, 8, cap, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    assert k8.numel() > 2 ** 32
    ke, ve = (torch.zeros(2, 8, cap // 128, dtype=torch.int8, device="cuda") for _ in range(2))
    L, start = 200, cap - 200
    q, k, v = randn(94, 2, 32, L, 128), randn(95, 2, 8, L, 128) * 4, randn(96, 2, 8, L, 128)
    kb.append_8bit(None, k, v, k8, v8, ke, ve, None, start, check=True)
    want, want_e = plain.blocks8(np.concatenate([np.zeros((8, start % 128, 128)), f64(k[1])], 1))
    n = want.shape[1]
    # (the first block's earlier keys are zeros of exponent 0)
    assert np.array_equal(ke[1, :, -2:].cpu().numpy(), np.maximum(want_e, [[0, -100]]))
    d = kb.decode_8bit(q[:, :, -1:].contiguous(), k8, v8, ke, ve, cap, check=True)
    # keys of zero have score zero and value zero
    kk = f64(kb.cache_values(k8[1:, :, -n:].contiguous(), ke[1:, :, -2:].contiguous()))[0]
    vv = f64(kb.cache_values(v8[1:, :, -n:].contiguous(), ve[1:, :, -2:].contiguous()))[0]
    for j in range(2):
        for g in range(8):
            rows = kk[g, 128 * j:128 * j + 128]
            src = np.concatenate([np.zeros((8, start % 128, 128)), f64(k[1])], 1)[g, 128 * j:128 * j + 128]
            assert np.array_equal(rows, plain.held8(src, int(ke[1, g, j - 2])))
    for g in (0, 7):
        s = f64(q)[1, 4 * g:4 * g + 4, -1] @ kk[g].T / np.sqrt(128.0)
        w = np.exp(s)
        total = w.sum(-1) + (cap - n)
        got, exact = f64(d)[1, 4 * g:4 * g + 4, 0], (w @ vv[g]) / total[:, None]
        # outputs are small beside the largest of them; fp32 sums over 4M keys
        assert np.all(np.abs(got - exact) <= 2.0 ** -7 * (w @ np.abs(vv[g])) / total[:, None])
