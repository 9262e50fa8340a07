"""Eviction of a cache's lightest keys against its plain definition, exactly."""

import numpy as np
import pytest

from tests import cache_plain as plain
from tests.test_gpu_append import bits, caches, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(*x):
    import torch

    return torch.tensor(x, dtype=torch.int32, device="cuda")


def weights_of(kind, B, cap, seed=5):
    import torch

    g = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.randn(B, 8, cap, generator=g) * 3)
    if kind == "ties":
        w = torch.randint(0, 4, (B, 8, cap), generator=g).float()
    elif kind == "equal":
        w = torch.full((B, 8, cap), 0.25)
    elif kind == "odd":                                           # what sums can come to, and what they cannot
        odd = torch.tensor([0.0, -0.0, float("inf"), float("nan"), -1.0, float("-inf"), 1e-45, -1e-45, 3.4e38])
        pick = torch.randint(0, 30, (B, 8, cap), generator=g)
        w = torch.where(pick < 9, odd[pick.clamp(max=8)], w)
    return w.cuda()


def run_and_check(kb, k, v, w, lens, keep, first, last, pages, seq, in_place=True):
    import torch

    B, cap = w.shape[0], w.shape[2]
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    w_out = w if in_place else torch.full_like(w, 5.0)
    kept = kb.evict(k, v, w, i32(*lens), keep, keep_first=first, keep_last=last, block_table=pages, weights_out=None if in_place else w_out,
                    check=True)
    assert tuple(kept.shape) == (B, 8, keep) and kept.dtype == torch.int32
    if not in_place:
        assert torch.equal(w.view(torch.int32), w0.view(torch.int32))
    host_w, host_kept = w0.cpu().numpy(), kept.cpu().numpy()
    for b in range(B):
        n = lens[b]
        m = min(n, keep)
        for g in range(8):
            want = plain.evict(host_w[b, g], n, keep, first, last)
            assert np.array_equal(host_kept[b, g, :m], want), (b, g)
            assert np.all(host_kept[b, g, m:] == -1)
            at = torch.from_numpy(want).cuda()
            for x, x0 in ((k, k0), (v, v0)):
                new, old = seq(x, b)[g], seq(x0, b)[g]
                assert torch.equal(bits(new[:m]), bits(old[at]))
                assert torch.equal(bits(new[m:]), bits(old[m:]))  # rows behind are as they were
            assert torch.equal(w_out[b, g, :m].view(torch.int32), w0[b, g][at].view(torch.int32))
            assert bool((w_out[b, g, m:].view(torch.int32) == 0).all())
    if pages is not None:
        free = sorted(set(range(k.shape[0])) - set(pages.view(-1).tolist()))
        assert torch.equal(bits(k[free]), bits(k0[free])) and torch.equal(bits(v[free]), bits(v0[free]))


@pytest.mark.parametrize("page", [0, 128, 384])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,keep,first,last", [((1152, 700, 0), 300, 4, 64), ((1151, 300, 301), 300, 0, 0), ((1, 500, 129), 128, 100, 28),
                                                  ((1152, 1000, 900), 899, 1, 0), ((640, 3, 1152), 1, 0, 1)])
def test_definition(kb, page, kind, lens, keep, first, last):
    B, cap = 3, 1152
    k, v, _, pages, seq = caches(B, cap, page, seed=20)
    run_and_check(kb, k, v, weights_of(kind, B, cap), lens, keep, first, last, pages, seq, in_place=kind != "ties")


@pytest.mark.parametrize("B,cap,keep", [(1, 20000, 2500), (1, 70001, 69000), (24, 300, 37)])
def test_sizes(kb, B, cap, keep):
    k, v, _, pages, seq = caches(B, cap, seed=30)
    run_and_check(kb, k, v, weights_of("spread", B, cap), [cap - b for b in range(B)], keep, 4, min(64, keep // 2), pages, seq)


@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 6, 8, 13, 40])
def test_any_number_of_planes(kb, page, B):
    """As many CTAs share a plane's rows as find a place: keeps that end inside and on the ends of their tiles."""
    cap = 1536
    for keep in (127, 1024, 1300):
        k, v, _, pages, seq = caches(B, cap, page, seed=50)
        run_and_check(kb, k, v, weights_of("ties", B, cap, seed=keep), [cap - 7 * (b % 20) for b in range(B)], keep, 4, 64, pages, seq)


def test_two_streams_at_once(kb):
    import torch

    cap, keep = 5000, 1700
    k, v, _, _, _ = caches(2, cap, seed=55)
    w = weights_of("spread", 2, cap)
    n = i32(cap, cap - 11)
    want = [t.clone() for t in (k, v, w)]
    kept = kb.evict(*want, n, keep, check=True)
    sets = [[t.clone() for t in (k, v, w)] for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [kb.evict(*x, n, keep, stream=streams[i % 3]) for i, x in enumerate(sets)]
    torch.cuda.synchronize()
    kb.check_device_status()
    for x, r in zip(sets, got):
        assert torch.equal(r, kept) and all(torch.equal(a, b) for a, b in zip(x, want))


def test_the_whole_cache_may_stay(kb):
    k, v, _, pages, seq = caches(2, 200, seed=40)
    run_and_check(kb, k, v, weights_of("odd", 2, 200), (200, 77), 200, 0, 200, pages, seq)


def test_bad_device_arguments_move_nothing(kb):
    import torch

    k, v, _, pages, _ = caches(2, 512, 128, seed=50)
    w = weights_of("spread", 2, 512)
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    for lens in (i32(-1, -5), i32(513, 600)):
        with pytest.raises(kb.KBError):
            kb.evict(k, v, w, lens, 100, block_table=pages, check=True)
    for bad in (-1, 10, 2 ** 31 - 1):
        broken = pages.clone()
        broken[:, 2] = bad
        with pytest.raises(kb.KBError):
            kb.evict(k, v, w, i32(400, 300), 100, block_table=broken, check=True)
    assert torch.equal(bits(k), bits(k0)) and torch.equal(bits(v), bits(v0)) and torch.equal(w, w0)
    # a page beyond the sequences' keys is never looked up
    broken = pages.clone()
    broken[:, 3] = -1
    kb.evict(k, v, w, i32(384, 300), 100, block_table=broken, check=True)


def test_refusals(kb):
    import torch

    k, v, _, _, _ = caches(1, 100, seed=60)
    w, n = torch.zeros(1, 8, 100, device="cuda"), i32(100)
    for args in ((k.float(), v, w, n, 50), (k, v, w.double(), n, 50), (k, v, w, n.long(), 50), (k, v, w, n.cpu(), 50)):
        with pytest.raises(TypeError):
            kb.evict(*args)
    with pytest.raises(kb.KBError):                               # one plane cannot be moved as two
        kb.evict(k, k, w, n, 90)
    for args in ((k, v, w, n, 0), (k, v, w, n, 101), (k, v, w, n, 50, 30, 30), (k, v[:, :, :99].contiguous(), w, n, 50)):
        with pytest.raises(ValueError):
            kb.evict(*args)


def test_captured_and_replayed(kb):
    import torch

    cap, keep = 700, 200
    k, v, _, _, _ = caches(1, cap, seed=70)
    w = weights_of("spread", 1, cap)
    n = i32(600)
    want = [t.clone() for t in (k, v, w)]
    kept = kb.evict(*want, n, keep, check=True)
    got = [torch.empty_like(t) for t in (k, v, w)]
    out = torch.empty_like(kept)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        kb.evict(*got, n, keep, kept=out)
    for _ in range(2):
        for a, b in zip(got, (k, v, w)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        kb.check_device_status()
        assert torch.equal(out, kept)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_far_rows(kb):
    """Caches beyond 2^32 bytes, the kept keys at their far end."""
    import torch

    cap, keep = 2_200_000, 1000
    k, v = (torch.zeros(1, 8, cap, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    k[:, :, -900:], v[:, :, -900:] = randn(80, 1, 8, 900, 128), randn(81, 1, 8, 900, 128)
    tail = [t[:, :, -900:].clone() for t in (k, v)]
    w = torch.zeros(1, 8, cap, device="cuda")
    w[:, :, -900:] = 1.0
    kept = kb.evict(k, v, w, i32(cap), keep, keep_first=10, keep_last=5, check=True)
    assert torch.equal(kept[0, 3, 100:].cpu(), torch.arange(cap - 900, cap, dtype=torch.int32))
    assert torch.equal(kept[0, 7, :100].cpu(), torch.arange(100, dtype=torch.int32))
    for t, x in zip((k, v), tail):
        assert torch.equal(bits(t[:, :, 100:1000]), bits(x))
