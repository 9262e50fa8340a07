"""Refusals of the 8-bit cache, key weight, eviction and several-axes entry
points, without a GPU: the shape rules of the binding and the C ABI's argument
checks; and the plain definitions the GPU tests compare with."""

import ctypes

import numpy as np
import pytest

from bitwise_aligned_causal_gb300 import shapes
from tests import cache_plain as plain

Q, K = (2, 32, 5, 128), (2, 8, 5, 128)
CACHE, POOL, TABLE, PAGES = (2, 8, 300, 128), (9, 8, 256, 128), (400, 64, 2), (2, 4)
EXP, POOL_EXP = (2, 8, 3), (9, 8, 2)


def refuse(f, *args):
    with pytest.raises(ValueError):
        f(*args)


def test_append_8bit_shapes():
    assert shapes.append_8bit(Q, K, K, CACHE, CACHE, EXP, EXP, TABLE)[:5] == (2, 32, 8, 5, 300)
    assert shapes.append_8bit(Q, K, K, POOL, POOL, POOL_EXP, POOL_EXP, TABLE, PAGES)[4:8] == (1024, 9, 256, 4)
    refuse(shapes.append_8bit, Q, K, K, CACHE, CACHE, (2, 8, 2), EXP, TABLE)
    refuse(shapes.append_8bit, Q, K, K, CACHE, CACHE, EXP, (2, 8, 300), TABLE)
    refuse(shapes.append_8bit, Q, K, K, POOL, POOL, EXP, EXP, TABLE, PAGES)
    refuse(shapes.append_8bit, Q, K, K, CACHE, (2, 8, 301, 128), EXP, EXP, TABLE)
    refuse(shapes.append_8bit, Q, K, K, (2, 8, 4, 128), (2, 8, 4, 128), (2, 8, 1), (2, 8, 1), TABLE)


def test_attend_8bit_and_values_shapes():
    assert shapes.attend_8bit(Q, CACHE, CACHE, EXP, EXP) == (2, 32, 8, 5, 300, 0, 0, 0)
    assert shapes.attend_8bit(Q, POOL, POOL, POOL_EXP, POOL_EXP, PAGES) == (2, 32, 8, 5, 1024, 9, 256, 4)
    refuse(shapes.attend_8bit, Q, CACHE, CACHE, EXP, (2, 8, 4))
    refuse(shapes.attend_8bit, (2, 32, 301, 128), CACHE, CACHE, EXP, EXP)
    refuse(shapes.attend_8bit, (1, 32, 5, 128), CACHE, CACHE, EXP, EXP)
    refuse(shapes.attend_8bit, Q, (9, 8, 200, 128), (9, 8, 200, 128), POOL_EXP, POOL_EXP, PAGES)
    assert shapes.cache_values(CACHE, EXP) == (2, 8, 300)
    refuse(shapes.cache_values, CACHE, (2, 8, 2))
    refuse(shapes.cache_values, CACHE, EXP, POOL)


def test_weights_and_evict_shapes():
    assert shapes.chunk_lse(Q, CACHE, CACHE, None, Q, (2, 32, 5))[3:5] == (5, 300)
    refuse(shapes.chunk_lse, Q, CACHE, CACHE, None, Q, (2, 32, 6))
    assert shapes.key_weights(Q, CACHE, (2, 32, 5), (2, 8, 300))[:5] == (2, 32, 8, 5, 300)
    assert shapes.key_weights(Q, POOL, (2, 32, 5), (2, 8, 1024), PAGES)[4:] == (1024, 9, 256, 4)
    refuse(shapes.key_weights, Q, CACHE, (2, 32, 4), (2, 8, 300))
    refuse(shapes.key_weights, Q, CACHE, (2, 32, 5), (2, 8, 299))
    refuse(shapes.key_weights, Q, POOL, (2, 32, 5), (2, 8, 256), PAGES)
    ok = (CACHE, CACHE, (2, 8, 300), (2,))
    assert shapes.evict(*ok, 100, 4, 64) == (2, 8, 300, 0, 0, 0)
    assert shapes.evict(POOL, POOL, (2, 8, 1024), (2,), 100, 100, 0, PAGES) == (2, 8, 1024, 9, 256, 4)
    for keep, first, last in ((0, 0, 0), (301, 0, 0), (100, 60, 41), (100, -1, 5), (100, 5, -1)):
        refuse(shapes.evict, *ok, keep, first, last)
    refuse(shapes.evict, CACHE, POOL, (2, 8, 300), (2,), 100, 0, 0)
    refuse(shapes.evict, CACHE, CACHE, (2, 8, 301), (2,), 100, 0, 0)
    refuse(shapes.evict, CACHE, CACHE, (2, 8, 300), (3,), 100, 0, 0)
    refuse(shapes.evict, *ok, 100, 0, 0, None, (2, 8, 299))
    refuse(shapes.evict, *ok, 100, 0, 0, None, None, (2, 8, 99))


def test_rope_axes_shapes():
    planes = [0] * 16 + [1] * 24 + [2] * 24
    assert shapes.rope_axes(Q, TABLE, (3, 2, 5), planes) == (2, 32, 5, 400, 128, 3)
    refuse(shapes.rope_axes, Q, TABLE, (2, 2, 5), planes)                 # an axis without positions
    refuse(shapes.rope_axes, Q, TABLE, (5, 2, 5), planes)                 # too many axes
    refuse(shapes.rope_axes, Q, TABLE, (3, 2, 6), planes)
    refuse(shapes.rope_axes, Q, TABLE, (2, 5), planes)
    refuse(shapes.rope_axes, Q, TABLE, (3, 2, 5), planes[:-1])
    refuse(shapes.rope_axes, Q, TABLE, (3, 2, 5), [-1] + planes[1:])
    refuse(shapes.rope_axes, Q, TABLE, (3, 2, 5), planes, K)


FAKE = 0x1000_0000      # aligned, non-null; the checks below fail before any CUDA call


@pytest.fixture(scope="module")
def kb():
    from bitwise_aligned_causal_gb300 import build

    build.build()
    from bitwise_aligned_causal_gb300 import kb_attn

    return kb_attn


def strides(*x):
    return (ctypes.c_longlong * len(x))(*x)


def changed(args, **new):
    a = dict(args, **new)
    return list(a.values())


def test_rope_axes_abi(kb):
    ok = dict(x=FAKE, strides=strides(128, 128, 128), out=FAKE, table=FAKE, n_pos=100, rot_dim=128, interleaved=0, inverse=0,
              positions=FAKE, n_axes=2, planes=bytes([0, 1] * 32), B=1, H=8, L=4)
    for new in (dict(x=None), dict(out=FAKE + 8), dict(positions=None), dict(positions=FAKE + 2), dict(n_axes=0),
                dict(planes=bytes([0, 2] * 32)), dict(planes=None), dict(strides=strides(128, 128, 12)), dict(L=0), dict(n_pos=0)):
        assert kb.kb_attn_rope_axes(*changed(ok, **new)) == kb.KB_ERR_INVALID_ARG, new
    for new in (dict(n_axes=5), dict(rot_dim=72)):
        assert kb.kb_attn_rope_axes(*changed(ok, **new)) == kb.KB_ERR_UNSUPPORTED, new


def test_append_8bit_abi(kb):
    ok = dict(q=FAKE, k=FAKE, v=FAKE, strides=strides(*[128] * 9), q_out=FAKE, kc=FAKE, vc=FAKE, ke=FAKE, ve=FAKE, table=FAKE,
              n_pos=100, rot_dim=128, interleaved=0, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None, lens=None, cap=100,
              bt=None, pps=0, page=0, pages=0)
    for new in (dict(k=None), dict(ke=None), dict(q=None), dict(kc=FAKE + 4), dict(strides=strides(*[128] * 8, 4)), dict(L=101),
                dict(start=97), dict(start=-1), dict(n_pos=3), dict(lens=FAKE), dict(cap=0), dict(B=0)):
        assert kb.kb_attn_append_8bit(*changed(ok, **new)) == kb.KB_ERR_INVALID_ARG, new
    for new in (dict(Hkv=4), dict(cap=1 << 23), dict(bt=FAKE, pps=2, page=200, pages=3)):
        assert kb.kb_attn_append_8bit(*changed(ok, **new)) == kb.KB_ERR_UNSUPPORTED, new


def test_attend_8bit_abi(kb):
    ok = dict(q=FAKE, k=FAKE, v=FAKE, ke=FAKE, ve=FAKE, o=FAKE, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None, lens=None, cap=100,
              bt=None, pps=0, page=0, pages=0, ws=None, nbytes=0)
    for new in (dict(v=None), dict(ve=None), dict(o=FAKE + 8), dict(starts=FAKE), dict(lens=FAKE), dict(start=97), dict(L=0), dict(L=101)):
        assert kb.kb_attn_chunk_8bit(*changed(ok, **new)) == kb.KB_ERR_INVALID_ARG, new
    assert kb.kb_attn_chunk_8bit(*changed(ok, Hq=8)) == kb.KB_ERR_UNSUPPORTED
    dec = dict(q=FAKE, k=FAKE, v=FAKE, ke=FAKE, ve=FAKE, o=FAKE, B=1, Hq=32, Hkv=8, ctx=4, lens=None, cap=100, bt=None, pps=0, page=0,
               pages=0, ws=None, nbytes=0)
    for new in (dict(ctx=0), dict(ctx=101), dict(ke=None), dict(lens=FAKE + 1)):
        assert kb.kb_attn_decode_8bit(*changed(dec, **new)) == kb.KB_ERR_INVALID_ARG, new
    assert kb.kb_attn_chunk_8bit_workspace_bytes(1, 8, 32, 1000) == 0                # one segment: nothing to share
    assert kb.kb_attn_chunk_8bit_workspace_bytes(3, 8, 5, 2049) == 3 * 32 * 5 * 3 * 528
    assert kb.kb_attn_chunk_8bit_workspace_bytes(64, 8, 1, 100000) == 0              # enough KV heads for every SM
    assert kb.kb_attn_chunk_8bit_workspace_bytes(30, 8, 32, 1 << 22) == 0            # too large
    assert kb.kb_attn_chunk_8bit_workspace_bytes(2, 8, 33, 1000) == 2 * 2 * 8 * 1000 * 256
    assert kb.kb_attn_chunk_8bit_workspace_bytes(1, 8, 33, 32) == 0
    val = (FAKE, FAKE, FAKE, 8, 100)
    for a in ((None, *val[1:]), (FAKE + 8, *val[1:]), (*val[:3], 0, 100), (*val[:4], 0)):
        assert kb.kb_attn_cache_values(*a) == kb.KB_ERR_INVALID_ARG
    assert kb.kb_attn_cache_values(FAKE, FAKE, FAKE, 1 << 30, 1 << 20) == kb.KB_ERR_UNSUPPORTED


def test_weights_and_evict_abi(kb):
    lse = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None, lens=None, cap=100, bt=None,
               pps=0, page=0, pages=0)
    for new in (dict(lse=None), dict(lse=FAKE + 1), dict(starts=FAKE), dict(start=97), dict(L=101), dict(q=None)):
        assert kb.kb_attn_chunk_lse(*changed(lse, **new)) == kb.KB_ERR_INVALID_ARG, new
    wts = dict(q=FAKE, k=FAKE, lse=FAKE, weights=FAKE, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None, lens=None, cap=100, bt=None,
               pps=0, page=0, pages=0)
    for new in (dict(weights=None), dict(lse=FAKE + 2), dict(k=FAKE + 8), dict(lens=FAKE), dict(start=97), dict(L=0)):
        assert kb.kb_attn_key_weights(*changed(wts, **new)) == kb.KB_ERR_INVALID_ARG, new
    assert kb.kb_attn_key_weights(*changed(wts, Hq=16)) == kb.KB_ERR_UNSUPPORTED
    ev = dict(k=FAKE, v=FAKE, w=FAKE, wo=FAKE, kept=FAKE, B=1, Hkv=8, lens=FAKE, keep=10, first=4, last=6, cap=100, bt=None, pps=0,
              page=0, pages=0)
    for new in (dict(lens=None), dict(kept=None), dict(keep=0), dict(keep=101), dict(first=5), dict(last=-1), dict(k=FAKE + 8),
                dict(B=0)):
        assert kb.kb_attn_evict(*changed(ev, **new)) == kb.KB_ERR_INVALID_ARG, new
    assert kb.kb_attn_evict(*changed(ev, bt=FAKE, pps=1, page=100, pages=2)) in (kb.KB_ERR_INVALID_ARG, kb.KB_ERR_UNSUPPORTED)


def test_plain_8_bits_are_the_format():
    """The plain form's values are e4m3 numbers (without subnormals) times the scale, and rounding again changes nothing."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 300, 128)) * np.exp(rng.standard_normal((2, 300, 1)) * 3)
    y, e = plain.blocks8(x)
    for h in range(2):
        for j in range(3):
            part, src = y[h, 128 * j:128 * j + 128], x[h, 128 * j:128 * j + 128]
            step = part / 2.0 ** e[h, j]
            assert np.abs(step).max() <= 448 and np.abs(src).max() > 224 * 2.0 ** e[h, j]
            m, _ = np.frexp(step)
            assert np.array_equal(m * 16, np.rint(m * 16))
            assert np.abs(step[step != 0]).min() >= 2.0 ** -6
            # four bits: half a step of 2^-4; what is zero was below the smallest number
            assert np.all(np.abs(part - src) <= np.maximum(2.0 ** -4 * np.abs(src), (part == 0) * 2.0 ** (e[h, j] - 6)))
            # keys that came while the block's exponent was three lower (those that fit there) end as the same values
            fit = np.abs(src).max(1) <= 448 * 2.0 ** (e[h, j] - 3)
            assert fit.any() and np.array_equal(plain.held8(plain.held8(src[fit], e[h, j] - 3), e[h, j]), part[fit])
    assert [plain.exponent8(a) for a in (0, 448, 448.01, 1e-40, 1e38, np.inf)] == [-100, 0, 1, -100, 100, 127]
