"""Refusals of the rotation, append and selection entry points, without a GPU:
the shape rules of the binding and the C ABI's argument checks."""

import ctypes

import pytest

from bitwise_aligned_causal_gb300 import shapes

Q, K = (2, 32, 5, 128), (2, 8, 5, 128)
CACHE, POOL, TABLE = (2, 8, 300, 128), (9, 8, 256, 128), (400, 64, 2)


def test_append_shapes():
    assert shapes.append(Q, K, K, CACHE, CACHE, TABLE)[:5] == (2, 32, 8, 5, 300)
    assert shapes.append(None, K, K, CACHE, CACHE, None, (2, 8, 3, 2, 128))[4] == 300
    assert shapes.append(Q, K, K, POOL, POOL, TABLE, (9, 8, 2, 2, 128), (2, 4))[4:8] == (1024, 9, 256, 4)


@pytest.mark.parametrize("args", [
    (Q, K, (2, 8, 6, 128), CACHE, CACHE, TABLE),                         # v differs from k
    (Q, (2, 4, 5, 128), (2, 4, 5, 128), CACHE, CACHE, TABLE),            # KV heads differ from the cache's
    ((2, 32, 6, 128), K, K, CACHE, CACHE, TABLE),                        # q of other rows
    ((2, 16, 5, 128), K, K, CACHE, CACHE, TABLE),                        # q heads
    (Q, K, K, (1, 8, 300, 128), (1, 8, 300, 128), TABLE),                # batch
    (Q, K, K, CACHE, (2, 8, 301, 128), TABLE),                           # caches differ
    (Q, K, K, (2, 8, 4, 128), (2, 8, 4, 128), TABLE),                    # more rows than the cache
    (Q, K, K, CACHE, CACHE, (400, 64)),                                  # table
    (Q, K, K, CACHE, CACHE, (400, 60, 2)),                               # rot_dim no multiple of 16
    (Q, K, K, CACHE, CACHE, (400, 72, 2)),                               # rot_dim above 128
    (Q, K, K, CACHE, CACHE, TABLE, (2, 8, 2, 2, 128)),                   # boxes of fewer blocks
    (Q, K, K, POOL, POOL, TABLE, (9, 8, 3, 2, 128), (2, 4)),             # boxes of another page size
    (Q, K, K, (9, 8, 200, 128), (9, 8, 200, 128), TABLE, None, (2, 4)),  # page size
    (None, K, K, CACHE, CACHE, TABLE, None, None, Q),                    # out without q
])
def test_append_refuses(args):
    with pytest.raises(ValueError):
        shapes.append(*args)


def test_select_and_rope_refuse():
    bx = (2, 8, 10, 2, 128)
    assert shapes.select(Q, bx, 4, 1, 1) == (2, 32, 8, 5, 10, 0, 0, 0)
    assert shapes.select(Q, (7, 8, 2, 2, 128), 4, 1, 1, (2, 3)) == (2, 32, 8, 5, 2, 7, 256, 3)
    for a in [(Q, bx, 0, 0, 1), (Q, bx, 129, 1, 1), (Q, bx, 4, 4, 1), (Q, bx, 4, 1, 0), (Q, bx, 4, -1, 1),
              (Q, (1, 8, 10, 2, 128), 4, 1, 1), (Q, (2, 8, 10, 128), 4, 1, 1), (Q, bx, 4, 1, 1, (3, 3)),
              (Q, bx, 4, 1, 1, None, (2, 8, 5, 5))]:
        with pytest.raises(ValueError):
            shapes.select(*a)
    assert shapes.rope(Q, TABLE, 395)[3:] == (400, 128)
    for a in [(Q, TABLE, 396), (Q, TABLE, -1), ((2, 32, 5, 64), TABLE, 0), (Q, TABLE, 0, K)]:
        with pytest.raises(ValueError):
            shapes.rope(*a)
    with pytest.raises(ValueError):
        shapes.per_sequence(3, starts=(2,))


FAKE = 0x1000_0000      # aligned, non-null; the checks below fail before any CUDA call


@pytest.fixture(scope="module")
def kb():
    from bitwise_aligned_causal_gb300 import build

    build.build()
    from bitwise_aligned_causal_gb300 import kb_attn

    return kb_attn


def strides(*x):
    return (ctypes.c_longlong * len(x))(*x)


def test_rope_abi(kb):
    st = strides(1024, 128, 1024)
    ok = (1, 8, 16, 0)
    f = kb.kb_attn_rope
    assert f(None, st, FAKE, FAKE, 64, 128, 0, 0, *ok) == kb.KB_ERR_INVALID_ARG
    assert f(FAKE, None, FAKE, FAKE, 64, 128, 0, 0, *ok) == kb.KB_ERR_INVALID_ARG
    assert f(FAKE + 8, st, FAKE, FAKE, 64, 128, 0, 0, *ok) == kb.KB_ERR_INVALID_ARG
    assert f(FAKE, strides(1024, 129, 1024), FAKE, FAKE, 64, 128, 0, 0, *ok) == kb.KB_ERR_INVALID_ARG
    assert f(FAKE, st, FAKE, FAKE, 64, 24, 0, 0, *ok) == kb.KB_ERR_UNSUPPORTED
    assert f(FAKE, st, FAKE, FAKE, 64, 144, 0, 0, *ok) == kb.KB_ERR_UNSUPPORTED
    assert f(FAKE, st, FAKE, FAKE, 15, 128, 0, 0, *ok) == kb.KB_ERR_INVALID_ARG       # positions past the table
    assert f(FAKE, st, FAKE, FAKE, 64, 128, 0, 0, 1, 8, 16, -1) == kb.KB_ERR_INVALID_ARG
    assert f(FAKE, st, FAKE, FAKE, 64, 128, 0, 0, 1, 0, 16, 0) == kb.KB_ERR_INVALID_ARG
    assert kb.kb_attn_rope_table(FAKE, 0, 128, FAKE) == kb.KB_ERR_INVALID_ARG
    assert kb.kb_attn_rope_table(FAKE, 8, 128, None) == kb.KB_ERR_INVALID_ARG
    assert kb.kb_attn_rope_table(FAKE, 1 << 23, 128, FAKE) == kb.KB_ERR_UNSUPPORTED


def test_append_abi(kb):
    st = strides(*([1024, 128, 1024] * 3))

    def f(q=FAKE, k=FAKE, out=FAKE, boxes=FAKE, table=FAKE, n_pos=64, rot=128, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None,
          lens=None, cap=64, bt=None, pps=0, page=0, pages=0, s=st):
        return kb.kb_attn_append(q, k, FAKE, s, out, FAKE, FAKE, boxes, table, n_pos, rot, 0, B, Hq, Hkv, L, start, starts,
                                 lens, cap, bt, pps, page, pages)

    bad = kb.KB_ERR_INVALID_ARG
    assert f(k=None) == bad and f(q=None) == bad and f(out=None) == bad and f(s=None) == bad
    assert f(boxes=FAKE + 8) == bad and f(starts=FAKE + 2) == bad and f(lens=FAKE) == bad
    assert f(start=61) == bad and f(start=-1) == bad and f(L=0) == bad and f(L=65) == bad and f(cap=0) == bad
    assert f(n_pos=3) == bad and f(s=strides(*([1024, 128, 4] * 3))) == bad
    assert f(Hq=8) == kb.KB_ERR_UNSUPPORTED and f(rot=8) == kb.KB_ERR_UNSUPPORTED and f(cap=1 << 23) == kb.KB_ERR_UNSUPPORTED
    assert f(bt=FAKE, pps=2, page=192, pages=4) == kb.KB_ERR_UNSUPPORTED
    assert f(bt=FAKE, pps=0, page=128, pages=4) == bad


def test_boxes_and_select_abi(kb):
    bad = kb.KB_ERR_INVALID_ARG
    b = kb.kb_attn_block_boxes
    assert b(None, FAKE, 1, 8, 10, None, 20, None, 0, 0, 0) == bad
    assert b(FAKE, FAKE, 1, 8, 21, None, 20, None, 0, 0, 0) == bad
    assert b(FAKE, FAKE, 1, 8, 0, None, 20, None, 0, 0, 0) == bad
    assert b(FAKE, FAKE, 1, 8, 10, FAKE + 1, 20, None, 0, 0, 0) == bad

    def s(q=FAKE, Hq=32, L=4, n=4, kf=1, kl=1, start=0, starts=None, lens=None, nb=2, bt=None, pps=0, page=0, pages=0):
        return kb.kb_attn_select_blocks(q, FAKE, FAKE, 1, Hq, 8, L, n, kf, kl, start, starts, lens, nb, bt, pps, page, pages)

    assert s(q=None) == bad and s(n=0) == bad and s(kf=-1) == bad and s(kl=0) == bad and s(kf=4) == bad
    assert s(n=129) == kb.KB_ERR_UNSUPPORTED and s(Hq=16) == kb.KB_ERR_UNSUPPORTED
    assert s(start=253) == bad and s(start=-1) == bad and s(nb=0) == bad and s(L=257) == bad and s(lens=FAKE) == bad
    assert s(nb=40_000) == kb.KB_ERR_UNSUPPORTED
    assert s(bt=FAKE, pps=2, page=100, pages=4) == bad


def test_sparse_shapes_and_abi(kb):
    blocks = (2, 8, 5, 3)
    assert shapes.sparse(Q, CACHE, CACHE, blocks) == (2, 32, 8, 5, 3, 300, 0, 0, 0)
    assert shapes.sparse(Q, POOL, POOL, blocks, (2, 4))[5:] == (1024, 9, 256, 4)
    for a in [(Q, CACHE, CACHE, (2, 8, 5, 129)), (Q, CACHE, CACHE, (2, 4, 5, 3)), (Q, CACHE, CACHE, (2, 8, 5)),
              (Q, CACHE, (2, 8, 301, 128), blocks), (Q, POOL, POOL, blocks, (3, 4))]:
        with pytest.raises(ValueError):
            shapes.sparse(*a)
    bad, ws = kb.KB_ERR_INVALID_ARG, kb.kb_attn_sparse_workspace_bytes(1, 8, 64, 4, 256)
    assert ws == 256 + 8 * 3 * 2 * 8                                # three position tiles, two blocks at most
    assert kb.kb_attn_sparse_workspace_bytes(1, 8, 64, 129, 256) == 0
    assert kb.kb_attn_sparse_backward_workspace_bytes(1, 8, 64, 4) > kb.kb_attn_sparse_workspace_bytes(1, 8, 64, 4, 64)

    def chunk(q=FAKE, blocks=FAKE, n=4, Hq=32, L=64, start=0, starts=None, lens=None, cap=256, bt=None, pps=0, page=0,
              pages=0):
        return kb.kb_attn_sparse_chunk(q, FAKE, FAKE, FAKE, blocks, n, 1, Hq, 8, L, start, starts, lens, cap, bt, pps, page,
                                       pages, FAKE, ws)

    assert chunk(q=None) == bad and chunk(blocks=None) == bad and chunk(blocks=FAKE + 2) == bad and chunk(n=0) == bad
    assert chunk(n=129) == kb.KB_ERR_UNSUPPORTED and chunk(Hq=8) == kb.KB_ERR_UNSUPPORTED
    assert chunk(start=193) == bad and chunk(start=-1) == bad and chunk(L=0) == bad and chunk(lens=FAKE) == bad
    assert chunk(cap=1 << 23) == kb.KB_ERR_UNSUPPORTED and chunk(bt=FAKE, pps=2, page=64, pages=4) == bad

    def decode(q=FAKE, n=4, ctx=10, lens=None, cap=256):
        return kb.kb_attn_sparse_decode(q, FAKE, FAKE, FAKE, FAKE, n, 1, 32, 8, ctx, lens, cap, None, 0, 0, 0)

    assert decode(q=None) == bad and decode(ctx=0) == bad and decode(ctx=257) == bad and decode(n=0) == bad
    assert decode(lens=FAKE + 2) == bad
    fwd = (FAKE,) * 4
    assert kb.kb_attn_sparse_prefill_lse(*fwd, None, FAKE, 4, 1, 32, 8, 64, FAKE, ws) == bad
    assert kb.kb_attn_sparse_prefill_lse(*fwd, FAKE, FAKE, 4, 1, 32, 8, 0, FAKE, ws) == bad
    bwd = (FAKE,) * 8
    assert kb.kb_attn_sparse_backward(*bwd, 4, FAKE, None, FAKE, 1, 32, 8, 64, FAKE, ws) == bad
    assert kb.kb_attn_sparse_backward(*bwd, 4, FAKE + 8, FAKE, FAKE, 1, 32, 8, 64, FAKE, ws) == bad
    assert kb.kb_attn_sparse_backward(*bwd, 4, FAKE, FAKE, FAKE, 1, 32, 4, 64, FAKE, ws) == kb.KB_ERR_UNSUPPORTED
