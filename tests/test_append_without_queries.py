"""Appends without queries look at no strides of queries: their three places may hold anything."""

import pytest

from tests.test_cache_shapes import FAKE, changed, kb, strides  # noqa: F401

PLAIN = dict(q=None, k=FAKE, v=FAKE, strides=None, q_out=None, kc=FAKE, vc=FAKE, boxes=None, table=FAKE, n_pos=100, rot_dim=128,
             interleaved=0, B=1, Hq=32, Hkv=8, L=4, start=0, starts=None, lens=None, cap=100, bt=None, pps=0, page=0, pages=0)
EIGHT = {x: y for a, b in PLAIN.items() for x, y in ([("ke", FAKE), ("ve", FAKE)] if a == "boxes" else [(a, b)])}


@pytest.mark.parametrize("name,args", [("kb_attn_append", PLAIN), ("kb_attn_append_8bit", EIGHT)])
@pytest.mark.parametrize("of_q", [(0, 0, 0), (-1, 128, 128), (128, 3, 128), (2 ** 62 + 1, -2 ** 62, 7)])
def test_strides_of_no_queries(kb, name, args, of_q):
    call = getattr(kb, name)
    want = call(*changed(args, strides=strides(*[128] * 9)))         # (what comes after the host's checks)
    assert call(*changed(args, strides=strides(*of_q, *[128] * 6))) == want
    for of_k in ((-8, 128, 128), (128, 128, 12)):
        assert call(*changed(args, strides=strides(*of_q, *of_k, *[128] * 3))) == kb.KB_ERR_INVALID_ARG
        assert call(*changed(args, strides=strides(*of_q, *[128] * 3, *of_k))) == kb.KB_ERR_INVALID_ARG
    for q in (dict(q=FAKE), dict(q_out=FAKE)):
        assert call(*changed(args, strides=strides(*[128] * 9), **q)) == kb.KB_ERR_INVALID_ARG
