"""Tensors and caches of more than 2^31 elements: rotation, append, block
selection and block-sparse attention at their far end."""

import numpy as np
import pytest

from tests import sparse_plain as plain
from tests.test_gpu_append import bits, f64, kb, randn  # noqa: F401
from tests.test_gpu_sparse import check_rows

pytestmark = pytest.mark.gpu


def test_rotation(kb):
    import torch

    S = 530_000
    x = torch.empty(1, 32, S, 128, dtype=torch.bfloat16, device="cuda").normal_()
    assert x.numel() > 2 ** 31
    table = kb.rope_table(S)
    y = kb.rope(x, table, check=True)
    for h, a in ((0, 0), (31, S - 100)):
        part = kb.rope(x[:, h:h + 1, a:a + 100], table, start=a, check=True)
        assert torch.equal(bits(y[:, h:h + 1, a:a + 100]), bits(part))


def test_a_contiguous_cache(kb):
    import torch

    cap, L = 2_200_000, 70                               # the last block has 64 rows
    nb = -(-cap // 128)
    assert 8 * cap * 128 > 2 ** 31
    kc, vc = (torch.zeros(1, 8, cap, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bx = torch.zeros(1, 8, nb, 2, 128, dtype=torch.bfloat16, device="cuda")
    for i, j in enumerate((0, 9, nb - 2)):
        kc[:, :, 128 * j:128 * j + 128], vc[:, :, 128 * j:128 * j + 128] = randn(910 + i, 1, 8, 128, 128), randn(920 + i, 1, 8, 128, 128)
    q, k, v = randn(930, 1, 32, L, 128), randn(931, 1, 8, L, 128), randn(932, 1, 8, L, 128)
    start = cap - L
    kb.block_boxes(kc, kv_len=start, boxes=bx, check=True)
    turned = kb.append(q, k, v, kc, vc, None, start, boxes=bx, check=True)
    assert torch.equal(bits(turned), bits(q))
    assert torch.equal(bits(kc[:, :, start:]), bits(k)) and torch.equal(bits(vc[:, :, start:]), bits(v))
    want = plain.boxes(f64(kc[0, :, 128 * (nb - 2):]))
    assert np.array_equal(f64(bx[0, :, nb - 2:]), want)
    # the choice of the last rows, alone and in a chunk
    n = 8
    lists = kb.select_blocks(q, bx, start, n, check=True)
    one = kb.select_blocks(q[:, :, -1:].contiguous(), bx, cap - 1, n, check=True)
    assert torch.equal(lists[:, :, -1:], one)
    for g in (0, 7):
        assert list(one[0, g, 0].cpu()) == list(plain.choose(f64(q[0, 4 * g:4 * g + 4, -1]), f64(bx[0, g]), cap - 1, n))
    # attention over four blocks, which a short cache holds one after another
    blocks = torch.tensor([0, 9, nb - 2, nb - 1], dtype=torch.int32, device="cuda").expand(1, 8, L, 4).contiguous()
    rows = torch.cat([torch.arange(128 * j, min(128 * j + 128, cap), device="cuda") for j in (0, 9, nb - 2, nb - 1)])
    small = [f64(c[0][:, rows]) for c in (kc, vc)]
    o = kb.sparse_chunk(q, kc, vc, start, blocks, check=True)
    pos = np.arange(start, cap) - 128 * (nb - 4)
    check_rows(f64(o[0]), f64(q[0]), *small, np.tile(np.arange(4), (8, L, 1)), pos)
    d = kb.sparse_decode(q[:, :, -1:].contiguous(), kc, vc, cap, blocks[:, :, -1:].contiguous(), check=True)
    assert torch.equal(bits(d), bits(o[:, :, -1:]))


def test_a_paged_cache(kb):
    import torch

    page, pages, L = 256, 8300, 300
    assert pages * 8 * page * 128 > 2 ** 31
    kp, vp = (torch.zeros(pages, 8, page, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bp = torch.zeros(pages, 8, page // 128, 2, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[8298, 3, 8299], [8297, 8296, 0]], dtype=torch.int32, device="cuda")
    cap = 3 * page
    kc, vc = (torch.zeros(2, 8, cap, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bc = torch.zeros(2, 8, cap // 128, 2, 128, dtype=torch.bfloat16, device="cuda")
    rope = kb.rope_table(cap)
    q, k, v = randn(940, 2, 32, L, 128), randn(941, 2, 8, L, 128), randn(942, 2, 8, L, 128)
    n = 3
    for step, first in enumerate((0, L)):
        starts = torch.tensor([first, first], dtype=torch.int32, device="cuda")
        lens = torch.tensor([L, L - 1], dtype=torch.int32, device="cuda") if step else torch.tensor([L, L], dtype=torch.int32, device="cuda")
        out = [torch.zeros_like(q) for _ in range(4)]
        a = kb.append_varlen(q, k, v, kp, vp, rope, starts, lens, block_table=table, boxes=bp, out=out[0], check=True)
        b = kb.append_varlen(q, k, v, kc, vc, rope, starts, lens, boxes=bc, out=out[1], check=True)
        assert torch.equal(bits(a), bits(b))
        lists = [torch.full((2, 8, L, n), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
        kb.select_blocks_varlen(a, bp, starts, n, lens, block_table=table, out=lists[0], check=True)
        kb.select_blocks_varlen(b, bc, starts, n, lens, out=lists[1], check=True)
        assert torch.equal(lists[0], lists[1])
        x = kb.sparse_chunk_varlen(a, kp, vp, starts, lists[0], lens, block_table=table, out=out[2], check=True)
        y = kb.sparse_chunk_varlen(b, kc, vc, starts, lists[1], lens, out=out[3], check=True)
        assert torch.equal(bits(x), bits(y)) and bool(x[0].any())
    ctx = torch.tensor([2 * L, 2 * L - 1], dtype=torch.int32, device="cuda")
    last = torch.stack([a[0, :, L - 1:], a[1, :, L - 2:L - 1]]).contiguous()
    chosen = torch.stack([lists[0][0, :, L - 1:], lists[0][1, :, L - 2:L - 1]]).contiguous()
    d = kb.sparse_decode_paged(last, kp, vp, table, ctx, chosen, check=True)
    assert torch.equal(bits(d[0]), bits(x[0, :, L - 1:])) and torch.equal(bits(d[1]), bits(x[1, :, L - 2:L - 1]))
