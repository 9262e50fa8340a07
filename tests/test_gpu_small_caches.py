"""The operators that make a cache smaller, together as a serving loop uses
them."""

import numpy as np
import pytest

from tests import cache_plain as plain
from tests.test_gpu_append import bits, caches, f64, kb, randn  # noqa: F401
from tests.test_gpu_cache8 import empty8

pytestmark = pytest.mark.gpu

SECTIONS = [0] * 16 + [1] * 24 + [2] * 24


@pytest.mark.parametrize("page", [0, 128])
def test_a_cache_that_evicts_as_it_grows(kb, page):
    """A prompt whose weights are summed, an eviction, tokens at rows behind with their true positions, another eviction:
    the last token's output is the attention over the keys that 64-bit bookkeeping keeps."""
    import torch

    B, cap, S, keep, first, last = 2, 768, 500, 256, 4, 16
    table = kb.rope_table(2000)
    kc, vc, _, pages, seq = caches(B, cap, page, seed=1)
    weights = torch.zeros(B, 8, cap, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(q, k, v, starts, lens, positions):
        """Rotate at `positions` [B, L], append at rows starts.., attend and add weights."""
        turned_q = kb.rope_axes(q, table, positions[None].contiguous(), [0] * 64)
        turned_k = kb.rope_axes(k, table, positions[None].contiguous(), [0] * 64)
        kb.append_varlen(turned_q, turned_k, v, kc, vc, None, starts, lens, block_table=pages)
        o, lse = kb.chunk_lse_varlen(turned_q, kc, vc, starts, lens, block_table=pages)
        kb.key_weights_varlen(turned_q, kc, lse, weights, starts, lens, block_table=pages)
        return o, turned_q

    L = [S, S - 77]
    q, k, v = (randn(10 + i, B, h, S, 128) for i, h in enumerate((32, 8, 8)))
    pos = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, S)
    step(q, k, v, i32(0, 0), i32(*L), pos)
    rows, at = i32(*L), i32(*L)                                   # rows in use; the next position
    for n in range(60):
        if n in (0, 40):
            kb.evict(kc, vc, weights, rows, keep, keep_first=first, keep_last=last, block_table=pages)
            rows = rows.clamp(max=keep)
        q, k, v = (randn(1000 + 3 * n + i, B, h, 1, 128) for i, h in enumerate((32, 8, 8)))
        before = weights.clone()
        o, turned_q = step(q, k, v, rows, i32(1, 1), at[:, None])
        rows, at = rows + 1, at + 1
        gained = (weights.double() - before.double()).sum(-1)
        assert torch.all((gained - 4).abs() < 1e-3)               # one token gives each group its four heads' weight
    kb.check_device_status()
    assert rows.tolist() == [276, 276]
    for b in range(B):
        n = int(rows[b])
        for g in range(8):
            want, _, mag = plain.attend(f64(turned_q)[b, 4 * g:4 * g + 4], f64(seq(kc, b)[g, :n]), f64(seq(vc, b)[g, :n]), np.array([n - 1]))
            assert np.all(np.abs(f64(o)[b, 4 * g:4 * g + 4] - want) <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * np.abs(want))
        # heads keep keys of their own, but all keep the first ones and the newest: row 275 is the last token's
        assert torch.equal(bits(seq(vc, b)[:, n - 1]), bits(v[b, :, 0]))


@pytest.mark.parametrize("page", [0, 256])
def test_a_prompt_of_patches_and_its_tokens_in_8_bits(kb, page):
    """Positions of three axes, an 8-bit cache, a prompt in two chunks, then tokens: every output has the bits of the
    bf16 attention over what the cache stands for, and the log-sum-exp path sees the same cache."""
    import torch

    B, cap, S = 1, 768, 600
    table = kb.rope_table(400)
    k8, v8, ke, ve, pages, seq = empty8(B, cap, page)
    i = torch.arange(S + 20, device="cuda")
    pos = torch.stack([i // 64, i // 8 % 8, i % 8]).to(torch.int32)[:, None]
    q, k, v = (randn(20 + n, B, h, S + 20, 128) for n, h in enumerate((32, 8, 8)))
    q, k = kb.rope_axes(q, table, pos, SECTIONS), kb.rope_axes(k, table, pos, SECTIONS)
    at = 0
    for L in (450, 150, *([1] * 20)):
        st, ln = (torch.full((B,), x, dtype=torch.int32, device="cuda") for x in (at, L))
        part = q[:, :, at:at + L].contiguous()
        kb.append_8bit_varlen(None, k[:, :, at:at + L], v[:, :, at:at + L], k8, v8, ke, ve, None, st, ln, block_table=pages)
        o = (kb.decode_8bit_paged(part, k8, v8, ke, ve, pages, st + ln) if L == 1 and page else
             kb.chunk_8bit_varlen(part, k8, v8, ke, ve, st, ln, block_table=pages))
        kc, vc = (torch.stack([seq(kb.cache_values(c, e), 0)])[:, :, :at + L].contiguous() for c, e in ((k8, ke), (v8, ve)))
        want, _ = kb.chunk_lse(part, kc, vc, at)
        assert torch.equal(bits(o), bits(want))
        at += L
    kb.check_device_status()
    # what 8 bits cost: an output is off by the values' half step of 2^-4 and what the keys' does to the weights
    exact = kb.chunk(part, k[:, :, :at].contiguous(), v[:, :, :at].contiguous(), at - 1, check=True)
    assert float((o.double() - exact.double()).norm() / exact.double().norm()) < 0.2
