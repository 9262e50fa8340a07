"""Calls over an 8-bit cache whose CTAs share keys through the workspace and fold partials in a second kernel: captured and
replayed on new contents, and several at once on different streams."""

import pytest

from tests.test_gpu_append import bits, kb, randn  # noqa: F401
from tests.test_gpu_cache8 import filled

pytestmark = pytest.mark.gpu

# batch, rows, context: shares of one token, runs of segments, few rows, a longer chunk over the bytes, one gathered into bf16
CALLS = [(1, 1, 20000), (20, 1, 9000), (2, 7, 12000), (1, 64, 20000), (1, 700, 3000)]


@pytest.mark.parametrize("B,L,ctx", CALLS)
def test_captured_and_replayed(kb, B, L, ctx):
    import torch

    cache, _, _ = filled(kb, B, ctx, seed=51)
    other, _, _ = filled(kb, B, ctx, seed=52)
    live = [t.clone() for t in cache]
    q, out = randn(53, B, 32, L, 128), torch.empty(B, 32, L, 128, dtype=torch.bfloat16, device="cuda")
    st, ln = (torch.full((B,), x, dtype=torch.int32, device="cuda") for x in (ctx - L, L))
    graphs = []
    for _ in range(2):                                            # (two graphs, each with a workspace of its own)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            kb.chunk_8bit_varlen(q, *live, st, ln, out=out)
        graphs.append(g)
    for i, contents in enumerate((cache, other, cache)):
        for t, x in zip(live, contents):
            t.view(torch.uint8).copy_(x.view(torch.uint8))
        q.copy_(randn(60 + i, B, 32, L, 128))
        st.fill_(ctx - L - i)
        want = kb.chunk_8bit_varlen(q, *contents, st, ln, check=True)
        for g in graphs:
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            kb.check_device_status()
            assert torch.equal(bits(out), bits(want))


def test_all_at_once(kb):
    import torch

    sets = []
    for i, (B, L, ctx) in enumerate(CALLS):
        cache, _, _ = filled(kb, B, ctx, seed=70 + i)
        q = randn(80 + i, B, 32, L, 128)
        sets.append((q, cache, ctx - L, kb.chunk_8bit(q, *cache, ctx - L, check=True)))
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[kb.chunk_8bit(q, *cache, start, stream=streams[(i + r) % len(streams)]) for i, (q, cache, start, _) in enumerate(sets)]
           for r in range(6)]
    torch.cuda.synchronize()
    kb.check_device_status()
    for rounds in got:
        for o, (_, _, _, want) in zip(rounds, sets):
            assert torch.equal(bits(o), bits(want))
