"""Cases of the operators that make a long KV cache smaller, with their plain forms.

Five operators, in the order in which a model step uses them:

  rope     rotate queries or keys by positions with one to four axes (time, height, width of a patch; or simply a
           position per token, as a cache needs whose rows are no longer the positions), and the gradient of that
  append   rotate the new queries and keys by their positions and write keys and values into a cache held in 8 bits,
           one scale for each block of 128 keys and KV head
  attend   attention of new query rows over such a cache (one token, a few rows, or a long chunk)
  weights  add the softmax weights that new query rows give to each cached key, over the rows and the heads of a group
  evict    keep the first, the last and the heaviest keys of a cache, moved together at its front

All tensors are bf16 with head_dim 128 and four query heads per KV head.  An 8-bit value has a sign, four exponent and
three mantissa bits (e4m3, without its subnormal numbers) and stands for itself times 2^E.  E is the smallest integer
in -100..100 for which the block's largest magnitude is at most 448 * 2^E; a value is rounded to four significant bits
(ties to even) and is zero where the rounded magnitude lies below 2^(E-6).  Rounding twice to four bits is rounding
once, so a block has the same bytes whether its keys came one by one or together.
"""

import math

import torch

own = False

D = 128          # head_dim
G = 4            # query heads per KV head
BLOCK = 128      # keys per scale
HKV = 8
HQ = G * HKV
SCALE = 1.0 / math.sqrt(D)
LOW, HIGH = -100, 100       # exponents of a scale
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one decode step of 16 short conversations in a paged cache: the smallest call, latency counts
        {"name": "append-1tok-b16", "op": "append", "B": 16, "L": 1, "ctx": 1000, "page": 256},
        # a prefill batch of four prompts of odd lengths (one of them empty) into a paged pool
        {"name": "append-ragged-b4", "op": "append", "B": 4, "L": 4096, "ctx": 4096, "page": 128},
        # one new token of one long conversation, and of a batch in a paged cache
        {"name": "attend-1tok-b1-ctx64k", "op": "attend", "B": 1, "L": 1, "ctx": 65536, "page": 0},
        {"name": "attend-1tok-b32-ctx16k", "op": "attend", "B": 32, "L": 1, "ctx": 16384, "page": 256},
        # a few drafted tokens of two conversations, checked at once
        {"name": "attend-7rows-b2-ctx32k", "op": "attend", "B": 2, "L": 7, "ctx": 32768, "page": 128},
        # a chunk of a 64K prompt
        {"name": "attend-chunk2k-ctx64k", "op": "attend", "B": 1, "L": 2048, "ctx": 65536, "page": 0},
        # what one new token of 16 conversations looks at, and what a whole prompt does
        {"name": "weights-1tok-b16-ctx16k", "op": "weights", "B": 16, "L": 1, "ctx": 16384, "page": 256},
        {"name": "weights-prefill-8k", "op": "weights", "B": 1, "L": 8192, "ctx": 8192, "page": 0},
        # a 64K cache cut to an eighth, and a ragged paged batch cut to 2000 keys each
        {"name": "evict-b1-64k", "op": "evict", "B": 1, "ctx": 65536, "keep": 8192, "page": 0},
        {"name": "evict-b16-4k", "op": "evict", "B": 16, "ctx": 4500, "keep": 2000, "page": 128},
        # the queries of 64 video frames of 16 x 16 patches (time, height, width), and the gradient of a ragged
        # batch's keys with a position per token
        {"name": "rope-3axes-q-16k", "op": "rope", "B": 1, "H": HQ, "L": 16384, "axes": 3, "inverse": False},
        {"name": "rope-1axis-grad-k-b3", "op": "rope", "B": 3, "H": HKV, "L": 4001, "axes": 1, "inverse": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "weights", "evict", "rope"])
    if op == "append":
        L = rng.choice([1, _log(rng, 2, 4096)])
        ctx = max(L, _log(rng, 64, 4096))
        return {"op": op, "B": rng.randint(1, 4 if L > 64 else 16), "L": L, "ctx": ctx, "page": rng.choice([0, 128, 256, 512])}
    if op in ("attend", "weights"):
        page = rng.choice([0, 128, 256, 512])
        kind = rng.randrange(3)
        if kind == 0:
            return {"op": op, "B": _log(rng, 1, 32), "L": 1, "ctx": _log(rng, 100, 16384), "page": page}
        if kind == 1:
            L = _log(rng, 2, 64)
            return {"op": op, "B": rng.randint(1, 4), "L": L, "ctx": max(L, _log(rng, 100, 32768)), "page": page}
        L = _log(rng, 65, 2048)
        return {"op": op, "B": 1, "L": L, "ctx": max(L, _log(rng, 500, 32768)), "page": page}
    if op == "evict":
        ctx = _log(rng, 200, 32768)
        return {"op": op, "B": rng.randint(1, 16 if ctx < 8192 else 4), "ctx": ctx, "keep": max(100, int(ctx * rng.uniform(0.1, 0.9))),
                "page": rng.choice([0, 128, 256, 512])}
    return {"op": op, "B": rng.randint(1, 3), "H": rng.choice([HQ, HKV]), "L": _log(rng, 100, 5000), "axes": rng.randint(1, 3),
            "inverse": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _passages(g, B, H, S, run, share, heads=1):
    """bf16 [B, H * heads, S, D] of unit variance: a text moves slowly through its topics, so positions of one passage
    (`run` of them) share a direction, and so do the heads of one group."""
    topic = _randn(g, B, H, 1, -(-S // run), 1, D)
    own_part = _randn(g, B, H, heads, -(-S // run), run, D)
    x = own_part.mul_(math.sqrt(1 - share)).add_(topic, alpha=math.sqrt(share))
    return x.view(B, H * heads, -1, D)[:, :, :S].to(torch.bfloat16)


def _values(g, B, S):
    """Values with a few loud channels and loud tokens, as caches have them: [B, HKV, S, D] bf16."""
    loud = torch.exp(_randn(g, 1, HKV, 1, D) * 0.7)
    token = torch.exp(_randn(g, B, HKV, S, 1) * 0.4)
    return (_randn(g, B, HKV, S, D) * loud * token).to(torch.bfloat16)


def _table(n):
    """(cos, sin) of position * 10000^(-2i/128), the angles formed in 64 bits: [n, 64, 2]."""
    inv = 10000.0 ** (-torch.arange(0, D, 2, device=DEVICE, dtype=torch.float64) / D)
    a = torch.arange(n, device=DEVICE, dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


def _lengths(case, seed):
    """Per-sequence starts and lens of a call."""
    B, L, ctx = case["B"], case["L"], case["ctx"]
    g = torch.Generator().manual_seed(seed + 77)
    if L == ctx and B > 1:                                           # prompts of odd lengths from position 0
        lens = torch.randint(max(1, L // 3), L + 1, (B,), generator=g)
        lens[0] = L
        if B > 2:
            lens[2] = 0
        return torch.zeros(B, dtype=torch.int64), lens
    starts = ctx - L - torch.randint(0, min(200, ctx - L) + 1, (B,), generator=g)
    return starts, torch.full((B,), L)


def _page_table(g, B, per_seq):
    order = torch.randperm(B * per_seq + 3, generator=g, device=DEVICE)[: B * per_seq]
    return order.view(B, per_seq).to(torch.int32)


def _to_pages(x, page, table):
    """[B, H, cap, ...] laid out as pools [pages, H, page, ...] by a page table (and by whole blocks, for exponents)."""
    B, H, cap = x.shape[:3]
    y = x.view(B, H, cap // page, page, *x.shape[3:]).transpose(1, 2).reshape(B * (cap // page), H, page, *x.shape[3:])
    pool = torch.zeros(table.numel() + 3, *y.shape[1:], dtype=x.dtype, device=x.device)
    pool[table.view(-1).long()] = y
    return pool


def _pad(x, cap):
    return torch.nn.functional.pad(x, (0, 0, 0, cap - x.shape[2]))


def _planes(axes):
    """The axis of each of the 64 planes: a quarter for time, the rest for height and width alike."""
    cut = {1: [64], 2: [32, 32], 3: [16, 24, 24]}[axes]
    return [a for a, n in enumerate(cut) for _ in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    op, B = case["op"], case["B"]
    s = {"op": op}
    if op == "rope":
        L, axes = case["L"], case["axes"]
        s["planes"] = _planes(axes)
        i = torch.arange(L, device=DEVICE)
        if axes == 1:                                                # each sequence from a position of its own
            pos = (i + torch.randint(0, 5000, (B, 1), generator=g, device=DEVICE))[None]
        else:                                                        # frames of 16 x 16 patches, behind some text
            parts = [i // 256, i // 16 % 16, i % 16][3 - axes:]
            pos = torch.stack(parts)[:, None] + torch.randint(0, 300, (1, B, 1), generator=g, device=DEVICE)
        s["positions"] = pos.to(torch.int32).contiguous()
        s["table"] = _table(L + 5000)
        # rows as a projection leaves them: [B, L, H * D], seen as [B, H, L, D]
        s["x"] = _randn(g, B, L, case["H"], D).to(torch.bfloat16).transpose(1, 2)
        s["inverse"] = case["inverse"]
        s["out"] = torch.empty(B, case["H"], L, D, dtype=torch.bfloat16, device=DEVICE)
        return s
    ctx = case["ctx"]
    page = case["page"]
    cap = -(-ctx // (page or BLOCK)) * (page or BLOCK)
    s["page_table"] = _page_table(g, B, cap // page) if page else None

    def place(x, per=page):
        return _to_pages(x, per, s["page_table"]) if page else x.contiguous()

    if op == "evict":
        k, v = _passages(g, B, HKV, cap, 100, 0.4), _values(g, B, cap)
        s["k"], s["v"] = place(k), place(v)
        lens = ctx - torch.randint(0, min(400, ctx // 2) + 1, (B,), generator=g, device=DEVICE) * (1 if B > 1 else 0)
        s["lens"], s["keep"] = lens.to(torch.int32), case["keep"]
        s["first"], s["last"] = 4, min(64, case["keep"] // 4)
        # heavy-tailed sums, some keys never looked at
        w = torch.exp(_randn(g, B, HKV, cap) * 2.0)
        s["weights"] = torch.where(torch.rand(B, HKV, cap, generator=g, device=DEVICE) < 0.2, 0.0, w)
        s["weights"] *= torch.arange(cap, device=DEVICE) < lens.view(-1, 1, 1)
        s["weights_out"] = torch.empty_like(s["weights"])
        return s
    L = case["L"]
    starts, lens = _lengths(case, seed)
    s["starts"], s["lens"] = starts.to(DEVICE, torch.int32), lens.to(DEVICE, torch.int32)
    s["ctx_lens"], s["start"] = s["starts"] + s["lens"], int(starts[0])
    if op == "append":
        fused = _randn(g, B, L, (HQ + 2 * HKV) * D).to(torch.bfloat16)       # one projection's rows: q | k | v
        cut = fused.view(B, L, HQ + 2 * HKV, D).transpose(1, 2)
        s["q"], s["k"], s["v"] = cut[:, :HQ], cut[:, HQ:HQ + HKV], cut[:, HQ + HKV:]
        s["table"] = _table(cap)
        seen = (torch.arange(cap, device=DEVICE) < s["starts"].view(-1, 1, 1))[..., None]      # what the cache holds
        old = [_randn(g, B, HKV, cap, D) * seen for _ in range(2)]
        s["out"] = torch.zeros(B, HQ, L, D, dtype=torch.bfloat16, device=DEVICE)
    else:
        k = _passages(g, B, HKV, ctx, 100, 0.4)
        s["q"] = _passages(g, B, HKV, L, 64, 0.7, G)
        if op == "weights":
            s["lse"] = _row_lse(s["q"], k, s["starts"])
            s["k"] = place(_pad(k, cap))
            s["weights"] = torch.rand(B, HKV, cap, generator=g, device=DEVICE)
            return s
        old = [_pad(x, cap).float() for x in (k, _values(g, B, ctx))]
        s["out"] = torch.zeros(B, HQ, L, D, dtype=torch.bfloat16, device=DEVICE)
    for name, x in zip(("k", "v"), old):
        c, e = _quantised(x.view(B, HKV, cap // BLOCK, BLOCK, D))
        s[name + "8"] = place(c.view(torch.uint8).view(B, HKV, cap, D)).view(torch.float8_e4m3fn)
        s[name + "_exp"] = place(e, page // BLOCK)
    return s


# --------------------------------------------------------------------------------------------------- plain forms

def _two(e):
    """2^e in 32 bits, exactly (a power function may be a last place off), e in -126..127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest E in -100..100 with amax <= 448 * 2^E."""
    m, e = torch.frexp(amax)
    return torch.where(amax == 0, LOW, e - 9 + (m > 0.875)).clamp(LOW, HIGH)


def _rounded(x, e):
    """x rounded to four significant bits, zero below 2^(e-6)."""
    m, at = torch.frexp(x)
    y = (m * 16).round() * _two(at.clamp(min=-120) - 4)              # (what is smaller still is zero in any block)
    return torch.where(y.abs() < _two(e - 6), 0.0, y)


def _quantised(x):
    """e4m3 values and exponents (int8) of blocks x [..., BLOCK, D] in 32 bits."""
    e = _exponent(x.abs().amax((-1, -2)))
    at = e[..., None, None]
    return (_rounded(x, at) * _two(-at)).to(torch.float8_e4m3fn), e.to(torch.int8)


def _held(c, e):
    """What a cache or pool [n, H, rows, D] of e4m3 values with exponents [n, H, rows / 128] stands for."""
    n, H, rows, _ = c.shape
    return c.float().view(n, H, rows // BLOCK, BLOCK, D).mul_(_two(e)[..., None, None]).view(n, H, rows, D)


def _of_sequences(x, table):
    """[B, H, cap, ...] of a pool by its page table (x itself where there is none)."""
    if table is None:
        return x
    y = x[table.long()].transpose(1, 2)                              # [B, H, pages, page, ...]
    return y.reshape(y.shape[0], y.shape[1], -1, *y.shape[4:])


def _turn(x, cs):
    """x [..., D] in 32 bits turned in pairs (i, i + 64) by cs [..., 64, 2]."""
    a, b = x[..., : D // 2], x[..., D // 2:]
    c, s = cs[..., 0], cs[..., 1]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _rope(s):
    at = s["positions"][torch.tensor(s["planes"], device=DEVICE)].permute(1, 2, 0).long()        # [B, L, 64]
    cs = s["table"][at, torch.arange(D // 2, device=DEVICE)][:, None]
    if s["inverse"]:
        cs = cs * torch.tensor([1.0, -1.0], device=DEVICE)
    return _turn(s["x"].float(), cs).to(torch.bfloat16)


def _append(s):
    B, L = s["q"].shape[0], s["q"].shape[2]
    live = torch.arange(L, device=DEVICE) < s["lens"][:, None]       # [B, L]
    pos = torch.where(live, s["starts"][:, None] + torch.arange(L, device=DEVICE), 0).long()
    cs = s["table"][pos][:, None]
    q = _turn(s["q"].float(), cs).to(torch.bfloat16)
    s["out"].copy_(torch.where(live[:, None, :, None], q, s["out"]))
    b, r = live.nonzero(as_tuple=True)
    # the blocks that the new keys fall into
    n = (L + BLOCK - 2) // BLOCK + 1
    block = s["starts"][:, None] // BLOCK + torch.arange(n, device=DEVICE)
    end = (s["starts"] + s["lens"])[:, None]
    bb, c = ((block * BLOCK < end) & (s["lens"][:, None] > 0)).nonzero(as_tuple=True)
    block = block[bb, c].long()
    key = block[:, None] * BLOCK + torch.arange(BLOCK, device=DEVICE)
    before = (key < s["starts"][bb, None])[:, None, :, None]
    for name, new in (("k", _turn(s["k"].float(), cs)), ("v", s["v"].float())):
        pool, exps = s[name + "8"], s[name + "_exp"]
        rows = torch.zeros(B, HKV, n + 1, BLOCK, D, device=DEVICE)   # the call's blocks of each sequence
        p = pos[b, r]
        first = s["starts"][b].long() // BLOCK
        rows[b, :, p // BLOCK - first, p % BLOCK] = new.transpose(1, 2)[b, r]
        fresh = rows[bb, :, c]
        if s["page_table"] is None:
            at, sub = bb, block
        else:
            per = pool.shape[2] // BLOCK
            at, sub = s["page_table"][bb, block // per].long(), block % per
        view = pool.view(torch.uint8).view(pool.shape[0], HKV, -1, BLOCK, D)
        old = view[at, :, sub].view(torch.float8_e4m3fn).float() * _two(exps[at, :, sub])[..., None, None]
        x = torch.where(before, old, fresh)
        e = _exponent(x.abs().amax((-1, -2)))
        e = torch.where(before.any(2)[..., 0], torch.maximum(e, exps[at, :, sub].int()), e)
        y = (_rounded(x, e[..., None, None]) * _two(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        # rows behind the sequence's last key keep their bytes
        view[at, :, sub] = torch.where((key < end[bb])[:, None, :, None], y, view[at, :, sub])
        exps[at, :, sub] = e.to(torch.int8)
    return s["out"], _held(s["k8"], s["k_exp"]).to(torch.bfloat16), _held(s["v8"], s["v_exp"]).to(torch.bfloat16), s["k_exp"], s["v_exp"]


def _scores(q, k, starts):
    """Scaled scores [B, HKV, G, L, S] in 32 bits, -inf where a row does not see the key."""
    B, _, L, _ = q.shape
    S = k.shape[2]
    sc = q.view(B, HKV, G * L, D).float() @ k.float().transpose(-1, -2)
    hidden = torch.arange(S, device=q.device) > (starts[:, None] + torch.arange(L, device=q.device))[..., None]   # [B, L, S]
    return sc.mul_(SCALE).view(B, HKV, G, L, S).masked_fill_(hidden[:, None, None], -math.inf)


def _row_lse(q, k, starts):
    sc = _scores(q, k, starts)
    m = sc.amax(-1, keepdim=True)
    return (m + sc.sub_(m).exp_().sum(-1, keepdim=True).log()).view(q.shape[0], HQ, q.shape[2])


def _attend(s):
    q = s["q"]
    B, _, L, _ = q.shape
    k, v = (_of_sequences(_held(s[n + "8"], s[n + "_exp"]), s["page_table"]) for n in ("k", "v"))
    sc = _scores(q, k, s["starts"])
    w = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    o = (w.view(B, HKV, G * L, -1) @ v).view(B, HKV, G, L, D) / w.sum(-1, keepdim=True)
    live = (torch.arange(L, device=DEVICE) < s["lens"][:, None])[:, None, :, None]
    return torch.where(live, o.view(B, HQ, L, D).to(torch.bfloat16), s["out"])


def _weights(s):
    q = s["q"]
    B, _, L, _ = q.shape
    sc = _scores(q, _of_sequences(s["k"], s["page_table"]), s["starts"])
    live = torch.arange(L, device=DEVICE) < s["lens"][:, None]
    lse = torch.where(live[:, None], s["lse"], math.inf).view(B, HKV, G, L, 1)
    s["weights"] += sc.sub_(lse).exp_().sum((2, 3))
    return s["weights"]


def _evict(s):
    w, keep = s["weights"], s["keep"]
    cap = w.shape[2]
    n = s["lens"].view(-1, 1, 1)
    row = torch.arange(cap, device=DEVICE)
    key = torch.where((row < s["first"]) | (row >= n - s["last"]), math.inf, w)
    order = torch.sort(torch.where(row < n, key, -math.inf), dim=-1, descending=True, stable=True).indices
    at = torch.where(row[:keep] < n, order[..., :keep], cap).sort(-1).values
    kept = torch.where(at < cap, at, -1).to(torch.int32)
    held = torch.nn.functional.pad(w, (0, 1)).gather(-1, at)
    s["weights_out"].copy_(torch.nn.functional.pad(held, (0, cap - keep)))
    to = row[:keep].expand_as(at)
    src = torch.where(at < cap, at, to)                              # a short sequence stays where it is
    b, h = torch.arange(w.shape[0], device=DEVICE)[:, None, None], torch.arange(HKV, device=DEVICE)[:, None]
    for x in (s["k"], s["v"]):
        if s["page_table"] is None:
            x[b, h, to] = x[b, h, src]
        else:
            page, t = x.shape[2], s["page_table"].long()
            x[t[b, to // page], h, to % page] = x[t[b, src // page], h, src % page]
    return s["k"], s["v"], s["weights_out"], kept


def run(s):
    op = s["op"]
    if own:
        from bitwise_aligned_causal_gb300 import kb_attn as kb

        if op == "rope":
            return kb.rope_axes(s["x"], s["table"], s["positions"], s["planes"], inverse=s["inverse"], out=s["out"])
        if op == "append":
            kb.append_8bit_varlen(s["q"], s["k"], s["v"], s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["table"], s["starts"], s["lens"],
                                  block_table=s["page_table"], out=s["out"])
            return s["out"], kb.cache_values(s["k8"], s["k_exp"]), kb.cache_values(s["v8"], s["v_exp"]), s["k_exp"], s["v_exp"]
        if op == "attend":
            cache = s["k8"], s["v8"], s["k_exp"], s["v_exp"]
            B, _, L, _ = s["q"].shape
            if L == 1 and s["page_table"] is not None:
                return kb.decode_8bit_paged(s["q"], *cache, s["page_table"], s["ctx_lens"], out=s["out"])
            if B == 1 and s["page_table"] is None:
                return kb.decode_8bit(s["q"], *cache, s["start"] + 1, out=s["out"]) if L == 1 else kb.chunk_8bit(s["q"], *cache, s["start"], out=s["out"])
            return kb.chunk_8bit_varlen(s["q"], *cache, s["starts"], s["lens"], block_table=s["page_table"], out=s["out"])
        if op == "weights":
            if s["q"].shape[0] == 1 and s["page_table"] is None:
                return kb.key_weights(s["q"], s["k"], s["lse"], s["weights"], s["start"])
            return kb.key_weights_varlen(s["q"], s["k"], s["lse"], s["weights"], s["starts"], s["lens"], block_table=s["page_table"])
        kept = kb.evict(s["k"], s["v"], s["weights"], s["lens"], s["keep"], keep_first=s["first"], keep_last=s["last"],
                        block_table=s["page_table"], weights_out=s["weights_out"])
        return s["k"], s["v"], s["weights_out"], kept
    return {"rope": _rope, "append": _append, "attend": _attend, "weights": _weights, "evict": _evict}[op](s)


# -------------------------------------------------------------------------------------------------------- floors

def work(case):
    op, B = case["op"], case["B"]
    if op == "rope":
        rows = B * case["H"] * case["L"]
        return {"bytes": 2 * rows * D * 2 + B * case["L"] * (D * 4 + 4 * case["axes"]), "flops": 3 * rows * D}
    ctx = case["ctx"]
    if op == "evict":
        n = min(case["keep"], ctx)
        return {"bytes": B * HKV * (2 * 2 * n * D * 2 + 4 * ctx + 8 * n), "flops": B * HKV * ctx}
    L = case["L"]
    if op == "append":
        rows = B * L if L != ctx or B == 1 else max(1, B * L * 2 // 3)      # ragged prompts: two thirds of the padded rows
        cap = -(-ctx // (case["page"] or BLOCK)) * (case["page"] or BLOCK)
        # the rows, and what the whole cache stands for
        return {"bytes": rows * ((2 * HQ + 2 * HKV) * D * 2 + 2 * HKV * D + D * 4) + 3 * 2 * B * HKV * cap * D, "flops": 3 * rows * (HQ + HKV) * D}
    pairs = B * HQ * sum(p + 1 for p in range(ctx - L, ctx)) * (0.6 if L == ctx and B > 1 else 1)
    if op == "attend":
        return {"bytes": 2 * B * HQ * L * D * 2 + 2 * B * HKV * ctx * D, "flops": 4 * D * pairs}
    return {"bytes": B * HQ * L * (D * 2 + 4) + B * HKV * ctx * (D * 2 + 8), "flops": 2 * D * pairs}


# --------------------------------------------------------------------------------- the definitions in 64 bits

def _turned(x, angle):
    """x [B, H, L, D] as complex numbers x_i + i x_(i+64) times e^(i angle), in 64 bits; angle [B, 1, L, 64]."""
    z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)


def _inv():
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEVICE), -torch.arange(64, device=DEVICE, dtype=torch.float64) / 64)


def _power(e):
    """2^e in 64 bits from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stands_for(c, e):
    return (c.double().unflatten(2, (-1, BLOCK)) * _power(e)[..., None, None]).flatten(2, 3)


def _in_8_bits(x, e):
    """x [H, n, D] in 64 bits on the grid of exponents e [H, 1, 1]."""
    step = _power(torch.floor(torch.log2(x.abs().clamp(min=1e-300))) - 3)
    y = torch.round(x / step) * step
    return torch.where(y.abs() < _power(e - 6), 0.0, y)


def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    if op == "rope":
        angle = s["positions"].double()[torch.tensor(s["planes"], device=DEVICE)].permute(1, 2, 0)[:, None] * _inv()
        return _turned(s["x"], -angle if case["inverse"] else angle)
    table = s["page_table"]

    def rows_of(pool, b):                                            # [H, cap, ...] of sequence b
        return pool[b] if table is None else pool[table[b].long()].transpose(0, 1).flatten(1, 2)

    if op == "evict":
        out = [s["k"].double(), s["v"].double(), torch.zeros_like(s["weights"]).double()]
        for b in range(B):
            n = int(s["lens"][b])
            m = min(n, s["keep"])
            w = s["weights"][b, :, :n].double()
            w[:, :s["first"]] = w[:, max(0, n - s["last"]):] = 1e300
            at = torch.argsort(-w, dim=-1, stable=True)[:, :m].sort(-1).values
            out[2][b, :, :m] = s["weights"][b].double().gather(-1, at)
            for x, pool in zip(out, (s["k"], s["v"])):
                y = rows_of(pool, b).double().gather(1, at[..., None].expand(-1, -1, D))
                if table is None:
                    x[b, :, :m] = y
                else:
                    i = torch.arange(m, device=DEVICE)
                    x[table[b].long()[i // pool.shape[2]], :, i % pool.shape[2]] = y.transpose(0, 1)
        return out[0], out[1], out[2], None
    L, ctx = case["L"], case["ctx"]
    if op == "append":
        out = s["out"].double()
        pools = {n: _stands_for(s[n + "8"], s[n + "_exp"]) for n in ("k", "v")}
        for b in range(B):
            n, p0 = int(s["lens"][b]), int(s["starts"][b])
            if n == 0:
                continue
            angle = torch.arange(p0, p0 + n, device=DEVICE).double()[None, None, :, None] * _inv()
            out[b, :, :n] = _turned(s["q"][b:b + 1, :, :n], angle)[0]
            for name, new in (("k", _turned(s["k"][b:b + 1, :, :n], angle)[0]), ("v", s["v"][b, :, :n].double())):
                for j in range(p0 // BLOCK, (p0 + n - 1) // BLOCK + 1):
                    lo, hi = max(p0, j * BLOCK), min(p0 + n, (j + 1) * BLOCK)
                    if table is None:
                        at, r = b, j * BLOCK
                    else:
                        page = s["k8"].shape[2]
                        at, r = int(table[b, j * BLOCK // page]), j * BLOCK % page
                    old, e = pools[name][at, :, r:r + lo - j * BLOCK], s[name + "_exp"][at, :, r // BLOCK].double()
                    x = new[:, lo - p0:hi - p0]
                    fit = torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448) - 1e-13)     # (a logarithm of 2^-7 may not be -7)
                    fit = fit.clamp(LOW, HIGH) if lo == j * BLOCK else torch.maximum(fit, e)
                    x = _in_8_bits(torch.cat([old, x], 1), fit[:, None, None])
                    pools[name][at, :, r:r + hi - j * BLOCK] = x
                    # what lies behind the sequence's keys keeps its bytes, and stands for them times the new scale
                    pools[name][at, :, r + hi - j * BLOCK:r + BLOCK] *= _power(fit - e)[:, None, None]
        return out, pools["k"], pools["v"], None, None
    if op == "attend":
        out = s["out"].double()
    else:
        out = s["weights"].double()
    for b in range(B):
        n, p0 = int(s["lens"][b]), int(s["starts"][b])
        if n == 0:
            continue
        hidden = torch.arange(p0 + n, device=DEVICE) > torch.arange(p0, p0 + n, device=DEVICE)[:, None]
        for h in range(HKV):
            q = s["q"][b, G * h:G * h + G, :n].double()
            if op == "attend":
                # (indexing has no 8-bit floating type everywhere: the pages are fetched as bytes)
                k, v = (_stands_for(rows_of(s[x + "8"].view(torch.uint8)[:, h:h + 1], b).contiguous().view(torch.float8_e4m3fn)[None],
                                    rows_of(s[x + "_exp"][:, h:h + 1], b)[None])[0, 0, :p0 + n] for x in ("k", "v"))
            else:
                k = rows_of(s["k"][:, h:h + 1], b)[0, :p0 + n].double()
            sc = (torch.einsum("grd,sd->grs", q, k) / math.sqrt(128.0)).masked_fill_(hidden, -math.inf)
            if op == "attend":
                out[b, G * h:G * h + G, :n] = torch.softmax(sc, -1) @ v
            else:
                out[b, h, :p0 + n] += torch.exp(sc - s["lse"][b, G * h:G * h + G, :n, None].double()).sum((0, 1))
    return out
