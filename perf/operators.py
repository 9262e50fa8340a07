"""Cases of the serving and training operators around block-sparse attention, with their plain forms.

Five operators, in the order in which a model step uses them:

  append  rotate the new queries and keys by their positions, write keys and values into the (contiguous or paged)
          cache and widen the boxes of the key blocks they fall into
  rope    the rotation alone over a whole sequence, and its gradient (the rotation by the negative angle)
  select  for each query row and KV head, the n blocks of 128 keys whose boxes allow the largest scores
  sparse  attention of each query row over its listed blocks (one token against a paged cache, or a chunk of rows)
  train   sparse attention of a whole sequence with the log-sum-exp, and its gradients

All tensors are bf16 with head_dim 128 and four query heads per KV head.  A box holds, per channel, an upper and a lower
bound of the block's keys on a grid of 127 steps either way: with E the smallest integer (within -100..100) for which the
block's largest |key| is at most 127 * 2^(E-7), the upper bound is ceil(max * 2^(7-E)) * 2^(E-7), the lower one
floor(min * 2^(7-E)) * 2^(E-7); both are bf16 values.  A row's query is the group's four heads summed as whole numbers:
t = rint(q * 2^(15-E)) with E as above for the four heads together, u = their sum, n = rint(u * 2^(7-E')) with E' as
above for u.  A block's score is sum_d max(n_d * upper_d, n_d * lower_d): whole numbers times one power of two, so it
has one value in any order of summation; ties go to the lowest block.
"""

import math

import torch

own = False

D = 128          # head_dim
G = 4            # query heads per KV head
BLOCK = 128      # keys per block
HKV = 8
HQ = G * HKV
SCALE = 1.0 / math.sqrt(D)
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one decode step of 16 conversations of about 8K tokens: the smallest call, latency counts
        {"name": "append-1tok-b16-ctx8k", "op": "append", "B": 16, "L": 1, "ctx": 8192, "page": 256},
        # a chunk of a long prompt, at a start that is no multiple of anything
        {"name": "append-chunk2k", "op": "append", "B": 1, "L": 2048, "ctx": 16385, "page": 0},
        # a prefill batch of four prompts of odd lengths (one of them empty) into a paged pool
        {"name": "append-ragged-b4", "op": "append", "B": 4, "L": 4096, "ctx": 4096, "page": 128},
        # the training forward's rotation of a long sequence's queries, and the gradient of keys of an odd length
        {"name": "rope-q-s16k", "op": "rope", "B": 1, "H": HQ, "S": 16384, "inverse": False},
        {"name": "rope-grad-k-b3", "op": "rope", "B": 3, "H": HKV, "S": 4001, "inverse": True},
        # choosing blocks for one new token of 16 long conversations, and for a whole 16K prompt
        {"name": "select-1tok-b16-ctx64k", "op": "select", "B": 16, "L": 1, "ctx": 65536, "n": 16},
        {"name": "select-prefill-16k", "op": "select", "B": 1, "L": 16384, "ctx": 16384, "n": 16},
        # one new token of one long conversation, and of a batch; then a chunk of a 64K prompt
        {"name": "sparse-1tok-b1-ctx64k", "op": "sparse", "B": 1, "L": 1, "ctx": 65536, "n": 16, "page": 128},
        {"name": "sparse-1tok-b32-ctx16k", "op": "sparse", "B": 32, "L": 1, "ctx": 16384, "n": 16, "page": 256},
        {"name": "sparse-chunk2k-ctx64k", "op": "sparse", "B": 1, "L": 2048, "ctx": 65536, "n": 16, "page": 0},
        # training steps: a long sequence, and a batch of a ragged shorter one
        {"name": "train-s8k", "op": "train", "B": 1, "S": 8192, "n": 16},
        {"name": "train-b3-s1999", "op": "train", "B": 3, "S": 1999, "n": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "rope", "select", "sparse", "sparse", "train"])
    if op == "append":
        L = rng.choice([1, _log(rng, 2, 4096)])
        ctx = max(L, _log(rng, 64, 16384))
        return {"op": op, "B": rng.randint(1, 4 if L > 64 else 16), "L": L, "ctx": ctx, "page": rng.choice([0, 128, 256, 512])}
    if op == "rope":
        return {"op": op, "B": rng.randint(1, 3), "H": rng.choice([HQ, HKV]), "S": _log(rng, 100, 5000), "inverse": rng.random() < 0.5}
    if op == "select":
        L = rng.choice([1, _log(rng, 2, 8192)])
        ctx = max(L, _log(rng, 200, 65536 if L <= 2048 else 16384))
        return {"op": op, "B": rng.randint(1, 16) if L == 1 else 1, "L": L, "ctx": ctx, "n": rng.randint(2, 24)}
    if op == "sparse":
        if rng.random() < 0.5:
            return {"op": op, "B": _log(rng, 1, 32), "L": 1, "ctx": _log(rng, 200, 16384), "n": rng.randint(2, 24),
                    "page": rng.choice([128, 256, 512])}
        L = _log(rng, 2, 2000)
        return {"op": op, "B": 1, "L": L, "ctx": max(L, _log(rng, 500, 65000)), "n": rng.randint(2, 16), "page": 0}
    S = _log(rng, 150, 6000)
    return {"op": op, "B": rng.randint(1, 2 if S > 2500 else 4), "S": S, "n": rng.randint(2, 16)}


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


def _table(n, dtype=torch.float32):
    """(cos, sin) of position * 10000^(-2i/128), the angles formed in 64 bits: [n, 64, 2]."""
    inv = 10000.0 ** (-torch.arange(0, D, 2, device=DEVICE, dtype=torch.float64) / D)
    a = torch.arange(n, device=DEVICE, dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).to(dtype)


def _lengths(case, seed):
    """Per-sequence starts and lens of an append, context lengths of a one-token call."""
    B, L, ctx = case["B"], case["L"], case["ctx"]
    g = torch.Generator().manual_seed(seed + 77)
    if L == ctx:                                                     # prompts of odd lengths from position 0
        lens = torch.randint(max(1, L // 3), L + 1, (B,), generator=g)
        lens[0] = L
        if B > 2:
            lens[2] = 0
        return torch.zeros(B, dtype=torch.int64), lens
    starts = ctx - L - torch.randint(0, min(200, ctx - L) + 1, (B,), generator=g)
    return starts, torch.full((B,), L)


def _to_pages(x, page, table, pages):
    """[B, H, cap, ...] laid out as pools [pages, H, page, ...] by a page table (and by whole blocks, for boxes)."""
    B, H, cap = x.shape[:3]
    y = x.view(B, H, cap // page, page, *x.shape[3:]).transpose(1, 2).reshape(B * (cap // page), H, page, *x.shape[3:])
    pool = torch.zeros(pages, *y.shape[1:], dtype=x.dtype, device=x.device)
    pool[table.view(-1).long()] = y
    return pool


def _page_table(g, B, per_seq):
    order = torch.randperm(B * per_seq + 3, generator=g, device=DEVICE)[: B * per_seq]
    return order.view(B, per_seq).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op}
    if op == "rope":
        s["table"] = _table(case["S"])
        # rows as a projection leaves them: [B, S, H * D], seen as [B, H, S, D]
        s["x"] = _randn(g, case["B"], case["S"], case["H"], D).to(torch.bfloat16).transpose(1, 2)
        s["inverse"] = case["inverse"]
        s["out"] = torch.empty(case["B"], case["H"], case["S"], D, dtype=torch.bfloat16, device=DEVICE)
        return s
    if op == "train":
        B, S = case["B"], case["S"]
        s["q"] = _passages(g, B, HKV, S, 64, 0.7, G)
        s["k"] = _passages(g, B, HKV, S, 100, 0.4)
        s["v"] = _randn(g, B, HKV, S, D).to(torch.bfloat16)
        s["dout"] = _randn(g, B, HQ, S, D).to(torch.bfloat16)
        s["blocks"] = _select(s["q"], _boxes(s["k"], S), torch.arange(S, device=DEVICE).expand(B, S), case["n"])
        return s
    B, L, ctx = case["B"], case["L"], case["ctx"]
    if op == "append":
        starts, lens = _lengths(case, seed)
        page = case["page"] or BLOCK
        cap = -(-ctx // page) * page
        fused = _randn(g, B, L, (HQ + 2 * HKV) * D).to(torch.bfloat16)       # one projection's rows: q | k | v
        cut = fused.view(B, L, HQ + 2 * HKV, D).transpose(1, 2)
        s["q"], s["k"], s["v"] = cut[:, :HQ], cut[:, HQ:HQ + HKV], cut[:, HQ + HKV:]
        s["table"] = _table(cap)
        s["starts"], s["lens"] = starts.to(DEVICE, torch.int32), lens.to(DEVICE, torch.int32)
        k, v = (_randn(g, B, HKV, cap, D).to(torch.bfloat16) for _ in range(2))
        boxes = _boxes(k, s["starts"])
        s["page_table"] = None
        if case["page"]:
            s["page_table"] = _page_table(g, B, cap // page)
            n = B * (cap // page) + 3
            k, v = (_to_pages(x, page, s["page_table"], n) for x in (k, v))
            boxes = _to_pages(boxes, page // BLOCK, s["page_table"], n)
        s["k_cache"], s["v_cache"], s["boxes"] = k, v, boxes
        s["out"] = torch.zeros(B, HQ, L, D, dtype=torch.bfloat16, device=DEVICE)
        return s
    s["start"] = ctx - L
    if op == "select":
        s["n"] = case["n"]
        s["q"] = _passages(g, B, HKV, L, 64, 0.7, G)
        s["boxes"] = _boxes(_passages(g, B, HKV, ctx, 100, 0.4), ctx)
        s["out"] = torch.empty(B, HKV, L, case["n"], dtype=torch.int32, device=DEVICE)
        return s
    # sparse: the blocks are the ones that select gives for these queries and keys
    k = _passages(g, B, HKV, ctx, 100, 0.4)
    v = _randn(g, B, HKV, ctx, D).to(torch.bfloat16)
    s["q"] = _passages(g, B, HKV, L, 64, 0.7, G)
    s["out"] = torch.empty(B, HQ, L, D, dtype=torch.bfloat16, device=DEVICE)
    s["page_table"] = None
    if case["page"]:                                                 # one token each, contexts of their own
        page = case["page"]
        cap = -(-ctx // page) * page
        lens = ctx - torch.randint(0, min(300, ctx), (B,), generator=g, device=DEVICE)
        s["ctx_lens"] = lens.to(torch.int32)
        s["blocks"] = _select(s["q"], _boxes(k, lens), lens[:, None] - 1, case["n"])
        s["page_table"] = _page_table(g, B, cap // page)
        k, v = (_to_pages(torch.nn.functional.pad(x, (0, 0, 0, cap - ctx)), page, s["page_table"], B * (cap // page) + 3)
                for x in (k, v))
    else:
        pos = torch.arange(s["start"], ctx, device=DEVICE).expand(B, L)
        s["blocks"] = _select(s["q"], _boxes(k, ctx), pos, case["n"])
    s["k"], s["v"] = k, v
    return s


# --------------------------------------------------------------------------------------------------- plain forms

def _exponent(amax):
    """The smallest E in -100..100 with amax <= 127 * 2^(E-7)."""
    m, e = torch.frexp(amax.float())
    return (e + (m > 127.0 / 128.0)).clamp(-100, 100)


def _boxes(k, n_keys):
    """Boxes [B, H, blocks, 2, D] (upper, lower; bf16) of the first n_keys (a number, or one per sequence) keys of k
    [B, H, S, D]; a block without keys is zero."""
    B, H, S, _ = k.shape
    n = -(-S // BLOCK)
    pos = torch.arange(n * BLOCK, device=k.device).view(1, 1, n, BLOCK, 1)
    n_keys = torch.as_tensor(n_keys, device=k.device).view(-1, 1, 1, 1, 1)
    kb = torch.nn.functional.pad(k, (0, 0, 0, n * BLOCK - S)).view(B, H, n, BLOCK, D)
    return _box_of(kb, pos < n_keys)


def _box_of(kb, seen):
    """Box of blocks of keys [..., BLOCK, D], of the keys that are `seen`."""
    none = ~seen.any(-2)
    hi = torch.where(seen, kb, -math.inf).amax(-2).float().masked_fill_(none, 0.0)
    lo = torch.where(seen, kb, math.inf).amin(-2).float().masked_fill_(none, 0.0)
    e = _exponent(torch.maximum(hi, -lo).amax(-1, keepdim=True))
    step = torch.ldexp(torch.ones_like(hi), e - 7)
    hi = torch.ldexp(hi, 7 - e).ceil().clamp(-127, 127) * step
    lo = torch.ldexp(lo, 7 - e).floor().clamp(-127, 127) * step
    return torch.stack([hi, lo], -2).to(torch.bfloat16)


def _whole_query(q):
    """The group's four heads summed as whole numbers within -127..127: [B, Hkv, L, D]."""
    B, Hq, L, _ = q.shape
    x = q.view(B, Hq // G, G, L, D).float()
    e = _exponent(x.abs().amax((2, 4), keepdim=True))
    u = torch.ldexp(x, 15 - e).round().sum(2)
    e = _exponent(u.abs().amax(-1, keepdim=True))
    return torch.ldexp(u, 7 - e).round()


def _select(q, boxes, pos, n):
    """Blocks [B, Hkv, L, n] int32, ascending, -1 behind the last: each row's first and own block, and the rest by
    score.  boxes [B, Hkv, blocks, 2, D]; pos [B, L] absolute positions."""
    u = _whole_query(q)
    score = torch.cat([u.clamp(min=0), u.clamp(max=0)], -1) @ boxes.float().flatten(-2).transpose(-1, -2)
    own_block = (pos // BLOCK)[:, None, :, None]
    j = torch.arange(boxes.shape[2], device=q.device)
    score.masked_fill_((j == 0) | (j == own_block), math.inf).masked_fill_(j > own_block, -math.inf)
    top, at = torch.sort(score, dim=-1, descending=True, stable=True)
    top, at = top[..., :n], at[..., :n]
    at = torch.where(top == -math.inf, 1 << 30, at).sort(-1).values
    at = torch.nn.functional.pad(at, (0, n - at.shape[-1]), value=1 << 30)
    return torch.where(at == 1 << 30, -1, at).to(torch.int32)


def _rotate(x, cs, inverse=False):
    """x [B, H, L, D] rotated in pairs (i, i + 64) by cs [B or 1, 1, L, 64, 2], in 32 bits."""
    x = x.float()
    a, b = x[..., : D // 2], x[..., D // 2:]
    c, s = cs[..., 0], cs[..., 1]
    if inverse:
        s = -s
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)


def _append(s):
    B, L = s["q"].shape[0], s["q"].shape[2]
    i = torch.arange(L, device=DEVICE)
    live = i < s["lens"][:, None]                                     # [B, L]
    pos = torch.where(live, s["starts"][:, None] + i, 0).long()
    cs = s["table"][pos][:, None]
    q, k = _rotate(s["q"], cs), _rotate(s["k"], cs)
    s["out"].copy_(torch.where(live[:, None, :, None], q, s["out"]))
    pool_k, pool_v, boxes = s["k_cache"], s["v_cache"], s["boxes"]
    b, r = live.nonzero(as_tuple=True)
    p = pos[b, r]
    if s["page_table"] is None:
        at, row = b, p
    else:
        page = pool_k.shape[2]
        at, row = s["page_table"][b, p // page].long(), p % page
    pool_k[at, :, row] = k.transpose(1, 2)[b, r]
    pool_v[at, :, row] = s["v"].transpose(1, 2)[b, r]
    # the boxes of the blocks that the new keys fall into, from all their keys so far
    n = (L + BLOCK - 2) // BLOCK + 1
    block = s["starts"][:, None] // BLOCK + torch.arange(n, device=DEVICE)
    end = (s["starts"] + s["lens"])[:, None]
    b, c = ((block * BLOCK < end) & (s["lens"][:, None] > 0)).nonzero(as_tuple=True)
    block = block[b, c].long()
    seen = (block[:, None] * BLOCK + torch.arange(BLOCK, device=DEVICE)) < end[b]
    if s["page_table"] is None:
        at, sub = b, block
    else:
        per = pool_k.shape[2] // BLOCK
        at, sub = s["page_table"][b, block // per].long(), block % per
    if pool_k.shape[2] % BLOCK:
        raise ValueError("the cache holds whole blocks")
    keys = pool_k.view(pool_k.shape[0], HKV, -1, BLOCK, D)[at, :, sub]
    boxes[at, :, sub] = _box_of(keys, seen[:, None, :, None])
    return s["out"], pool_k, pool_v, boxes


def _chosen(blocks, n_keys, pos):
    """Which keys a row sees: [B, Hkv, 1, L, n_keys] truth values (its blocks, up to its position)."""
    n = -(-n_keys // BLOCK)
    hit = torch.zeros(*blocks.shape[:3], n + 1, dtype=torch.bool, device=blocks.device)
    hit.scatter_(-1, torch.where(blocks < 0, n, blocks).long(), True)
    hit = hit[..., :n].repeat_interleave(BLOCK, -1)[..., :n_keys]
    return (hit & (torch.arange(n_keys, device=blocks.device) <= pos[:, None, :, None]))[:, :, None]


def _softmax_parts(q, k, blocks, pos):
    """Weights [B, Hkv, G, L, S] of each row over its keys, and the log-sum-exp [B, Hkv, G, L]."""
    B, Hq, L, _ = q.shape
    sc = q.view(B, HKV, G * L, D).float() @ k.float().transpose(-1, -2)
    sc = sc.mul_(SCALE).view(B, HKV, G, L, -1).masked_fill_(~_chosen(blocks, k.shape[2], pos), -math.inf)
    m = sc.amax(-1, keepdim=True)
    w = sc.sub_(m).exp_()
    l = w.sum(-1, keepdim=True)
    return w.div_(l), (m + l.log()).squeeze(-1)


def _sparse_rows(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, _, L, _ = q.shape
    if s["page_table"] is None:
        w, _ = _softmax_parts(q, k, s["blocks"], torch.arange(s["start"], s["start"] + L, device=DEVICE).expand(B, L))
        return (w.view(B, HKV, G * L, -1) @ v.float()).view(B, HQ, L, D).to(torch.bfloat16)
    # one token each: only the listed blocks are fetched
    per = k.shape[2] // BLOCK
    ids = s["blocks"][:, :, 0].long()                                 # [B, Hkv, n]
    b = torch.arange(B, device=DEVICE)[:, None, None]
    h = torch.arange(HKV, device=DEVICE)[None, :, None]
    page = s["page_table"][b, ids.clamp(min=0) // per].long()
    kb, vb = (x.view(x.shape[0], HKV, per, BLOCK, D)[page, h, ids.clamp(min=0) % per].float() for x in (k, v))
    sc = torch.einsum("bhgd,bhnkd->bhgnk", q.view(B, HKV, G, D).float(), kb) * SCALE
    key = ids[..., None] * BLOCK + torch.arange(BLOCK, device=DEVICE)
    seen = (ids[..., None] >= 0) & (key < s["ctx_lens"].view(B, 1, 1, 1))
    sc = sc.masked_fill(~seen[:, :, None], -math.inf).flatten(-2)
    w = (sc - sc.amax(-1, keepdim=True)).exp()
    w = (w / w.sum(-1, keepdim=True)).view(B, HKV, G, -1, BLOCK)
    return torch.einsum("bhgnk,bhnkd->bhgd", w, vb).reshape(B, HQ, 1, D).to(torch.bfloat16)


def _train(s):
    q, k, v, dout = s["q"], s["k"], s["v"], s["dout"]
    B, _, S, _ = q.shape
    p, lse = _softmax_parts(q, k, s["blocks"], torch.arange(S, device=DEVICE).expand(B, S))
    p = p.view(B, HKV, G * S, S)
    do = dout.view(B, HKV, G * S, D).float()
    o = p @ v.float()
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.float().transpose(-1, -2)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    dq = ds @ k.float()
    dk = ds.transpose(-1, -2) @ q.view(B, HKV, G * S, D).float()
    shaped = [x.view(B, HQ, S, D).to(torch.bfloat16) for x in (o, dq)]
    return shaped[0], lse.view(B, HQ, S), shaped[1], dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        from bitwise_aligned_causal_gb300 import kb_attn as kb

        if op == "append":
            kb.append_varlen(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["starts"], s["lens"],
                             block_table=s["page_table"], boxes=s["boxes"], out=s["out"])
            return s["out"], s["k_cache"], s["v_cache"], s["boxes"]
        if op == "rope":
            return kb.rope(s["x"], s["table"], inverse=s["inverse"], out=s["out"])
        if op == "select":
            return kb.select_blocks(s["q"], s["boxes"], s["start"], s["n"], out=s["out"])
        if op == "sparse":
            if s["page_table"] is None:
                return kb.sparse_chunk(s["q"], s["k"], s["v"], s["start"], s["blocks"], out=s["out"])
            return kb.sparse_decode_paged(s["q"], s["k"], s["v"], s["page_table"], s["ctx_lens"], s["blocks"], out=s["out"])
        o, lse = kb.sparse_prefill_lse(s["q"], s["k"], s["v"], s["blocks"])
        dq, dk, dv, _ = kb.sparse_backward(s["q"], s["k"], s["v"], o, s["dout"], lse, s["blocks"])
        return o, lse, dq, dk, dv
    if op == "append":
        return _append(s)
    if op == "rope":
        return _rotate(s["x"], s["table"][None, None], s["inverse"])
    if op == "select":
        B, _, L, _ = s["q"].shape
        return _select(s["q"], s["boxes"], torch.arange(s["start"], s["start"] + L, device=DEVICE).expand(B, L), s["n"])
    return _sparse_rows(s) if op == "sparse" else _train(s)


# -------------------------------------------------------------------------------------------------------- floors

def _visible(n, first, rows):
    """Keys that rows at first..first+rows-1 see in all, with n blocks each."""
    return sum((min(n, p // BLOCK + 1) - 1) * BLOCK + p % BLOCK + 1 for p in range(first, first + rows))


def work(case):
    op, B = case["op"], case["B"]
    if op == "rope":
        rows = B * case["H"] * case["S"]
        return {"bytes": 2 * rows * D * 2 + case["S"] * D * 4, "flops": 3 * rows * D}
    if op == "train":
        S, n = case["S"], case["n"]
        keys = B * HQ * _visible(n, 0, S)
        q, kv = B * HQ * S * D * 2, B * HKV * S * D * 2
        # the pair: q, k, v, dout and the lists read once, o, lse, dq, dk, dv written; two products forward, five back
        return {"bytes": 4 * q + 4 * kv + B * HQ * S * 4 + B * HKV * S * n * 4, "flops": 14 * D * keys}
    L, ctx = case["L"], case["ctx"]
    if op == "append":
        rows = B * L if L != ctx else max(1, B * L * 2 // 3)            # ragged prompts: two thirds of the padded rows
        per = (2 * HQ + 4 * HKV) * D * 2 + D * 4
        return {"bytes": rows * per, "flops": 3 * rows * (HQ + HKV) * D}
    n_blocks = -(-ctx // BLOCK)
    if op == "select":
        pairs = B * HKV * sum(p // BLOCK + 1 for p in range(ctx - L, ctx))
        return {"bytes": B * (HQ * L * D * 2 + HKV * n_blocks * 2 * D * 2 + HKV * L * case["n"] * 4), "flops": 4 * D * pairs}
    keys = B * HQ * _visible(case["n"], ctx - L, L)
    cache = 2 * B * HKV * min(case["n"] * L, n_blocks) * BLOCK * D * 2
    return {"bytes": 2 * B * HQ * L * D * 2 + cache + B * HKV * L * case["n"] * 4, "flops": 4 * D * keys}


# --------------------------------------------------------------------------------- the definitions in 64 bits

def _turned(x, pos, inverse=False):
    """x [B, H, L, D] as complex numbers x_i + i x_(i+64) times e^(+-i angle), in 64 bits; pos [B or 1, L]."""
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device), -torch.arange(64, device=x.device, dtype=torch.float64) / 64)
    angle = pos[:, None, :, None].double() * inv
    z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    return torch.cat([z.real, z.imag], -1)


def _exact_rows(q, keys, vals, seen):
    """Softmax attention of q [G, R, D] over keys, vals [S, D] with seen [R, S], in 64 bits: o, weights, log-sum-exp."""
    sc = torch.einsum("grd,sd->grs", q.double(), keys.double()) / math.sqrt(128.0)
    sc = torch.where(seen, sc, torch.tensor(-math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(sc, -1)
    p = torch.exp(sc - lse[..., None])
    return p @ vals.double(), p, lse


def _exact_seen(lists, pos, S):
    """Truth values [R, S]: key j's block is in row r's list and j <= pos[r]."""
    j = torch.arange(S, device=lists.device)
    listed_blocks = torch.zeros(len(lists), S // BLOCK + 2, dtype=torch.bool, device=lists.device)
    listed_blocks[torch.arange(len(lists), device=lists.device)[:, None], lists.long()] = True    # -1: a column of its own
    return listed_blocks[:, j // BLOCK] & (j <= pos[:, None])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"], torch.arange(case["S"], device=DEVICE)[None], s["inverse"])
    if op == "train":
        B, S = case["B"], case["S"]
        o, dq = (torch.empty(B, HQ, S, D, dtype=torch.float64, device=DEVICE) for _ in range(2))
        lse = torch.empty(B, HQ, S, dtype=torch.float64, device=DEVICE)
        dk, dv = (torch.empty(B, HKV, S, D, dtype=torch.float64, device=DEVICE) for _ in range(2))
        pos = torch.arange(S, device=DEVICE)
        for b in range(B):
            for h in range(HKV):
                heads = slice(G * h, G * h + G)
                q, do = s["q"][b, heads].double(), s["dout"][b, heads].double()
                k, v = s["k"][b, h].double(), s["v"][b, h].double()
                y, p, z = _exact_rows(q, k, v, _exact_seen(s["blocks"][b, h], pos, S))
                o[b, heads], lse[b, heads] = y, z
                dv[b, h] = torch.einsum("grs,grd->sd", p, do)
                p = p * (do @ v.T - (do * y).sum(-1, keepdim=True)) / math.sqrt(128.0)
                dq[b, heads] = p @ k
                dk[b, h] = torch.einsum("grs,grd->sd", p, q)
        return o, lse, dq, dk, dv
    B, L, ctx = case["B"], case["L"], case["ctx"]
    if op == "append":
        # the new rows alone change; a box is a rounding of rounded keys and has no value in 64 bits
        out, kc, vc = s["out"].double(), s["k_cache"].double(), s["v_cache"].double()
        for b in range(B):
            n, p0 = int(s["lens"][b]), int(s["starts"][b])
            if n == 0:
                continue
            pos = torch.arange(p0, p0 + n, device=DEVICE)
            out[b, :, :n] = _turned(s["q"][b:b + 1, :, :n], pos[None])[0]
            new_k, new_v = _turned(s["k"][b:b + 1, :, :n], pos[None])[0], s["v"][b, :, :n].double()
            if s["page_table"] is None:
                kc[b, :, p0:p0 + n], vc[b, :, p0:p0 + n] = new_k, new_v
            else:
                page = kc.shape[2]
                at = s["page_table"][b][(pos // page)].long()
                kc[at, :, pos % page], vc[at, :, pos % page] = new_k.transpose(0, 1), new_v.transpose(0, 1)
        return out, kc, vc, None
    if op == "select":
        q = s["q"].double().view(B, HKV, G, L, D)
        fit = lambda a: torch.ceil(torch.log2(a * (128.0 / 127.0)) - 1e-13)  # noqa: E731  (no largest value is that near a border)
        u = torch.round(q * 2.0 ** (15 - fit(q.abs().amax((2, 4), keepdim=True)))).sum(2)
        u = torch.round(u * 2.0 ** (7 - fit(u.abs().amax(-1, keepdim=True))))
        hi, lo = s["boxes"].double().unbind(-2)
        score = (u > 0) * u @ hi.transpose(-1, -2) + (u < 0) * u @ lo.transpose(-1, -2)
        nb = hi.shape[2]
        mine = torch.arange(ctx - L, ctx, device=DEVICE).view(1, 1, L, 1) // BLOCK
        j = torch.arange(nb, device=DEVICE).view(1, 1, 1, nb)
        rank = torch.where((j == 0) | (j == mine), 1e300, score)
        order = torch.argsort(torch.where(j <= mine, rank, -1e300), dim=-1, descending=True, stable=True)[..., : case["n"]]
        take = torch.zeros(B, HKV, L, nb, dtype=torch.bool, device=DEVICE).scatter_(-1, order, True) & (j <= mine)
        found = torch.where(take, j, nb).sort(-1).values[..., : case["n"]]
        found = torch.nn.functional.pad(found, (0, case["n"] - found.shape[-1]), value=nb)
        return torch.where(found == nb, -1, found).to(torch.int32)
    out = torch.empty(B, HQ, L, D, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        for h in range(HKV):
            heads = slice(G * h, G * h + G)
            if s["page_table"] is None:
                k, v, pos = s["k"][b, h], s["v"][b, h], torch.arange(ctx - L, ctx, device=DEVICE)
            else:
                at = s["page_table"][b].long()
                k, v = s["k"][at, h].reshape(-1, D), s["v"][at, h].reshape(-1, D)
                pos = s["ctx_lens"][b:b + 1] - 1
            out[b, heads] = _exact_rows(s["q"][b, heads], k, v, _exact_seen(s["blocks"][b, h], pos, k.shape[0]))[0]
    return out
