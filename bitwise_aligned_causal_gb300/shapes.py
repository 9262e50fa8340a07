"""Shape rules of the entry points, as pure functions over shape tuples.

The C ABI receives plain pointers and sizes, so it cannot see how large the
caller's buffers are: a key cache shorter than the sequence, or an output
smaller than the query, would turn into reads or writes past an allocation.
The torch binding therefore checks every tensor's full shape against the
others with these functions before it makes any call into the library.
They hold no attention arithmetic and need neither a GPU nor the library, so
the CPU tests cover every mismatch.

Layouts (KernelBraid README, "Features": contiguous [batch, heads, seq,
head_dim], head_dim 128; "Usage": the output has the query's shape):
  q, o      [B, Hq, L, 128]
  k, v      [B, Hkv, cap, 128]                (contiguous cache)
  pools     [num_pages, Hkv, page_size, 128]  (paged cache)
Each function raises ValueError naming the first mismatch and returns the
sizes the C call takes.
"""

from __future__ import annotations

HEAD_DIM = 128


def _shape(t) -> tuple:
    return tuple(int(d) for d in t)


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _rows(name: str, s: tuple) -> None:
    _need(len(s) == 4, f"{name} must have 4 dimensions [batch, heads, seq, head_dim], got {s}")
    _need(s[3] == HEAD_DIM, f"{name} must have head_dim {HEAD_DIM}, got {s}")
    _need(min(s) >= 1, f"{name} has an empty dimension: {s}")


def _same(name: str, s: tuple, ref_name: str, ref: tuple) -> None:
    _need(s == ref, f"{name} must have the shape of {ref_name} {ref}, got {s}")


def query_and_cache(q, k, v, out=None) -> tuple[int, int, int, int, int]:
    """q [B,Hq,L,128]; k = v [B,Hkv,cap,128]; out = q.  Returns (B, Hq, Hkv, L, cap)."""
    q, k, v = _shape(q), _shape(k), _shape(v)
    _rows("q", q)
    _rows("k", k)
    _same("v", v, "k", k)
    _need(k[0] == q[0], f"k must have q's batch {q[0]}, got {k[0]}")
    if out is not None:
        _same("out", _shape(out), "q", q)
    return q[0], q[1], k[1], q[2], k[2]


def prefill(q, k, v, out=None) -> tuple[int, int, int, int]:
    """Whole sequence: the cache holds exactly the query's S positions.  Returns (B, Hq, Hkv, S)."""
    B, Hq, Hkv, S, cap = query_and_cache(q, k, v, out)
    _need(cap == S, f"prefill needs k and v of q's sequence length {S}, got {cap}")
    return B, Hq, Hkv, S


def chunk(q, k, v, start: int, out=None) -> tuple[int, int, int, int, int]:
    """Rows start..start+L-1 against a cache of capacity cap >= start + L.  Returns (B, Hq, Hkv, L, cap)."""
    B, Hq, Hkv, L, cap = query_and_cache(q, k, v, out)
    _need(int(start) >= 0, f"start must be >= 0, got {start}")
    _need(int(start) + L <= cap, f"start + L = {int(start) + L} exceeds the cache capacity {cap}")
    return B, Hq, Hkv, L, cap


def decode(q, k, v, ctx_len: int, out=None) -> tuple[int, int, int, int]:
    """One query row at position ctx_len - 1.  Returns (B, Hq, Hkv, cap)."""
    B, Hq, Hkv, L, cap = query_and_cache(q, k, v, out)
    _need(L == 1, f"decode takes one query row per (batch, head), got {L}")
    _need(1 <= int(ctx_len) <= cap, f"ctx_len must lie in 1..{cap} (the cache capacity), got {ctx_len}")
    return B, Hq, Hkv, cap


def pools(q, k_pages, v_pages, block_table, out=None) -> tuple[int, int, int, int, int, int, int]:
    """Paged cache: pools [num_pages,Hkv,page,128], block_table [B, pages_per_seq].
    Returns (B, Hq, Hkv, L, num_pages, page_size, pages_per_seq)."""
    q, kp, vp, bt = _shape(q), _shape(k_pages), _shape(v_pages), _shape(block_table)
    _rows("q", q)
    _rows("k_pages", kp)
    _same("v_pages", vp, "k_pages", kp)
    _need(len(bt) == 2 and bt[0] == q[0] and bt[1] >= 1,
          f"block_table must be [batch {q[0]}, pages_per_seq >= 1], got {bt}")
    if out is not None:
        _same("out", _shape(out), "q", q)
    return q[0], q[1], kp[1], q[2], kp[0], kp[2], bt[1]


def chunk_paged(q, k_pages, v_pages, block_table, start: int, out=None):
    B, Hq, Hkv, L, num_pages, page, pps = pools(q, k_pages, v_pages, block_table, out)
    _need(int(start) >= 0, f"start must be >= 0, got {start}")
    _need(int(start) + L <= pps * page, f"start + L = {int(start) + L} exceeds the page table's {pps * page} rows")
    return B, Hq, Hkv, L, num_pages, page, pps


def decode_paged(q, k_pages, v_pages, block_table, ctx_lens, out=None):
    B, Hq, Hkv, L, num_pages, page, pps = pools(q, k_pages, v_pages, block_table, out)
    _need(L == 1, f"decode takes one query row per (batch, head), got {L}")
    _need(_shape(ctx_lens) == (B,), f"ctx_lens must have shape ({B},), got {_shape(ctx_lens)}")
    return B, Hq, Hkv, num_pages, page, pps


def varlen(q, k, v, starts, lens, block_table=None, out=None):
    """Ragged batch: starts, lens [B]; k/v a contiguous cache or (with block_table) pools.
    Returns (B, Hq, Hkv, L_max) plus (cap,) or (num_pages, page_size, pages_per_seq)."""
    qs = _shape(q)
    _rows("q", qs)
    B = qs[0]
    for name, t in (("starts", starts), ("lens", lens)):
        _need(_shape(t) == (B,), f"{name} must have shape ({B},), got {_shape(t)}")
    if block_table is None:
        B, Hq, Hkv, L_max, cap = query_and_cache(q, k, v, out)
        _need(L_max <= cap, f"L_max {L_max} exceeds the cache capacity {cap}")
        return B, Hq, Hkv, L_max, cap
    B, Hq, Hkv, L_max, num_pages, page, pps = pools(q, k, v, block_table, out)
    _need(L_max <= pps * page, f"L_max {L_max} exceeds the page table's {pps * page} rows")
    return B, Hq, Hkv, L_max, num_pages, page, pps


def vector_f32(name: str, t, B: int, Hq: int, S: int) -> None:
    """Per-row float32 outputs (log-sum-exp, delta): [B, Hq, S]."""
    _need(_shape(t) == (B, Hq, S), f"{name} must have shape {(B, Hq, S)}, got {_shape(t)}")


def backward(q, k, v, o, dout, dq=None, dk=None, dv=None) -> tuple[int, int, int, int]:
    """Gradients of the whole-sequence prefill: o, dout, dq like q; dk, dv like k.  Returns (B, Hq, Hkv, S)."""
    B, Hq, Hkv, S = prefill(q, k, v, o)
    qs, ks = _shape(q), _shape(k)
    _same("dout", _shape(dout), "q", qs)
    for name, t, ref_name, ref in (("dq", dq, "q", qs), ("dk", dk, "k", ks), ("dv", dv, "v", ks)):
        if t is not None:
            _same(name, _shape(t), ref_name, ref)
    return B, Hq, Hkv, S


# ------------------------------------------------- cache append, rotation, block selection

BLOCK = 128          # keys per block
MAX_SELECT = 128


def rope_table(table) -> tuple[int, int]:
    """(cos, sin) table [n_pos, rot_dim/2, 2].  Returns (n_pos, rot_dim)."""
    t = _shape(table)
    _need(len(t) == 3 and t[2] == 2 and t[0] >= 1, f"table must be [positions, rot_dim/2, 2], got {t}")
    _need(t[1] % 8 == 0 and 8 <= t[1] <= HEAD_DIM // 2, f"table's rot_dim must be a multiple of 16 up to {HEAD_DIM}, "
          f"got {2 * t[1]}")
    return t[0], 2 * t[1]


def rope(x, table, start: int, out=None) -> tuple[int, int, int, int, int]:
    """x [B,H,L,128] at positions start..start+L-1.  Returns (B, H, L, n_pos, rot_dim)."""
    x = _shape(x)
    _rows("x", x)
    n_pos, rot_dim = rope_table(table)
    _need(int(start) >= 0 and int(start) + x[2] <= n_pos,
          f"positions {start}..{int(start) + x[2] - 1} must lie in the table's 0..{n_pos - 1}")
    if out is not None:
        _same("out", _shape(out), "x", x)
    return x[0], x[1], x[2], n_pos, rot_dim


def _box_planes(boxes, planes: int, what: str, Hkv: int, blocks: int) -> None:
    _need(_shape(boxes) == (planes, Hkv, blocks, 2, HEAD_DIM),
          f"boxes must have shape {(planes, Hkv, blocks, 2, HEAD_DIM)} ({what}), got {_shape(boxes)}")


def block_boxes(k, block_table=None, boxes=None) -> tuple:
    """Key cache [B,Hkv,cap,128], or pools with block_table [B, pages_per_seq], and its boxes.
    Returns (B, Hkv, cap, num_pages, page_size, pages_per_seq, box shape); the page sizes are 0 without a table."""
    k = _shape(k)
    _rows("k", k)
    if block_table is None:
        box = (k[0], k[1], (k[2] + BLOCK - 1) // BLOCK, 2, HEAD_DIM)
        if boxes is not None:
            _box_planes(boxes, k[0], "one per block of the cache", k[1], box[2])
        return k[0], k[1], k[2], 0, 0, 0, box
    bt = _shape(block_table)
    _need(len(bt) == 2 and min(bt) >= 1, f"block_table must be [batch, pages_per_seq >= 1], got {bt}")
    _need(k[2] % BLOCK == 0, f"page_size must be a multiple of {BLOCK}, got {k[2]}")
    box = (k[0], k[1], k[2] // BLOCK, 2, HEAD_DIM)
    if boxes is not None:
        _box_planes(boxes, k[0], "one per block of the pool", k[1], box[2])
    return bt[0], k[1], bt[1] * k[2], k[0], k[2], bt[1], box


def append(q, k, v, k_cache, v_cache, table=None, boxes=None, block_table=None, out=None) -> tuple:
    """New rows q [B,Hq,L,128] (or None), k = v [B,Hkv,L,128] for a cache as in block_boxes.
    Returns (B, Hq, Hkv, L, cap, num_pages, page_size, pages_per_seq, n_pos, rot_dim)."""
    k = _shape(k)
    _rows("k", k)
    _same("v", _shape(v), "k", k)
    B, Hkv, cap, num_pages, page, pps, _ = block_boxes(k_cache, block_table, boxes)
    _same("v_cache", _shape(v_cache), "k_cache", _shape(k_cache))
    _need(k[0] == B, f"k must have the cache's batch {B}, got {k[0]}")
    _need(k[1] == Hkv, f"k must have the cache's {Hkv} KV heads, got {k[1]}")
    _need(k[2] <= cap, f"{k[2]} new rows exceed the cache's {cap} positions")
    Hq = 4 * Hkv
    if q is not None:
        qs = _shape(q)
        _need(qs == (B, Hq, k[2], HEAD_DIM), f"q must have shape {(B, Hq, k[2], HEAD_DIM)}, got {qs}")
        if out is not None:
            _same("out", _shape(out), "q", qs)
    else:
        _need(out is None, "out is q's: it must be None without q")
    n_pos, rot_dim = (0, 0) if table is None else rope_table(table)
    return B, Hq, Hkv, k[2], cap, num_pages, page, pps, n_pos, rot_dim


def per_sequence(B: int, **arrays) -> None:
    """Device arrays of one int32 per sequence (None: absent)."""
    for name, t in arrays.items():
        _need(t is None or _shape(t) == (B,), f"{name} must have shape ({B},), got {None if t is None else _shape(t)}")


def select(q, boxes, n: int, keep_first: int, keep_last: int, block_table=None, out=None) -> tuple:
    """q [B,Hq,L,128]; boxes [B,Hkv,blocks,2,128], or pools' boxes [num_pages,Hkv,page/128,2,128] with block_table;
    out [B,Hkv,L,n].  Returns (B, Hq, Hkv, L, blocks per plane, num_pages, page_size, pages_per_seq)."""
    q, bx = _shape(q), _shape(boxes)
    _rows("q", q)
    _need(len(bx) == 5 and bx[3:] == (2, HEAD_DIM) and min(bx) >= 1,
          f"boxes must be [planes, kv_heads, blocks, 2, {HEAD_DIM}], got {bx}")
    _need(1 <= n <= MAX_SELECT, f"n must lie in 1..{MAX_SELECT}, got {n}")
    _need(keep_first >= 0 and keep_last >= 1 and keep_first + keep_last <= n,
          f"keep_first >= 0 and keep_last >= 1 must add up to at most n = {n}, got {keep_first} and {keep_last}")
    num_pages = page = pps = 0
    if block_table is None:
        _need(bx[0] == q[0], f"boxes must have q's batch {q[0]}, got {bx[0]}")
    else:
        bt = _shape(block_table)
        _need(len(bt) == 2 and bt[0] == q[0] and bt[1] >= 1,
              f"block_table must be [batch {q[0]}, pages_per_seq >= 1], got {bt}")
        num_pages, page, pps = bx[0], bx[2] * BLOCK, bt[1]
    if out is not None:
        _need(_shape(out) == (q[0], bx[1], q[2], n), f"out must have shape {(q[0], bx[1], q[2], n)}, got {_shape(out)}")
    return q[0], q[1], bx[1], q[2], bx[2], num_pages, page, pps


def sparse(q, k, v, blocks, block_table=None, out=None) -> tuple:
    """q [B,Hq,L,128]; caches [B,Hkv,cap,128], or pools with block_table; blocks [B,Hkv,L,n].
    Returns (B, Hq, Hkv, L, n, cap, num_pages, page_size, pages_per_seq)."""
    if block_table is None:
        B, Hq, Hkv, L, cap = query_and_cache(q, k, v, out)
        num_pages = page = pps = 0
    else:
        B, Hq, Hkv, L, num_pages, page, pps = pools(q, k, v, block_table, out)
        cap = pps * page
    bl = _shape(blocks)
    _need(len(bl) == 4 and bl[:3] == (B, Hkv, L), f"blocks must have shape [{B}, {Hkv}, {L}, n], got {bl}")
    _need(1 <= bl[3] <= MAX_SELECT, f"blocks must list 1..{MAX_SELECT} per row, got {bl[3]}")
    return B, Hq, Hkv, L, bl[3], cap, num_pages, page, pps
