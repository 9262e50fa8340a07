"""Plain 64-bit definitions of the operators around block-sparse attention,
for the tests: rotation, key-block boxes, block scores and choices, attention
over chosen blocks and its gradient.  They share no code with the kernels."""

import numpy as np

BLOCK = 128


# ------------------------------------------------------------------ rotation

def rotate(x, pos, rot_dim=128, theta=10000.0, interleaved=False, inverse=False):
    """x [..., L, 128] float64 at positions pos [L]: each plane turned by pos * theta^(-2i/rot_dim)."""
    x = np.asarray(x, dtype=np.float64)
    i = np.arange(rot_dim // 2)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * theta ** (-2.0 * i / rot_dim)
    if inverse:
        ang = -ang
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
    a, b = x[..., a_at], x[..., b_at]
    y = x.copy()
    y[..., a_at] = a * np.cos(ang) - b * np.sin(ang)
    y[..., b_at] = b * np.cos(ang) + a * np.sin(ang)
    return y


# --------------------------------------------------------------------- boxes

def exponent(amax):
    """Smallest E in -100..100 with amax <= 127 * 2^(E-7)."""
    m, e = np.frexp(np.asarray(amax, dtype=np.float64))
    e = np.where(m > 127.0 / 128.0, e + 1, e)
    return np.clip(np.where(np.asarray(amax) == 0, -100, e), -100, 100)


def box(keys):
    """Upper and lower bounds [2, 128] of keys [n, 128] (n >= 1)."""
    hi, lo = keys.max(0).astype(np.float64), keys.min(0).astype(np.float64)
    e = exponent(max(np.abs(hi).max(), np.abs(lo).max()))
    up, step = 2.0 ** (7 - e), 2.0 ** (e - 7)
    return np.stack([np.clip(np.ceil(hi * up), -127, 127) * step, np.clip(np.floor(lo * up), -127, 127) * step])


def boxes(k):
    """[H, S, 128] -> [H, ceil(S/128), 2, 128]."""
    return np.stack([[box(h[j:j + BLOCK]) for j in range(0, h.shape[0], BLOCK)] for h in k])


# -------------------------------------------------------------------- choice

def whole_query(q):
    """q [4, 128] -> whole numbers within -127..127."""
    q = np.asarray(q, dtype=np.float64)
    u = np.rint(q * 2.0 ** (15 - exponent(np.abs(q).max()))).sum(0)
    return np.rint(u * 2.0 ** (7 - exponent(np.abs(u).max()))).astype(np.int64)


def choose(q, bx, pos, n, keep_first=1, keep_last=1):
    """Blocks of one row: q [4, 128], bx [blocks, 2, 128] float64, position pos."""
    nb = pos // BLOCK + 1
    w = whole_query(q).astype(np.float64)
    score = np.maximum(w * bx[:nb, 0], w * bx[:nb, 1]).sum(-1)     # exact: see kb_boxes.cuh
    forced = [j for j in range(nb) if j < keep_first or j >= nb - keep_last]
    if nb <= n:
        got = list(range(nb))
    else:
        rest = sorted((j for j in range(nb) if j not in forced), key=lambda j: (-score[j], j))
        got = sorted(forced + rest[:n - len(forced)])
    return np.array(got + [-1] * (n - len(got)))


# ----------------------------------------------------------------- attention

def attention(q, k, v, blocks, pos):
    """Rows q [4, R, 128] of one KV head over the listed blocks [R, n] of k, v [S, 128], row r at position pos[r].
    Returns (o, p, lse) in float64; a row without keys is zero with lse -inf."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    S = k.shape[0]
    j = np.arange(S)
    seen = np.zeros((q.shape[1], S), dtype=bool)
    for r in range(q.shape[1]):
        lst = np.asarray(blocks[r])
        seen[r] = np.isin(j // BLOCK, lst[lst >= 0]) & (j <= pos[r])
    s = np.where(seen, q @ k.T / np.sqrt(128.0), -np.inf)
    m = s.max(-1, keepdims=True)
    w = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = w.sum(-1, keepdims=True)
    p = w / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m + np.log(np.where(l > 0, l, 1.0)), -np.inf)[..., 0]
    return p @ v, p, lse


def gradients(q, k, v, dout, blocks):
    """(dq, dk, dv) of the whole-sequence attention above for one KV head (row r at position r)."""
    q, k, v, dout = (np.asarray(x, dtype=np.float64) for x in (q, k, v, dout))
    o, p, _ = attention(q, k, v, blocks, np.arange(q.shape[1]))
    ds = p * (dout @ v.T - (dout * o).sum(-1, keepdims=True)) / np.sqrt(128.0)
    return ds @ k, np.einsum("grs,grd->sd", ds, q), np.einsum("grs,grd->sd", p, dout)
