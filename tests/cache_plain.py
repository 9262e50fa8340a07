"""Plain definitions of the operators that make a KV cache smaller, for the
tests: 8-bit blocks, key weights, eviction, rotation by several axes.  They
share no code with the kernels."""

import numpy as np

BLOCK = 128


# --------------------------------------------------------------------- 8 bits

def exponent8(amax):
    """Smallest E in -100..100 with amax <= 448 * 2^E; 127 for a magnitude that is not finite."""
    amax = float(amax)
    if not np.isfinite(amax):
        return 127
    e = -100
    while e < 100 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def held8(x, e):
    """What values x (any shape, finite) become in a block of exponent e, in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    if e == 127:
        return np.full_like(x, np.nan)
    m, at = np.frexp(x)
    y = np.ldexp(np.rint(m * 16.0), at - 4)                     # four significant bits, ties to even
    y = np.where(np.abs(y) < 2.0 ** (e - 6), np.copysign(0.0, x), y)
    return np.clip(y, -448.0 * 2.0 ** e, 448.0 * 2.0 ** e)


def blocks8(x):
    """x [H, S, 128]: held values [H, S, 128] and exponents [H, ceil(S/128)] of its blocks."""
    x = np.asarray(x, dtype=np.float64)
    H, S, _ = x.shape
    y, e = np.empty_like(x), np.empty((H, -(-S // BLOCK)), dtype=np.int64)
    for h in range(H):
        for j in range(e.shape[1]):
            part = x[h, BLOCK * j:BLOCK * j + BLOCK]
            e[h, j] = exponent8(np.abs(part).max() if np.isfinite(part).all() else np.inf)
            y[h, BLOCK * j:BLOCK * j + BLOCK] = held8(part, e[h, j])
    return y, e


def rotate32(x, cs, interleaved=False, inverse=False):
    """x [..., L, 128] turned by the table rows cs [L, planes, 2] (float32), two products and a sum, each rounded to
    fp32: float32 [..., L, 128]."""
    x, cs = np.asarray(x, dtype=np.float32), np.asarray(cs, dtype=np.float32)
    n = cs.shape[1]
    i = np.arange(n)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    c, s = cs[..., 0], cs[..., 1] * np.float32(-1.0 if inverse else 1.0)
    a, b = x[..., a_at], x[..., b_at]
    y = x.copy()
    y[..., a_at] = a * c - b * s
    y[..., b_at] = b * c + a * s
    return y


# ------------------------------------------------------------------ attention

def attend(q, k, v, pos):
    """q [4, R, 128], k and v [S, 128], positions pos [R], 64 bits: outputs [4, R, 128], log-sum-exp [4, R], and the
    sum of weight times |v|."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    s = q @ k.T / np.sqrt(128.0)
    s = np.where(np.arange(k.shape[0])[None, None] <= np.asarray(pos)[None, :, None], s, -np.inf)
    m = s.max(-1, keepdims=True)
    w = np.exp(s - m)
    total = w.sum(-1, keepdims=True)
    p = w / total
    return p @ v, (m + np.log(total))[..., 0], p @ np.abs(v)


def key_weights(q, k, lse, pos):
    """q [4, R, 128], k [S, 128], lse [4, R]: weights [S], and how far fp32 may be off each.

    A score is a sum of 128 products: in fp32, in any order and even truncated, it is off by at most 128 * 2^-23 of the
    sum of magnitudes.  The exponent's fused product and its offset round three times (2^-24 of their magnitude, times
    log2 e), the exponential is off by 2^-22, and a sum of n terms, n <= 128 a step and a step at a time, by (96 + steps)
    * 2^-24."""
    q, k, lse = (np.asarray(t, dtype=np.float64) for t in (q, k, lse))
    gives = np.isfinite(lse)[..., None]                          # a row that saw nothing has no weights to give
    lse = np.where(gives, lse[..., None], 0.0)
    s = q @ k.T / np.sqrt(128.0)
    mag = np.abs(q) @ np.abs(k).T / np.sqrt(128.0)
    off = 128 * 2.0 ** -23 * mag + 3 * 2.0 ** -24 * 1.4427 * (np.abs(s) + np.abs(lse)) + 2.0 ** -22
    seen = np.arange(k.shape[0])[None, None] <= np.asarray(pos)[None, :, None]
    p = np.where(seen & gives, np.exp(np.where(seen, s, 0) - lse), 0.0)
    w = p.sum((0, 1))
    steps = 4 * (-(-q.shape[1] // 128) + 1)
    return w, (p * off).sum((0, 1)) + (96 + steps) * 2.0 ** -24 * w


# ------------------------------------------------------------------- eviction

def evict(w, n, keep, first, last):
    """Rows kept of n keys with weights w [>= n] (float32): ascending."""
    if n <= keep:
        return np.arange(n)
    w = np.asarray(w[:n], dtype=np.float64)
    rank = np.where(np.isnan(w), np.inf, w)
    must = (np.arange(n) < first) | (np.arange(n) >= n - last)
    order = sorted(range(n), key=lambda i: (not must[i], not np.isnan(w[i]), -rank[i], i))
    return np.array(sorted(order[:keep]))
