"""The bound of gradient_error on the CPU: the kernels' roundings, made in numpy, stay below it, and gradients that are zero,
negated, short of a row, or have one twice do not."""

import numpy as np
import pytest

from tests import sparse_plain as plain
from tests.gradient_error import LIMIT, Exact


def bf16(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def inputs(seed, S, n, none, first=False):
    rng = np.random.default_rng(seed)
    q, dout = (bf16(rng.standard_normal((4, S, 128))) for _ in range(2))
    k, v = (bf16(rng.standard_normal((S, 128))) for _ in range(2))
    blocks = np.full((S, n), -1)
    for i in range(S):
        if rng.random() >= none:
            nb = i // 128 + 1
            m = min(n, nb, int(rng.integers(1, n + 1)))
            blocks[i, :m] = rng.choice(nb, size=m, replace=False)
    if first:
        blocks[:, -1] = 0
    return q, k, v, dout, blocks


def rounded(q, k, v, dout, blocks, rows=None):
    """The gradients with the kernels' roundings; `rows`: how often each row counts in dk and dv."""
    o, p, _ = plain.attention(q, k, v, blocks, np.arange(q.shape[1]))
    delta = (dout * bf16(bf16(p) @ v)).sum(-1, keepdims=True)
    ds = p * (dout @ v.T - delta)
    times = np.ones(q.shape[1]) if rows is None else rows
    dq = bf16(ds @ k / np.sqrt(128.0))                              # dS goes into dq in two parts
    p, ds = (bf16(x).transpose(0, 2, 1) * times for x in (p, ds))
    return dq, bf16((ds @ q).sum(0) / np.sqrt(128.0)), bf16((p @ dout).sum(0))


CASES = [(129, 2, 0.0, False), (130, 1, 0.2, False), (300, 2, 0.95, False), (700, 3, 0.05, False), (1300, 5, 0.0, True)]


@pytest.mark.parametrize("S,n,none,first", CASES)
def test_the_roundings_stay_below_the_limit(S, n, none, first):
    args = inputs(S, S, n, none, first)
    got = Exact(*args).worst(rounded(*args))
    assert max(got.values()) <= 0.8 * LIMIT, got


@pytest.mark.parametrize("S,n,none,first", CASES[1:])
def test_wrong_gradients_do_not(S, n, none, first):
    args = inputs(S, S, n, none, first)
    exact, good, lists = Exact(*args), rounded(*args), args[4]
    for change in (lambda x: 0 * x, lambda x: -x, lambda x: 1.02 * x):
        errors = exact.errors([change(x) for x in good])
        assert min(e for es in errors.values() for e in es if e > 0) > 2 * LIMIT, errors
    for block in {0, S // 256}:
        listing = [i for i in range(128 * (block + 1), S) if block in lists[i]]
        if not listing:
            continue
        rows = np.ones(S)
        for times in (0.0, 2.0):
            rows[listing[len(listing) // 2]] = times
            errors = exact.errors(rounded(*args, rows=rows))
            assert errors["dk"][block] > 2 * LIMIT and errors["dv"][block] > 2 * LIMIT, (block, times, errors)
