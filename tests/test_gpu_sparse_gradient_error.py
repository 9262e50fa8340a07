"""The gradients of block-sparse attention within the roundings of the kernels, block by block, root mean square: a bound that
a lost row, a row counted twice or a wrong sign does not meet (test_gradient_error.py)."""

import pytest

from tests.gradient_error import LIMIT, Exact
from tests.test_gpu_append import f64, kb, randn  # noqa: F401
from tests.test_gpu_sparse import all_blocks, random_lists

pytestmark = pytest.mark.gpu


def check(kb, q, k, v, dout, lists, heads):
    o, lse = kb.sparse_prefill_lse(q, k, v, lists)
    got = kb.sparse_backward(q, k, v, o, dout, lse, lists, check=True)[:3]
    q, k, v, dout, lists = f64(q), f64(k), f64(v), f64(dout), lists.cpu().numpy()
    got = [f64(x) for x in got]
    for b in range(q.shape[0]):
        for g in heads:
            h = slice(4 * g, 4 * g + 4)
            exact = Exact(q[b, h], k[b, g], v[b, g], dout[b, h], lists[b, g])
            errors = exact.worst((got[0][b, h], got[1][b, g], got[2][b, g]))
            assert max(errors.values()) <= LIMIT, (b, g, errors)


@pytest.mark.parametrize("B,S,n,none", [(1, 129, 2, 0.0), (2, 130, 1, 0.2), (2, 300, 2, 0.95), (1, 700, 3, 0.05),
                                        (1, 1300, 5, 0.0), (1, 2100, 16, 0.1)])
def test_random_lists(kb, B, S, n, none):
    q, k, v, dout = (randn(6000 + S + i, B, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    check(kb, q, k, v, dout, random_lists(6010 + S, B, S, 0, n, none), range(8))


@pytest.mark.parametrize("S", [128, 1025])
def test_every_block(kb, S):
    q, k, v, dout = (randn(6100 + S + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    check(kb, q, k, v, dout, all_blocks(1, S, 0), range(8))


def test_first_block_shared_by_two_ctas(kb):
    """Every row keeps the first block (4500 rows: two CTAs), which alone makes its dk and dv."""
    S, n = 4500, 3
    q, k, v, dout = (randn(6200 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
    lists = random_lists(6204, 1, S, 0, n)
    lists[..., n - 1] = 0
    check(kb, q, k, v, dout, lists, (0, 7))


def test_a_scale_of_the_inputs(kb):
    """Sharp and flat softmaxes."""
    S = 400
    lists = random_lists(6300, 1, S, 0, 3)
    for scale in (0.05, 3.0):
        q, k, v, dout = (randn(6301 + i, 1, h, S, 128) for i, h in enumerate((32, 8, 8, 32)))
        check(kb, (q * scale).contiguous(), k, v, dout, lists, (0, 5))
