"""How far the gradients of block-sparse attention are off, as a root mean square over each block of 128 rows or keys.

The kernels round P, dS, the output behind delta and the results to bf16.  A rounding is off by at most half a step, 2^-8 of the
value, and by 2^-8 / sqrt 3 of the largest value it can have root mean square; roundings of different terms are independent,
so their squares add.  Four of them make 2 * 2^-8 / sqrt 3 = 0.0045 of the size of the terms; the fp32 steps do not count
beside that.  LIMIT is held against the root of the summed squares of the terms before any of them cancel.  delta's error is
common to a row's keys, so a block of a single row with few keys that matter may be further off and is not a case for it."""

import numpy as np

from tests import sparse_plain as plain

LIMIT = 2 * 2.0 ** -8 / np.sqrt(3.0)
BLOCK = 128


def blocks_of(x):
    return [x[..., i:i + BLOCK, :] for i in range(0, x.shape[-2], BLOCK)]


class Exact:
    """The gradients of one KV head in 64 bits: q, dout [4, S, 128], k, v [S, 128], blocks [S, n], all float64."""

    def __init__(self, q, k, v, dout, blocks):
        self.want = plain.gradients(q, k, v, dout, blocks)
        o, p, _ = plain.attention(q, k, v, blocks, np.arange(q.shape[1]))
        ds2 = p ** 2 * ((dout @ v.T) ** 2 + (dout * o).sum(-1, keepdims=True) ** 2) / 128.0
        self.size2 = (ds2 @ k ** 2, (ds2.transpose(0, 2, 1) @ q ** 2).sum(0),
                      ((p ** 2).transpose(0, 2, 1) @ dout ** 2).sum(0))

    def errors(self, got):
        """{"dq", "dk", "dv"}: per block of rows or keys, rms(got - exact) / size of the terms.  A block without terms must
        be zero, and has the error 0."""
        out = {}
        for name, x, y, z in zip(("dq", "dk", "dv"), got, self.want, self.size2):
            out[name] = []
            for a, b, c in zip(blocks_of(x), blocks_of(y), blocks_of(z)):
                assert c.max() > 0 or not a.any(), name
                out[name].append(float(np.sqrt(((a - b) ** 2).mean() / c.mean())) if c.max() > 0 else 0.0)
        return out

    def worst(self, got):
        return {name: max(e) for name, e in self.errors(got).items()}
