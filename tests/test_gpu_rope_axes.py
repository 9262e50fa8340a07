"""Rotation by positions of several axes against its 64-bit definition, the
rotation by one start, and its own gradient."""

import numpy as np
import pytest

from tests import cache_plain, sparse_plain as plain
from tests.test_gpu_append import BF16_HALF_STEP, assert_rotated, bits, f64, kb, randn  # noqa: F401

pytestmark = pytest.mark.gpu

SECTIONS = [0] * 16 + [1] * 24 + [2] * 24


def positions(seed, axes, B, L, n):
    import torch

    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, n, (axes, B, L), generator=g).to(torch.int32).cuda()


def defined(x, pos, planes, rot_dim, **how):
    """64 bits: every plane taken from the rotation by its own axis's positions."""
    turned = [plain.rotate(x, p, rot_dim, **how) for p in pos]
    y = np.array(x, dtype=np.float64)
    for i, a in enumerate(planes):
        at = [2 * i, 2 * i + 1] if how.get("interleaved") else [i, i + rot_dim // 2]
        y[..., at] = turned[a][..., at]
    return y


@pytest.mark.parametrize("rot_dim,interleaved,planes", [
    (128, False, SECTIONS), (128, True, SECTIONS), (128, False, [i % 3 for i in range(64)]), (64, False, [0] * 5 + [3] * 20 + [1] * 7),
    (16, True, [2, 1, 0, 0, 1, 2, 0, 1]), (80, False, [0] * 40)])
@pytest.mark.parametrize("inverse", [False, True])
def test_definition(kb, rot_dim, interleaved, planes, inverse):
    B, H, L, n = 2, 7, 37, 900
    table = kb.rope_table(n, rot_dim)
    x = randn(1, B, L, H, 128).transpose(1, 2)                   # rows as a projection leaves them, 7 heads
    pos = positions(2, max(planes) + 1, B, L, n)
    y = kb.rope_axes(x, table, pos, planes, inverse=inverse, interleaved=interleaved, check=True)
    assert y.is_contiguous() and tuple(y.shape) == (B, H, L, 128)
    for b in range(B):
        want = defined(f64(x)[b], pos[:, b].cpu().numpy(), planes, rot_dim, interleaved=interleaved, inverse=inverse)
        assert_rotated(f64(y)[b], f64(x), want)


def test_bits_of_the_rotation_by_a_start(kb):
    """Equal positions on every axis, and one axis of consecutive ones, are rope."""
    import torch

    x = randn(5, 3, 32, 130, 128)
    table = kb.rope_table(400)
    want = kb.rope(x, table, start=200)
    pos = (200 + torch.arange(130, dtype=torch.int32, device="cuda")).expand(4, 3, 130).contiguous()
    for planes in ([0] * 64, [i % 4 for i in range(64)], [3] * 30 + [1] * 34):
        assert torch.equal(bits(kb.rope_axes(x, table, pos, planes)), bits(want))
    y = x.clone()
    assert kb.rope_axes(y, table, pos[:1].contiguous(), [0] * 64, out=y, check=True) is y      # in place
    assert torch.equal(bits(y), bits(want))


@pytest.mark.parametrize("B,H,L", [(1, 1, 1), (1, 32, 1), (5, 8, 3), (2, 33, 129), (1, 2, 4097)])
def test_odd_sizes(kb, B, H, L):
    n = 60
    table = kb.rope_table(n)
    x, pos = randn(7, B, H, L, 128), positions(8, 3, B, L, n)
    y = kb.rope_axes(x, table, pos, SECTIONS, check=True)
    cs = table.cpu().numpy()
    for b in range(B):
        p = pos[:, b].cpu().numpy()
        rows = cs[p[np.array(SECTIONS)], np.arange(64)[:, None]].transpose(1, 0, 2)            # [L, 64, 2]
        want = cache_plain.rotate32(x[b].float().cpu().numpy(), rows)
        import torch

        assert torch.equal(bits(y[b].cpu()), bits(torch.from_numpy(want).to(torch.bfloat16)))


def test_gradient(kb):
    """sum(dout * rope_axes(x)) differentiated along dx equals sum(inverse(dout) * dx), by a difference, which is exact
    for a linear map up to the roundings of both sides."""
    L, n = 300, 700
    table, pos = kb.rope_table(n), positions(11, 3, 1, L, n)
    x, dx, dout = randn(12, 1, 8, L, 128), randn(13, 1, 8, L, 128), randn(14, 1, 8, L, 128)
    grad = f64(kb.rope_axes(dout, table, pos, SECTIONS, inverse=True, check=True))
    p = pos[:, 0].cpu().numpy()
    h = 1.0 / 1024
    diff = (f64(dout) * (defined(f64(x) + h * f64(dx), p, SECTIONS, 128) - defined(f64(x) - h * f64(dx), p, SECTIONS, 128))).sum() / (2 * h)
    assert abs((grad * f64(dx)).sum() - diff) <= BF16_HALF_STEP * np.abs(grad * f64(dx)).sum() + 1e-6
    assert_rotated(grad[0], f64(dout), defined(f64(dout)[0], p, SECTIONS, 128, inverse=True))


def test_positions_outside_the_table_are_reported(kb):
    table, x = kb.rope_table(50), randn(15, 1, 8, 9, 128)
    for bad in (-1, 50, 2 ** 31 - 1):
        pos = positions(16, 2, 1, 9, 50)
        pos[1, 0, 4] = bad
        out = x * 0 + 7
        with pytest.raises(kb.KBError):
            kb.rope_axes(x, table, pos, [0] * 32 + [1] * 32, out=out, check=True)
        assert bool((out[:, :, 4] == 7).all())


def test_refusals(kb):
    import torch

    table, x, pos = kb.rope_table(50), randn(17, 1, 8, 9, 128), positions(18, 1, 1, 9, 50)
    planes = [0] * 64
    for args in ((x.float(), table, pos, planes), (x, table.double(), pos, planes), (x, table, pos.long(), planes),
                 (x, table, pos.cpu(), planes), (x.cpu(), table, pos, planes)):
        with pytest.raises(TypeError):
            kb.rope_axes(*args)
    for args in ((x, table, pos, [1] * 64), (x, table, pos[:, :, :8].contiguous(), planes), (x[..., ::2], table, pos, planes)):
        with pytest.raises(ValueError):
            kb.rope_axes(*args)
    assert torch.equal(bits(x), bits(x))


def test_captured_on_another_stream(kb):
    import torch

    table, x, pos = kb.rope_table(500), randn(19, 2, 8, 65, 128), positions(20, 3, 2, 65, 500)
    out = torch.empty(2, 8, 65, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kb.rope_axes(x, table, pos, SECTIONS, out=out)
    new = positions(21, 3, 2, 65, 500)
    pos.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    kb.check_device_status()
    assert torch.equal(bits(out), bits(kb.rope_axes(x, table, new, SECTIONS, check=True)))
