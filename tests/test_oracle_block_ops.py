"""Pins of the oracle's rotary positions, layer norm and 4-bit linear layer: invariants, finite differences
and closed forms.  No GPU."""
import numpy as np
import pytest

from oracle import linear4 as l4
from oracle import norm, rope


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("axes", [(4, 6, 6), (0, 8, 8), (2, 0, 10)])
def test_rotation_keeps_norms_and_relative_positions(axes, halves):
    rng = np.random.default_rng(1)
    x, z = rng.standard_normal((2, 5, 3, 16))
    pos = rng.integers(0, 50, (5, 3)).astype(float)
    y = rope.rotate(x, pos, axes, halves=halves)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(rope.rotate(y, pos, axes, halves=halves, inverse=True), x)
    shift = np.array([3.0, -7.0, 11.0])
    dots = (y * rope.rotate(z, pos + 2.0, axes, halves=halves)).sum(-1)
    moved = (rope.rotate(x, pos + shift, axes, halves=halves) * rope.rotate(z, pos + shift + 2.0, axes, halves=halves)).sum(-1)
    assert np.allclose(dots, moved)                       # q . k depends on the positions' difference alone
    assert np.array_equal(y[..., sum(axes):], x[..., sum(axes):])
    g = rng.standard_normal(y.shape)                      # the adjoint is the inverse
    assert np.allclose((g * y).sum(), (rope.rotate(g, pos, axes, halves=halves, inverse=True) * x).sum())


def test_grid_positions_count_columns_first():
    p = rope.grid_positions(14, 2, 3, origin=(5.0, 0.0, -1.0), step=(2.0, 1.0, 0.5))
    assert p[0].tolist() == [5.0, 0.0, -1.0] and p[4].tolist() == [5.0, 1.0, -0.5] and p[13].tolist() == [9.0, 0.0, -0.5]


@pytest.mark.parametrize("rpg,unit", [(0, False), (3, True), (1, False)])
def test_norm_gradient_against_differences(rpg, unit):
    rng = np.random.default_rng(2)
    rows, cols = 7, 5
    groups = -(-rows // rpg) if rpg else 1
    x, dy = rng.standard_normal((2, rows, cols))
    w, b = rng.standard_normal((2, groups, cols))

    def loss(x, w, b):
        return (norm.forward(x, w, b, 1e-6, rpg, unit)[0] * dy).sum()

    _, mean, rstd = norm.forward(x, w, b, 1e-6, rpg, unit)
    grads = norm.backward(dy, x, mean, rstd, w, rpg, unit)
    for k, v in enumerate((x, w, b)):
        for at in np.ndindex(v.shape):
            args = [x, w, b]
            h = 1e-6
            up, down = v.copy(), v.copy()
            up[at] += h
            down[at] -= h
            args[k] = up
            hi = loss(*args)
            args[k] = down
            assert abs((hi - loss(*args)) / (2 * h) - grads[k][at]) < 1e-6 * (1 + abs(grads[k][at]))


def test_four_bit_codes_round_trip():
    rng = np.random.default_rng(3)
    w = l4.round_bf16(rng.standard_normal((9, 96)).astype(np.float32))
    w[4, 32:64] = 0.0
    codes, scales = l4.quantize(w, 64)
    assert scales.shape == (9, 2) and codes.min() >= -7 and codes.max() == 7
    assert np.array_equal(l4.unpack(l4.pack(codes)), codes)
    s = np.repeat(scales, 64, axis=1)[:, :96]
    # half a step of the code, the scale's own rounding (7 steps of 2^-8), the weight's rounding
    assert np.all(np.abs(l4.dequantize(codes, scales, 64) - w) <= s * (0.5 + 7 * 2.0 ** -8 + 7 * 2.0 ** -8))
    full = np.arange(-8, 8, dtype=np.int8)[None].repeat(2, 1)
    assert np.array_equal(l4.unpack(l4.pack(full)), full)
