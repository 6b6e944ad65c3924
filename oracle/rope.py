"""Rotary positions over (time, height, width).  Test infrastructure (see package header).

The pages give the latent grid (papers.ananclaw.com "这是什么") and no formula.  The definition written out:
an axis with d channels has d / 2 pairs; pair i turns by p * theta^(-2 i / d) for a token at position p of
the axis; pairs are neighbouring channels ("interleaved") or channel i and i + d / 2 ("halves"); channels
that no axis holds keep their values.  All in fp64, one pair at a time.
"""
from __future__ import annotations

import numpy as np


def grid_positions(tokens: int, grid_h: int, grid_w: int, origin=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0)) -> np.ndarray:
    """fp64 [tokens][3]: frame, row and column of every token in memory order."""
    out = np.empty((tokens, 3))
    for n in range(tokens):
        at = (n // (grid_h * grid_w), n // grid_w % grid_h, n % grid_w)
        out[n] = [o + s * i for o, s, i in zip(origin, step, at)]
    return out


def rotate(x: np.ndarray, positions: np.ndarray, axis_dims, theta: float = 10000.0, halves: bool = False,
           inverse: bool = False) -> np.ndarray:
    """x [tokens][heads][D], positions [tokens][3]; fp64 result."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    c0 = 0
    for a, d in enumerate(axis_dims):
        for i in range(d // 2):
            c1, c2 = (c0 + i, c0 + i + d // 2) if halves else (c0 + 2 * i, c0 + 2 * i + 1)
            angle = positions[:, a].astype(np.float64) * theta ** (-2.0 * i / d) * (-1.0 if inverse else 1.0)
            cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
            y[:, :, c1] = x[:, :, c1] * cos - x[:, :, c2] * sin
            y[:, :, c2] = x[:, :, c1] * sin + x[:, :, c2] * cos
        c0 += d
    return y


def partner_abs(x: np.ndarray, axis_dims, halves: bool = False) -> np.ndarray:
    """|x1| + |x2| of the pair that each channel belongs to (0 where it passes through)."""
    x = np.abs(np.asarray(x, np.float64))
    out = np.zeros_like(x)
    c0 = 0
    for d in axis_dims:
        for i in range(d // 2):
            c1, c2 = (c0 + i, c0 + i + d // 2) if halves else (c0 + 2 * i, c0 + 2 * i + 1)
            out[:, :, c1] = out[:, :, c2] = x[:, :, c1] + x[:, :, c2]
        c0 += d
    return out
