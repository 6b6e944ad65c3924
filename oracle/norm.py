"""Layer norm with a weight and bias row per group of rows, and its gradient, in fp64.  Test infrastructure
(see package header).  The formulas are stated in nomas.h; the pages name no norm.
"""
from __future__ import annotations

import numpy as np


def _per_row(p, rows, rows_per_group):
    """A parameter row for every row of x."""
    p = np.asarray(p, np.float64)
    p = p.reshape(-1, p.shape[-1])
    if not rows_per_group:
        return np.repeat(p, rows, axis=0)
    return p[np.arange(rows) // rows_per_group]


def factor(w, shape, rows_per_group=0, unit_offset=False):
    """u + w for every element (1 without a weight)."""
    if w is None:
        return np.ones(shape)
    return _per_row(w, shape[0], rows_per_group) + (1.0 if unit_offset else 0.0)


def forward(x, w=None, b=None, eps=1e-6, rows_per_group=0, unit_offset=False):
    """(y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * factor(w, x.shape, rows_per_group, unit_offset)
    if b is not None:
        y = y + _per_row(b, x.shape[0], rows_per_group)
    return y, mean, rstd


def group_sums(v, rows_per_group=0):
    rows = v.shape[0]
    step = rows_per_group or max(rows, 1)
    starts = range(0, rows, step) if rows else ([0] if not rows_per_group else [])
    return np.stack([v[r:r + step].sum(axis=0) for r in starts]) if len(starts) else np.zeros((0, v.shape[1]))


def backward(dy, x, mean, rstd, w=None, rows_per_group=0, unit_offset=False):
    """(dx, dw, db) for the given statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xhat = (x - np.asarray(mean, np.float64)[:, None]) * r
    g = dy * factor(w, x.shape, rows_per_group, unit_offset)
    dx = r * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx, group_sums(dy * xhat, rows_per_group), group_sums(dy, rows_per_group)
