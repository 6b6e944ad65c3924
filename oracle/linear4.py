"""Linear layer with 4-bit weights and bf16 group scales.  Test infrastructure (see package header).

The layout and the formulas are this library's own (nomas.h); the pages store weights in INT8 only:
    s = bf16(RN(absmax / 7)) per row and group of columns, code = clamp(rint(w / s), -7, 7), stored + 8 in
    the half byte of its column (even columns low);  weight = bf16(code * s);  y = x W^T.
"""
from __future__ import annotations

import numpy as np

from oracle.linear import round_bf16


def quantize(w: np.ndarray, group: int):
    """w float32 [N][K] holding finite bf16 values -> (codes int8 [N][K], scales float32 holding bf16)."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    groups = -(-k // group)
    codes, scales = np.zeros((n, k), np.int8), np.zeros((n, groups), np.float32)
    for g in range(groups):
        part = w[:, g * group:(g + 1) * group]
        s = round_bf16((np.abs(part).max(axis=1) / np.float32(7.0)).astype(np.float32))
        q = np.rint((part / np.where(s > 0, s, np.float32(1.0))[:, None]).astype(np.float32))
        codes[:, g * group:(g + 1) * group] = np.where((s > 0)[:, None], np.clip(q, -7, 7), 0)
        scales[:, g] = s
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    u = (np.asarray(codes, np.int16) + 8).astype(np.uint8)
    return u[:, 0::2] | (u[:, 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    p = np.asarray(packed, np.uint8)
    out = np.empty((p.shape[0], 2 * p.shape[1]), np.int8)
    out[:, 0::2] = (p & 15).astype(np.int8) - 8
    out[:, 1::2] = (p >> 4).astype(np.int8) - 8
    return out


def dequantize(codes: np.ndarray, scales: np.ndarray, group: int) -> np.ndarray:
    """bf16(code * scale) as float32 (the fp32 product of a 4-bit code and a bf16 scale is exact)."""
    s = np.repeat(np.asarray(scales, np.float32), group, axis=1)[:, :codes.shape[1]]
    return round_bf16(codes.astype(np.float32) * s)


def linear(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, group: int):
    """(y, sum |x| |w|) in fp64."""
    w = dequantize(codes, scales, group).astype(np.float64)
    x = np.asarray(x, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T
