"""Reference of the 4-bit weights and of the block norm (oracle).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Values are computed in fp64 from exactly widened operands.  Where the
definition itself rounds (scales and offsets to the type they are kept in, the
quotient that becomes an integer in fp32) the rounding is made here, once, in
numpy's IEEE fp32.
"""
from __future__ import annotations

import numpy as np

from . import int8 as o8

TINY = np.float32(2.0 ** -126)


def groups(cols: int, group: int) -> int:
    return (cols + group - 1) // group


def spread(v: np.ndarray, cols: int, group: int) -> np.ndarray:
    """[groups, rows] as one value per row and column."""
    return np.repeat(np.asarray(v), group, axis=0)[:cols].T


def _kept(v: np.ndarray, bf16: bool) -> np.ndarray:
    return o8.to_bf16(v.astype(np.float64)).astype(np.float32) if bf16 else v.astype(np.float32)


def quantize(p: np.ndarray, group: int, affine: bool, bf16_scales: bool):
    """(q, scale, offset): integers as int8 [rows, cols], scale and offset as
    fp32 [groups, rows] (offset None without affine), to the bit."""
    p = np.asarray(p, np.float32)
    rows, cols = p.shape
    n = groups(cols, group)
    scale, offset = np.empty((n, rows), np.float32), np.zeros((n, rows), np.float32)
    q = np.empty((rows, cols), np.int8)
    f = np.float32
    with np.errstate(all="ignore"):
        for g in range(n):
            w = p[:, g * group: (g + 1) * group]
            fine = np.isfinite(w).all(axis=1)
            if affine:
                top, low = w.max(axis=1), w.min(axis=1)
                s = _kept(np.maximum(top * (f(1) / f(15)) - low * (f(1) / f(15)), TINY), bf16_scales)
                m = _kept((low * f(0.5) + top * f(0.5)) + s * f(0.5), bf16_scales)
            else:
                s = _kept(np.maximum(np.abs(w).max(axis=1) * (f(1) / f(7)), TINY), bf16_scales)
                m = np.zeros_like(s)
            t = (w - m[:, None]).astype(np.float32) if affine else w
            k = np.clip(np.rint((t / s[:, None]).astype(np.float32)), -8, 7)
            q[:, g * group: (g + 1) * group] = np.where(fine[:, None], k, 0).astype(np.int8)
            scale[g] = np.where(fine, s, f(np.nan))
            offset[g] = np.where(fine, m, f(np.nan))
    return q, scale, offset if affine else None


def pack(q: np.ndarray) -> np.ndarray:
    """Integers as packed bytes [rows, ceil(cols / 2)]: q + 8, the even column
    in the low half, 8 behind the last column of an odd number."""
    u = (np.asarray(q, np.int16) + 8).astype(np.uint8)
    if u.shape[1] % 2:
        u = np.concatenate([u, np.full((u.shape[0], 1), 8, np.uint8)], axis=1)
    return u[:, ::2] | (u[:, 1::2] << 4)


def unpack(packed: np.ndarray, cols: int) -> np.ndarray:
    b = np.asarray(packed, np.uint8)
    u = np.stack([b & 15, b >> 4], axis=2).reshape(b.shape[0], -1)[:, :cols]
    return u.astype(np.int16) - 8


def values(q: np.ndarray, scale: np.ndarray, offset, group: int) -> np.ndarray:
    """What the integers stand for, in fp64."""
    cols = q.shape[1]
    v = q.astype(np.float64) * spread(np.asarray(scale, np.float64), cols, group)
    return v if offset is None else v + spread(np.asarray(offset, np.float64), cols, group)


def dequantize_f32(q: np.ndarray, scale: np.ndarray, offset, group: int) -> np.ndarray:
    """The same as the definition rounds it: the product to fp32, then the sum."""
    cols = q.shape[1]
    with np.errstate(all="ignore"):
        v = q.astype(np.float32) * spread(np.asarray(scale, np.float32), cols, group)
        return v if offset is None else (v + spread(np.asarray(offset, np.float32), cols, group)).astype(np.float32)


def gemm(q, scale, offset, group, x, bias=None):
    """(y, mass) in fp64: the product, and what its rounding errors go by: the
    sum of the magnitudes of (q + 8) x s, -8 x s and m x."""
    x = np.asarray(x, np.float64)
    y = x @ values(q, scale, offset, group).T
    mass = np.abs(x) @ values(np.asarray(q, np.int64) + 16, np.abs(scale), None if offset is None else np.abs(offset), group).T
    return (y if bias is None else y + np.asarray(bias, np.float64)), mass


def join(x, r, post_norm, post, post_eps, gate, branch, keep):
    """(h before it is rounded to the residual's type, the branch's part of it), fp64."""
    p = np.asarray(x, np.float64)
    if post_norm:
        p = p * o8.rstd(p, post_eps)[:, None]
        if post is not None:
            p = p * np.asarray(post, np.float64)
    if gate is not None:
        p = p * np.asarray(gate, np.float64)
    p = p * float(np.float32(branch))
    return float(np.float32(keep)) * np.asarray(r, np.float64) + p, p
