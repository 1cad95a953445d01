"""Reference of the 8-bit activation path (oracle): norm, gated activation,
rows in 8-bit integers, and their product.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Values are computed in fp64 from exactly widened operands.  Where the
definition itself rounds (h to the residual's type; p, the step and its
reciprocal in fp32, so that the integers are defined to the last bit) the
rounding is made here, once, in numpy's IEEE fp32.
"""
from __future__ import annotations

import numpy as np

from . import products

TINY = np.float32(2.0 ** -126)


def to_bf16(v: np.ndarray) -> np.ndarray:
    """Values rounded once to bf16, as fp64."""
    return products.bf16_to_f64(products.round_to_bf16(v))


def norm_h(x: np.ndarray, r: np.ndarray | None, r_is_bf16: bool) -> np.ndarray:
    """h = x + r as it is kept, as fp64.  The sum of two fp32 values is rounded
    to fp32 first (the adder's rounding), then to the residual's type."""
    if r is None:
        return np.asarray(x, np.float64)
    s = (np.asarray(x, np.float32) + np.asarray(r, np.float32)).astype(np.float64)
    return to_bf16(s) if r_is_bf16 else s


def rstd(h: np.ndarray, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt(np.mean(h * h, axis=1) + float(np.float32(eps)))


def rmsnorm(h: np.ndarray, gain: np.ndarray | None, eps: float) -> np.ndarray:
    y = h * rstd(h, eps)[:, None]
    return y if gain is None else y * np.asarray(gain, np.float64)


def silu_mul(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * np.asarray(u, np.float64)


def quantize(p: np.ndarray):
    """(q, s) of fp32 rows p: integers as int8 and steps as fp32, to the bit."""
    p = np.asarray(p, np.float32)
    with np.errstate(all="ignore"):
        top = np.max(np.abs(p), axis=1)
        fine = np.isfinite(p).all(axis=1)
        s = np.maximum(top / np.float32(127), TINY).astype(np.float32)
        inv = (np.float32(1) / s).astype(np.float32)
        q = np.rint((p * inv[:, None]).astype(np.float32))
    q = np.where(fine[:, None], q, 0).astype(np.int8)
    return q, np.where(fine, s, np.float32(np.nan)).astype(np.float32)


def gemm(w: np.ndarray, ws: np.ndarray, x: np.ndarray, xs: np.ndarray, bias: np.ndarray | None = None):
    """(y, product) in fp64; the integer sums are exact (|sum| < 2^53)."""
    sums = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    prod = sums * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]
    return (prod if bias is None else prod + np.asarray(bias, np.float64)), prod
