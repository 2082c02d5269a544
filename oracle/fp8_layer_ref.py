"""CPU oracle of the FP8 layer operators: RMS norm with the residual's
addition, the gated unit, the quantiser by blocks of 128 columns, and the
block-scaled matrix product, dense and grouped by expert.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this file.  All
functions take float64 values and compute in float64, except ``quantize_f32``,
which repeats the quantiser's float32 steps so that codes and scales can be
compared exactly.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-10


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even, saturating at +-448, NaN kept)."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.where(np.isnan(v), 0.0, np.minimum(np.abs(v), E4M3_MAX))
    _, e = np.frexp(np.maximum(mag, 2.0 ** -6))
    step = np.ldexp(1.0, e - 1 - 3)
    out = np.minimum(np.rint(mag / step) * step, E4M3_MAX)
    return np.where(np.isnan(v), np.nan, np.copysign(out, v))


def rmsnorm(x, weight, eps, residual=None):
    """(y, h) in float64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rms = np.sqrt((h * h).sum(axis=1, keepdims=True) / h.shape[1] + eps)
    return h / rms * np.asarray(weight, np.float64), h


def silu_mul(x):
    x = np.asarray(x, np.float64)
    g, u = np.split(x, 2, axis=1)
    return g / (1.0 + np.exp(-g)) * u


def block_amax(v) -> np.ndarray:
    """[blocks, rows] largest magnitudes (NaN where a block holds one)."""
    v = np.asarray(v)
    return np.stack([np.abs(v[:, b * BLOCK:(b + 1) * BLOCK]).max(axis=1) for b in range(blocks(v.shape[1]))])


def spread(scales: np.ndarray, width: int) -> np.ndarray:
    """Block scales [blocks, rows] as a [rows, width] matrix."""
    return np.repeat(scales.T, BLOCK, axis=1)[:, :width]


def quantize_f32(v: np.ndarray):
    """Codes (as values, [rows, cols]) and scales ([blocks, rows], float32) of
    float32 ``v`` by the quantiser's own float32 steps."""
    v = np.asarray(v, np.float32)
    amax = block_amax(v)
    amax = np.where(amax < np.float32(AMAX_FLOOR), np.float32(AMAX_FLOOR), amax)
    scale = (amax / np.float32(E4M3_MAX)).astype(np.float32)
    inv = (np.float32(1.0) / scale).astype(np.float32)
    return round_e4m3((v * spread(inv, v.shape[1])).astype(np.float32)), scale


def gemm(a, a_scales, w, w_scales):
    """(out, mag): the product, and the sum of its terms' magnitudes, from code
    values a [m, k], w [n, k] and scales [blocks, m], [row blocks, blocks]."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    a = a * spread(np.asarray(a_scales, np.float64), a.shape[1])
    ws = np.repeat(np.repeat(np.asarray(w_scales, np.float64), BLOCK, 0)[:w.shape[0]], BLOCK, 1)[:, :w.shape[1]]
    w = w * ws
    return a @ w.T, np.abs(a) @ np.abs(w).T


def grouped_gemm(a, a_scales, w, w_scales, offsets):
    """``gemm`` by expert; rows without an expert are NaN."""
    m, n = a.shape[0], w.shape[1]
    out, mag = np.full((m, n), np.nan), np.full((m, n), np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi], mag[lo:hi] = gemm(a[lo:hi], a_scales[:, lo:hi], w[e], w_scales[e])
    return out, mag
