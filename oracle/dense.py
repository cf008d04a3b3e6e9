"""fp64 forms of the 8-bit integer product and of the gated block on bf16 weights (NumPy).

Inputs are plain arrays (bf16 inputs already widened); sums are exact integers
or fp64.  The roundings that belong to a definition (codes, the fp32 products
with the scales, the bf16 activation) are made here too.
"""

from __future__ import annotations

import numpy as np

from .stq1 import bf16_bits_from_f64, bf16_to_f64, silu

I8_MIN_AMAX = 2.0 ** -119


def quantize_i8(src) -> tuple[np.ndarray, np.ndarray]:
    """fp32 rows [R, K] -> (int8 codes, fp32 scales)."""
    v = np.asarray(src, dtype=np.float32)
    amax = np.abs(v).max(axis=1)                      # a NaN anywhere makes it NaN
    amax = np.where(np.isnan(v).any(axis=1), np.float32(np.nan), amax).astype(np.float32)
    live = np.isfinite(amax) & (amax >= np.float32(I8_MIN_AMAX))
    safe = np.where(live, amax, np.float32(1)).astype(np.float32)
    inv = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.rint((v * inv[:, None]).astype(np.float32))
    q = np.where(live[:, None], q, 0).astype(np.int8)
    scales = np.where(live, safe / np.float32(127), np.where(np.isfinite(amax), np.float32(0), amax))
    return q, scales.astype(np.float32)


def i8_matmul(xq, sx, wq, sw) -> np.ndarray:
    """fp32 [T, N]: the exact sum rounded to fp32, then the two fp32 products."""
    acc = (np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        return ((acc * np.asarray(sx, np.float32)[:, None]) * np.asarray(sw, np.float32)[None, :]).astype(np.float32)


def i8_ffn(x, gu_q, gu_s, dn_q, dn_s) -> np.ndarray:
    """fp32 [T, H] of the 8-bit gated layer for x already widened to fp32."""
    y = i8_matmul(*quantize_i8(x), gu_q, gu_s).astype(np.float64)
    half = y.shape[1] // 2
    act = bf16_to_f64(bf16_bits_from_f64(silu(y[:, :half]) * y[:, half:]))
    return i8_matmul(*quantize_i8(act.astype(np.float32)), dn_q, dn_s)


def glu(x, w):
    """(act, y, s) in fp64: the activation, the gate/up sums and sum_k |x w| behind each sum."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = x @ w.T
    half = w.shape[0] // 2
    return silu(y[:, :half]) * y[:, half:], y, np.abs(x) @ np.abs(w).T


def glu_dy(dact, y) -> np.ndarray:
    """[T, N] fp64: the gradient at the gate/up sums."""
    y = np.asarray(y, np.float64)
    half = y.shape[1] // 2
    g, u, d = y[:, :half], y[:, half:], np.asarray(dact, np.float64)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], axis=1)


def glu_backward(dact, y, x, w):
    """(dx, dw) in fp64."""
    dy = glu_dy(dact, y)
    return dy @ np.asarray(w, np.float64), dy.T @ np.asarray(x, np.float64)
