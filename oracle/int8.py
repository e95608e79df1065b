"""Oracle of the int8 (SmoothQuant W8A8) layer and of the channels-last group norm (numpy, CPU).

The quantizer's decisions are its definition's binary32 steps, one numpy float32 operation each; every
sum and product around them is float64 or an exact integer ("From SmoothQuant to SVDQuant", section
Smooth Quant (W8A8): per-channel smoothing, then 8-bit integers for both operands).
"""
from __future__ import annotations

import math

import numpy as np

TINY = np.float32(2.0 ** -100)


def quantize_rows(x: np.ndarray):
    """(codes int8, scales float32) of each row of a float32 matrix."""
    assert x.dtype == np.float32
    codes = np.zeros(x.shape, dtype=np.int8)
    scales = np.zeros(x.shape[0], dtype=np.float32)
    for m, row in enumerate(x):
        a = np.max(np.abs(row))                    # NaN if any element is
        if not np.isfinite(a):
            scales[m] = np.nan
        elif a >= TINY:
            scales[m] = np.divide(a, np.float32(127))
            mul = np.divide(np.float32(127), a)
            codes[m] = np.rint(np.multiply(row, mul, dtype=np.float32)).astype(np.int8)
    return codes, scales


def smooth(x: np.ndarray, inv_s) -> np.ndarray:
    """f32(x * inv_s), one rounding an element."""
    x = x.astype(np.float32)
    return x if inv_s is None else np.multiply(x, np.asarray(inv_s, dtype=np.float32)[None, :], dtype=np.float32)


def linear(xq, sx, wq, sw, bias=None) -> np.ndarray:
    """float64 Y from the exact integer product (M x K codes, N x K codes)."""
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    y = acc.astype(np.float64) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)[None, :]


def activation(y: np.ndarray, act: str) -> np.ndarray:
    if act == "silu":
        e = np.exp(-np.abs(y))
        return y * np.where(y >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    if act == "gelu":
        return 0.5 * y * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def group_norm(x, G: int, gamma=None, beta=None, eps: float = 1e-5, act: str = "none") -> np.ndarray:
    """x [B, S, C] -> float64 [B, S, C]; statistics over the rows and the channels of a group."""
    x = np.asarray(x, dtype=np.float64)
    B, S, C = x.shape
    g = x.reshape(B, S, G, C // G)
    mean = g.mean(axis=(1, 3), keepdims=True)
    var = ((g - mean) ** 2).mean(axis=(1, 3), keepdims=True)
    y = ((g - mean) / np.sqrt(var + eps)).reshape(B, S, C)
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return activation(y, act)
