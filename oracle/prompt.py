"""The prompt operators: MXFP8 quantisation, residual norm, grouping by expert,
ragged expert products and the weighted combination.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The block format is the GC-MoE summary's (onedev.kr/papers/1690, "How it is
used"): routed activations as FP8 E4M3 with one UE8M0 scale per 32 values
along K. How a block's scale is chosen follows the usual MX recipe (shared
exponent floor(log2 amax) - 8, elements saturated to 448 and rounded to
nearest, ties to even). Everything is float64.
"""
from __future__ import annotations

import numpy as np

from .bf16 import bf16_rne
from .moe import silu
from .mxfp4 import dequantize as dequantize_mxfp4
from .mxfp8 import BLOCK, dequantize


def e4m3_rne(a) -> np.ndarray:
    """float64 -> the nearest E4M3 value (ties to even), saturated to 448."""
    a = np.asarray(a, dtype=np.float64)
    _, ex = np.frexp(a)                           # |a| = m * 2^ex, m in [0.5, 1)
    q = np.maximum(ex, -5) - 4                    # 4 significant bits, steps of 2^-9 below 2^-6
    return np.clip(np.ldexp(np.rint(np.ldexp(a, -q)), q), -448.0, 448.0)


def mx_exponent(v) -> np.ndarray:
    """Shared exponents [..., K/32] of rows [..., K]."""
    b = np.asarray(v, dtype=np.float64).reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    amax = np.abs(b).max(-1)
    _, ex = np.frexp(amax)
    return np.where(amax == 0, 0, np.clip(ex - 1 - 8, -127, 127)).astype(np.int64)


def quantize_mxfp8(v):
    """(elements float64 [..., K], scale codes uint8 [..., K/32]) of finite rows."""
    e = mx_exponent(v)
    q = e4m3_rne(np.ldexp(v, -np.repeat(e, BLOCK, axis=-1)))
    return q, (e + 127).astype(np.uint8)


def add_rms_norm(x, weight, residual=None, eps=1e-6):
    """(s, n): the bf16 residual stream and the normalised rows before rounding."""
    s = bf16_rne(x + residual) if residual is not None else np.asarray(x, dtype=np.float64)
    return s, s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + eps) * weight


def group(ids, E):
    """(offsets [E + 1], rows [T * k], slots [T, k]) by scanning the slots of
    every expert in turn."""
    ids = np.asarray(ids)
    T, k = ids.shape
    offsets = np.zeros(E + 1, dtype=np.int32)
    rows = np.full(T * k, -1, dtype=np.int32)
    slots = np.full((T, k), -1, dtype=np.int32)
    at = 0
    for e in range(E):
        for p in np.flatnonzero(ids.reshape(-1) == e):
            rows[at] = p // k
            slots[p // k, p % k] = at
            at += 1
        offsets[e + 1] = at
    return offsets, rows, slots


def product(w, w_scales, a, a_scales, offsets, rows=None, fmt="mxfp8"):
    """(Y, S) float64 [R, N] of every grouped row: W[e] a, and the sum of the
    products' magnitudes, which bounds what an FP32 sum can lose. Rows outside
    every group are NaN."""
    deq = dequantize if fmt == "mxfp8" else dequantize_mxfp4
    av = dequantize(a, a_scales)
    if rows is not None:
        av = av[np.maximum(rows, 0)]
    R, N = av.shape[0], w.shape[1]
    Y, S = np.full((R, N), np.nan), np.full((R, N), np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            wv = deq(w[e], w_scales[e])
            Y[lo:hi] = av[lo:hi] @ wv.T
            S[lo:hi] = np.abs(av[lo:hi]) @ np.abs(wv).T
    return Y, S


def silu_mul(Y):
    """SiLU(gate) * up of rows [R, 2I]."""
    I = Y.shape[1] // 2
    return silu(Y[:, :I]) * Y[:, I:]


def combine(y, slots, w, residual=None):
    """(out, S) float64 [T, H] before rounding, and the sum of magnitudes."""
    y = np.asarray(y, dtype=np.float64)
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < y.shape[0]:
                term = float(w[t, j]) * y[slots[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag
