"""fp64 oracle of the low-rank adapters, from the formula, with the error bound of a kernel that sums in fp32,
passes the product with the first matrix on as two 16-bit terms and rounds each output once.

Operands are values (fp64); formats as in oracle.attention ("f16", "bf16")."""

from __future__ import annotations

import numpy as np

from .attention import FP32, ROUNDOFF, rounding_bound


def lora(x, a, b, ids, fmt, scales=None, ranks=None, widths=None, base=None):
    """x [T][K], a [adapters][slices][rank][K], b [adapters][N][rank]; returns (out [T][N], bound [T][N])."""
    T, K = x.shape
    n, S, R, _ = a.shape
    N = b.shape[1]
    widths = [N] if widths is None else widths
    out = np.zeros((T, N)) if base is None else base.astype(np.float64).copy()
    err = np.zeros((T, N))
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < n:
            continue   # the base as it is: no bound is needed, but the rounding of an equal value is no error
        r = R if ranks is None else min(R, (max(0, int(ranks[i])) + 7) // 8 * 8)
        if r == 0:
            continue
        s = 1.0 if scales is None else float(scales[i])
        at = 0
        for j, w in enumerate(widths):
            A, B = a[i, j, :r], b[i, at:at + w, :r]
            y = A @ x[t]
            # K products summed in fp32 in any order (each partial sum at most the sum of magnitudes)
            y_err = FP32 * (K + 40) * (np.abs(A) @ np.abs(x[t]))
            # two 16-bit terms of y over a power of two in (max / 2, max]: the second's rounding, and fp16's last place
            top = np.abs(y).max() + y_err.max()
            y_err = y_err + ROUNDOFF[fmt] ** 2 * (np.abs(y) + y_err) + (2.0 ** -25 * top if fmt == "f16" else 0.0)
            mag = np.abs(B) @ (np.abs(y) + y_err)
            # twice r products and sums, the factor (two roundings) and the sum with the base
            delta = abs(s) * (np.abs(B) @ y_err + FP32 * (2 * r + 4) * mag)
            out[t, at:at + w] += s * (B @ y)
            err[t, at:at + w] = delta + FP32 * (np.abs(out[t, at:at + w]) + delta)
            at += w
    return out, rounding_bound(out, err, fmt)
