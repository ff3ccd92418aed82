"""fp64 oracle of the attention operators: norm, rotation and store into a paged cache, and
attention over it, from the formulas, plus the error bounds of a kernel that computes in fp32
and rounds its results (and softmax weights) to 16 bits.

16-bit values are exchanged as uint16 bit patterns ("f16", "bf16"), e4m3 values as uint8 codes
("fp8"), so nothing here depends on another library's conversions.
"""

from __future__ import annotations

import numpy as np

# unit roundoff and the spacing of the smallest values
ROUNDOFF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp8": 2.0 ** -4}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "fp8": 2.0 ** -9}
FP32 = 2.0 ** -24
FP8_MAX = 448.0


# --------------------------------------------------------------------------------- number formats
def _e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = np.nan
        t[c] = -x if s else x
    return t


E4M3 = _e4m3_table()


def decode(bits, fmt: str):
    """The values (fp64) of bit patterns."""
    bits = np.asarray(bits)
    if fmt == "fp8":
        return E4M3[bits.astype(np.uint8)]
    if fmt == "bf16":
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return bits.astype(np.uint16).view(np.float16).astype(np.float64)


def encode(x, fmt: str):
    """Bit patterns of fp64 values, rounded to nearest even (e4m3: saturated)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "f16":
        return x.astype(np.float16).view(np.uint16)
    if fmt == "bf16":
        b = x.astype(np.float32).view(np.uint32)
        r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
        return np.where(np.isnan(x), np.uint16(0x7FC0), r)
    pos = E4M3[:127]
    a = np.minimum(np.abs(x), FP8_MAX)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(x), 127, c)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


# ------------------------------------------------------------------------------ norm and rotation
def norm_rotate(x, weight, eps: float, angles, interleaved: bool):
    """x [heads][dim] fp64, weight [dim] or None, angles: (cos, sin) of the rotated pairs, each [rot/2].
    Returns the result and the bound of an fp32 computation's error before any rounding of the result."""
    D = x.shape[1]
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps) * weight
    # sum of D squares (D roundings), division, addition, square root, reciprocal, two products
    err = FP32 * (D / 2 + 8) * np.abs(y) if weight is not None else np.zeros_like(y)
    out, bound = y.copy(), err.copy()
    cos, sin = angles
    half = len(cos)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[:, a] = y[:, a] * cos - y[:, b] * sin
    out[:, b] = y[:, b] * cos + y[:, a] * sin
    mag = np.abs(y[:, a]) + np.abs(y[:, b])
    turn = err[:, a] + err[:, b] + 3 * FP32 * mag
    bound[:, a] = turn
    bound[:, b] = turn
    return out, bound


def rounding_bound(ref, computed, fmt: str):
    """Bound of |result - ref| for a value computed within `computed` of ref and rounded to fmt."""
    return computed + ROUNDOFF[fmt] * (np.abs(ref) + computed) + TINY[fmt] / 2


# ------------------------------------------------------------------------------------- attention
def visible(pos: int, length: int, window: int, sinks: int):
    """Truth value per cached token: what a query at position `pos` sees."""
    j = np.arange(length)
    see = j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    return see


def attend(q, k, v, see, scale: float):
    """q [heads][dim], k and v [tokens][heads][dim] (fp64, one per query head), see [tokens].
    Returns (out [heads][dim], sum of weights times |v|, bound of a score's fp32 error per head)."""
    H, D = q.shape
    if not see.any():
        return np.zeros((H, D)), np.zeros((H, D)), np.zeros((H, 1))
    k, v = k[see], v[see]
    s = np.einsum("hd,nhd->hn", q, k) * scale
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    mag = np.einsum("hd,nhd->hn", np.abs(q), np.abs(k)).max(axis=1, keepdims=True) * scale
    # D products and sums, the scaling to log2 units, the subtraction of the maximum
    score_err = FP32 * ((D + 4) * mag + 2 * np.abs(s).max(axis=1, keepdims=True))
    return np.einsum("hn,nhd->hd", w, v), np.einsum("hn,nhd->hd", w, np.abs(v)), score_err


def attention_bound(ref, mag, score_err, tokens: int, fmt: str, weight_roundoff: float):
    """Bound of an output's error: the output's rounding, and relative errors of the weights (their
    rounding, twice the score's error, exp2 and the sums over the tokens in fp32) times sum w |v|."""
    weights = weight_roundoff + 2 * 1.01 * score_err + FP32 * (2 * tokens + 32)
    return rounding_bound(ref, weights * mag, fmt)
