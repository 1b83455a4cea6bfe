"""64-bit restatement of the 8-bit KV cache and of attention over it.

value = code * 2^(byte - 127); codes are e4m3 (sign, four exponent bits of bias 7, three fraction bits, no
infinities). A vector x gets the smallest exponent e in [-40, 40] with max|x| <= 448 * 2^e.
"""
from __future__ import annotations

import numpy as np

E_LO, E_HI, BIAS, BAD, TOP = -40, 40, 127, 255, 448.0


def e4m3_values() -> np.ndarray:
    """The 256 codes' values (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[c] = np.nan if e == 15 and f == 7 else (-x if c & 128 else x)
    return v


def nearest_codes(y: np.ndarray) -> np.ndarray:
    """e4m3 codes nearest to y (ties to the even code), |y| > 448 saturated, -0 kept."""
    grid = e4m3_values()[:127]                       # 0 .. 448, increasing with the code
    a = np.minimum(np.abs(y), TOP)
    hi = np.clip(np.searchsorted(grid, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """(codes [..., d], bytes [...]) of vectors x [..., d] in float64."""
    fine = np.isfinite(x).all(-1)
    top = np.where(fine, np.abs(np.where(np.isfinite(x), x, 0)).max(-1), 0.0)
    e = np.full(top.shape, E_LO)
    for cand in range(E_LO, E_HI):                   # the smallest exponent that covers the maximum
        e = np.where(top > TOP * 2.0 ** cand, cand + 1, e)
    codes = nearest_codes(np.where(fine[..., None], x, 0.0) * 2.0 ** -e.astype(float)[..., None])
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, e + BIAS, BAD).astype(np.uint8)


def dequantise(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    s = np.where(byte == BAD, np.nan, 2.0 ** (byte.astype(float) - BIAS))
    with np.errstate(invalid="ignore"):
        return e4m3_values()[codes] * s[..., None]


def attend(q: np.ndarray, K: np.ndarray, V: np.ndarray, see: np.ndarray, scale: float):
    """One head: q [n, d], K and V [S, d], see [n, S]. Returns (out [n, d], weight [n, d] = sum p |v| / sum p,
    reach [n] = the largest sum_i |q_i k_i| * scale of a seen key). Hidden keys take no part, whatever they
    hold; a row that sees nothing gives zeros."""
    n, d = q.shape
    out, weight, reach = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n)
    for i in range(n):
        at = np.nonzero(see[i])[0]
        if at.size == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = K[at] @ q[i] * scale
            reach[i] = np.max(np.abs(K[at]) @ np.abs(q[i])) * scale
            p = np.exp(s - s.max())
            out[i] = p @ V[at] / p.sum()
            weight[i] = p @ np.abs(V[at]) / p.sum()
    return out, weight, reach
