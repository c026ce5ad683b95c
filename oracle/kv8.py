"""Plain definitions of the 8-bit cache (numpy): its codes, its blocks, and
attention over it in 64 bits with what its roundings may add up to.  Shares
no code with the CUDA path."""
from __future__ import annotations

import numpy as np

PAGE = 16
TOP = {"e4m3": np.float32(448.0), "int8": np.float32(127.0)}


def e4m3_values() -> np.ndarray:
    """The values of codes 0x00 .. 0x7e (0x7f is NaN)."""
    c = np.arange(0x7f)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def encode(y, code):
    """Nearest codes (ties to even) of values within [-top, top]: uint8."""
    y = np.asarray(y, dtype=np.float64)
    if code == "int8":
        return np.rint(y).astype(np.int8).view(np.uint8)
    v = e4m3_values()
    a = np.abs(y)
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)
    lo = hi - 1
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def decode(codes, code) -> np.ndarray:
    """The values that codes (uint8) stand for; NaN codes of e4m3 as NaN."""
    codes = np.asarray(codes, dtype=np.uint8)
    if code == "int8":
        return codes.view(np.int8).astype(np.float64)
    v = np.append(e4m3_values(), np.nan)
    return np.where(codes & 0x80, -1.0, 1.0) * v[codes & 0x7f]


def block(x, code):
    """One block [16][d] (fp32 values): (codes uint8 [16][d], scale fp32,
    whether it held infinities or NaN)."""
    x = np.array(x, dtype=np.float32)
    odd = ~np.isfinite(x)
    top, one = TOP[code], np.float32(1.0)
    amax = np.max(np.where(odd, np.float32(0), np.abs(x)))
    scale = np.maximum(amax * (one / top), np.float32(2.0 ** -126))
    x[np.isnan(x)] = 0.0
    with np.errstate(over="ignore"):
        y = np.clip(x * (one / scale), -top, top)
    return encode(y, code), scale, bool(odd.any())


def attn(q, k, v, seen, scale, v_top):
    """q [rows][d], k and v [keys][d] (values), seen [rows][keys] truth
    values, all in 64 bits; v_top: the largest scale of V times its code's top.
    Returns (out [rows][d], bound of the kernel's error beside it).

    The bound: a probability enters the second product in fp16, off by half a
    step, 2^-11 of itself, or by 2^-25 where it is smaller than fp16's normal
    numbers, of values that are relative to at most twice the largest scale and
    in which the largest probability is at least 2^8.  A score
    is a sum of head_dim products in fp32: off by at most D 2^-23 of sum |q k|
    scale; and by 2^-21 of itself and of the maximum for the factors and the
    subtraction, each of which moves p by as much relatively, in numerator and
    denominator (twice).  exp2 and the sums add below 2^-12 (sums of up to 2^11
    terms a chain, joined)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    s = (q @ k.T) * scale
    mag = (np.abs(q) @ np.abs(k).T) * scale
    e = np.where(seen, s, -np.inf)
    m = e.max(-1, keepdims=True)
    some = np.isfinite(m)
    p = np.where(seen, np.exp(e - np.where(some, m, 0.0)), 0.0)
    l = p.sum(-1, keepdims=True)
    ln = np.where(l > 0, l, 1.0)
    out = (p @ v) / ln
    spread = (p @ np.abs(v)) / ln
    d = q.shape[1]
    shift = np.where(seen, mag, 0.0).max(-1, keepdims=True) * (d * 2.0 ** -23 + 2.0 ** -20)
    few = 2.0 ** -25 * 2.0 / 2.0 ** 8 * v_top * (p > 0).sum(-1, keepdims=True) / ln
    return out, spread * (2.0 ** -11 + 2.0 ** -12 + 2 * shift) + few
