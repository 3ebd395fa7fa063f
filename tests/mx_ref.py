"""The microscaled formats and their products in 64 bits (numpy), for the tests:
codes from values, values from codes, and the tolerances of fp32 sums."""
from __future__ import annotations

import numpy as np

FP4, FP8 = 0, 1
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
MAX = {FP4: 6.0, FP8: 448.0}


def e4m3_table():
    c = np.arange(128)
    e, m = c >> 3, (c & 7) / 8
    v = np.where(e > 0, (1 + m) * 2.0 ** (e - 7), m * 2.0 ** -6)
    v[127] = np.nan
    return v


MAGS = {FP4: E2M1, FP8: e4m3_table()}


def exponent(m, fmt):
    """Smallest e >= -126 with m <= M 2^e (m >= 0, finite), by comparing."""
    m = np.asarray(m, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(m > 0, np.ceil(np.log2(np.where(m > 0, m, 1) / MAX[fmt])), -126.0)
    e = np.where((m > 0) & (MAX[fmt] * 2.0 ** (e - 1) >= m), e - 1, e)
    e = np.where((m > 0) & (MAX[fmt] * 2.0 ** e < m), e + 1, e)
    return np.maximum(e, -126).astype(np.int64)


def nearest_code(v, fmt):
    """Index of the nearest magnitude, ties to the even code (v >= 0, at most M)."""
    t = MAGS[fmt] if fmt == FP4 else MAGS[fmt][:127]
    hi = np.searchsorted(t, v)  # t[hi - 1] < v <= t[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - t[lo], t[hi] - v
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantize(x, fmt):
    """x [T][n] float64 -> (codes uint8 [T][n] one a byte, scale bytes uint8 [T][n/32])."""
    x = np.asarray(x, np.float64)
    T, n = x.shape
    g = x.reshape(T, n // 32, 32)
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    e = exponent(np.abs(g).max(-1), fmt)
    c = nearest_code(np.abs(g) * 2.0 ** -e[..., None].astype(np.float64), fmt)
    sign = (np.signbit(g) & fine[..., None]).astype(np.int64) << (3 if fmt == FP4 else 7)
    return (c | sign).astype(np.uint8).reshape(T, n), np.where(fine, e + 127, 255).astype(np.uint8)


def pack(codes, fmt):
    return codes if fmt == FP8 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed, fmt):
    if fmt == FP8:
        return packed
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)


def values(packed, scales, fmt):
    """Packed codes and scale bytes -> float64 values (a group of byte 255: 0)."""
    c = unpack(np.asarray(packed), fmt).astype(np.int64)
    bits = 3 if fmt == FP4 else 7
    v = MAGS[fmt][c & ((1 << bits) - 1)] * np.where(c >> bits, -1.0, 1.0)
    s = np.repeat(np.asarray(scales).astype(np.float64), 32, -1)
    return np.where(s == 255, 0.0, v * 2.0 ** (s - 127))


def product(a, w, b=None):
    """a w^T and sum |a||w|, float64 (a [T][n], w [N][n] values)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def half_step(v, e, fmt):
    """Half the distance between the codes around |v| (v a value, e the group's exponent)."""
    a = np.abs(v) * 2.0 ** -e.astype(np.float64)
    t = MAGS[fmt] if fmt == FP4 else MAGS[fmt][:127]
    hi = np.clip(np.searchsorted(t, a), 1, len(t) - 1)
    return 0.5 * (t[hi] - t[hi - 1]) * 2.0 ** e.astype(np.float64)


def check_quantised(packed, scales, ref, tol, fmt, what):
    """q is the quantisation of some fp32 row within `tol` (per entry) of `ref`: every group's exponent is that of a
    largest entry within tol of ref's, and every value within tol and half a step of ref."""
    T, n = ref.shape
    s = np.asarray(scales).astype(np.int64)
    assert np.all(s < 255), f"{what}: a group of finite values marked as not finite"
    m = np.abs(ref).reshape(T, -1, 32)
    t = np.broadcast_to(tol, ref.shape).reshape(T, -1, 32)
    lo, hi = exponent(np.maximum(m - t, 0).max(-1), fmt), exponent((m + t).max(-1), fmt)
    assert np.all((s - 127 >= lo) & (s - 127 <= hi)), f"{what}: scale bytes off"
    e = np.repeat(s - 127, 32, -1)
    v = values(packed, scales, fmt)
    # the step is that of the interval the fp32 value lies in: the one around ref or, within tol of a border, its neighbour
    step = np.maximum(half_step(np.abs(ref) + tol, e, fmt), half_step(np.maximum(np.abs(ref) - tol, 0), e, fmt))
    bad = np.abs(v - ref) > step + tol
    assert not bad.any(), f"{what}: {bad.sum()} values off, first {np.argwhere(bad)[:3].tolist()}"


def mx_bytes(rng, rows, n, fmt, lo=118, hi=132, p255=0.0):
    """Random packed codes (no NaN code) and scale bytes."""
    if fmt == FP4:
        codes = rng.integers(0, 256, (rows, n // 2), dtype=np.uint8)
    else:
        codes = rng.integers(0, 256, (rows, n), dtype=np.uint8)
        codes = np.where((codes & 127) == 127, codes - 1, codes).astype(np.uint8)
    s = rng.integers(lo, hi + 1, (rows, n // 32), dtype=np.uint8)
    s[rng.random(s.shape) < p255] = 255
    return codes, s
