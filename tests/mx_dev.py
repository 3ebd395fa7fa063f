"""The microscaled formats in 64 bits on the device (torch), for tests whose sizes numpy would take minutes for.
Elementary operations on float64 only; the format's tables are mx_ref's."""
from __future__ import annotations

import torch

from tests import mx_ref


def pow2(e):
    """2^e exactly, e an integer tensor in [-1022, 1023] (the device's pow and exp2 are off by an ulp here and there)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


BITS = {torch.float32: (24, -149), torch.bfloat16: (8, -133), torch.float16: (11, -24)}  # significand, smallest step


def rounded(x, dtype):
    """float64 values rounded once to `dtype` (to nearest, ties to even; no overflow), as float64."""
    bits, least = BITS[dtype]
    _, e = torch.frexp(x)
    ulp = pow2((e - bits).clamp(min=least))
    return torch.round(x / ulp) * ulp


def grid(x, fmt):
    """float64 [T][n] -> the values its groups take in the format (the definition the quantiser's tests use)."""
    top, bits, emin = (6.0, 2, 0) if fmt == mx_ref.FP4 else (448.0, 4, -6)  # largest, significand, lowest exponent
    g = x.reshape(x.shape[0], -1, 32)
    m = g.abs().amax(-1, keepdim=True)
    frac, e = torch.frexp(m / top)  # m = top * frac * 2^e, frac in [1/2, 1): 2^e fits, and 2^(e-1) where frac is 1/2
    e = torch.where(frac == 0.5, e - 1, e)
    e = torch.where(m == 0, -126, e).clamp(min=-126)
    v = g * pow2(-e)
    _, ev = torch.frexp(v)
    ulp = pow2((ev - bits).clamp(min=emin + 1 - bits))
    return (torch.round(v / ulp) * ulp * pow2(e)).reshape(x.shape)


def values(codes, scales, fmt):
    """Packed codes and scale bytes (device tensors) -> float64 values, 0 for a group of byte 255."""
    t = torch.from_numpy(mx_ref.MAGS[fmt]).to(codes.device)
    if fmt == mx_ref.FP4:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
        v = torch.where(c >= 8, -t[c & 7], t[c & 7])
    else:
        c = codes.int()
        v = torch.where(c >= 128, -t[c & 127], t[c & 127])
    s = scales.int().repeat_interleave(32, -1)
    return torch.where(s == 255, 0.0, v * pow2(s - 127))


def mx_bytes(gen, rows, n, fmt, lo=118, hi=132, p255=0.01):
    """Random packed codes (no NaN code) and scale bytes on the device."""
    c = torch.randint(0, 256, (rows, n // 2 if fmt == mx_ref.FP4 else n), dtype=torch.uint8, device="cuda", generator=gen)
    if fmt == mx_ref.FP8:
        c = torch.where((c & 127) == 127, c - 1, c)
    s = torch.randint(lo, hi + 1, (rows, n // 32), dtype=torch.uint8, device="cuda", generator=gen)
    s[torch.rand(s.shape, device="cuda", generator=gen) < p255] = 255
    return c, s


def placed(t, offset):
    """t's values `offset` bytes behind an allocation's start, with marked bytes around them."""
    buf = torch.full((offset + t.numel() + 64,), 0x5A, dtype=t.dtype, device=t.device)
    out = buf[offset:offset + t.numel()].view(t.shape)
    out.copy_(t)
    return out
