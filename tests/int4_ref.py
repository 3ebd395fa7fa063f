"""int4 weights in 64 bits on the device (torch): random ones, their values, and the
magnitudes that bound an fp32 sum's rounding. Elementary operations on float64 only."""
from __future__ import annotations

import torch

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def random_weights(gen, lead, n, group, scale_t, zeros, exact=False):
    """packed uint8 [*lead, n/2], scales [*lead, n/group], zeros uint8 or None. exact: scales are powers of two."""
    packed = torch.randint(0, 256, (*lead, n // 2), dtype=torch.uint8, device="cuda", generator=gen)
    shape = (*lead, n // group)
    if exact:
        s = torch.exp2(torch.randint(-3, 2, shape, device="cuda", generator=gen).float())
    else:
        s = (0.2 + torch.rand(shape, device="cuda", generator=gen)) * 2e-2
    s = torch.where(torch.rand(shape, device="cuda", generator=gen) < 0.3, -s, s).to(scale_t)  # a scale has any sign
    z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return packed, s, z


def values(packed, scales, zeros):
    """The matrix [rows, n] and the magnitudes scale * (code + zero) that its products are summed with."""
    n = packed.shape[-1] * 2
    code = torch.empty(*packed.shape[:-1], n, dtype=torch.float64, device=packed.device)
    code[..., 0::2] = (packed & 15).double()
    code[..., 1::2] = (packed >> 4).double()
    g = n // scales.shape[-1]
    z = torch.full_like(scales, 8, dtype=torch.float64) if zeros is None else zeros.double()
    z, s = z.repeat_interleave(g, -1), scales.double().repeat_interleave(g, -1)
    return (code - z) * s, (code + z) * s.abs()


def roundings(n, group):
    """Roundings, at most, of an output next to its sum of magnitudes: in a group 5 levels of a 32-term instruction, up
    to 12 instructions one behind the other, z times the sum; then a sum over the row's groups and 8 wavefronts."""
    return 18 + n // group + 8


def out_tolerance(want, mag, steps, t):
    f = torch.finfo(t)
    return (f.eps / 2) * want.abs() + steps * 2.0 ** -24 * (1 + f.eps) * mag + f.smallest_normal * f.eps / 2


def check(got, want, mag, steps):
    tol = out_tolerance(want, mag, steps, got.dtype)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} entries off, the worst {float((err / tol).nan_to_num(9e9).max()):.2f} "
                           f"of its tolerance, first at {bad.nonzero()[0].tolist()}")


def rows_of(gen, T, n, t, pad=0, exact=False):
    """T rows of n, `pad` entries apart, behind an odd number of entries of a buffer."""
    m = T * (n + pad) + 3
    b = torch.randint(-4, 5, (m,), device="cuda", generator=gen).float() if exact else torch.randn(m, device="cuda", generator=gen)
    return b.to(t)[3:].view(T, n + pad)[:, :n]
