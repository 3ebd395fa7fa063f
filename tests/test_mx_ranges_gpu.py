"""Microscaled products at the ends of the formats' and fp32's ranges (GPU, 64-bit references): scale bytes 0 to 254 on
either side, results in fp32's subnormal numbers and past its largest, NaN codes. Streamed and tiled.

The bar is the library's 1e-5 * sum |a||w|, and for subnormal results half their step for each of the additions of a
sum (an MFMA step of 128 entries adds at most 32 partial sums to a result, lo and hi of an e4m3 operand twice that).
"""
import pytest

from tests import mx_dev
from tests.helpers import REL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SHAPES = [(3, 70, 512), (40, 10240, 512), (40, 10240, 480)]  # streamed; 128 x 32 tiles; odd scales


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def operands(k3g, seed, T, rows, n, fmt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ac, asc = mx_dev.mx_bytes(g, T, n, fmt, p255=0)
    wc, wsc = mx_dev.mx_bytes(g, rows, n, 0, p255=0)
    return g, ac, asc, wc, wsc


def product(k3g, ac, asc, wc, wsc, fmt):
    y = torch.empty(ac.shape[0], wc.shape[0], device="cuda")
    k3g.k3g_mx_matmul(y, k3g.mx(ac, asc, fmt), k3g.mxfp4(wc, wsc))
    a, w = mx_dev.values(ac, asc, fmt), mx_dev.values(wc, wsc, 0)
    return y, a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,rows,n", SHAPES)
def test_every_scale_byte_on_both_sides(k3g, T, rows, n, fmt):
    """2^(s-127) on one side and 2^(127-s) on the other, s from 0 to 254 over the groups."""
    g, ac, asc, wc, wsc = operands(k3g, 1, T, rows, n, fmt)
    G = n // 32
    for first in range(0, 255, G):
        s = torch.arange(first, first + G, device="cuda").clamp(max=254)
        asc[:], wsc[:] = s.to(torch.uint8), (254 - s).to(torch.uint8)
        print(f"scales from {first} T={T} n={n} fmt={fmt}", flush=True)
        y, ref, nrm = product(k3g, ac, asc, wc, wsc, fmt)
        assert bool(((y.double() - ref).abs() <= REL * nrm).all()), f"bytes from {first}"


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,rows,n", SHAPES)
def test_results_below_fp32s_normal_numbers(k3g, T, rows, n, fmt):
    g, ac, asc, wc, wsc = operands(k3g, 2, T, rows, n, fmt)
    for total in (-126, -132, -140, -146):  # the exponent of both scales together
        sa = torch.randint(0, 127, asc.shape, device="cuda", generator=g)
        sa[:] = sa[:1]
        asc[:], wsc[:] = sa.to(torch.uint8), (254 + total - sa[:1]).clamp(0, 254).to(torch.uint8)
        print(f"2^{total} T={T} n={n} fmt={fmt}", flush=True)
        y, ref, nrm = product(k3g, ac, asc, wc, wsc, fmt)
        bad = ~((y.double() - ref).abs() <= REL * nrm + (2 if fmt else 1) * 32 * ((n + 127) // 128) * 2.0 ** -150)
        assert not bool(bad.any()), f"2^{total}: {int(bad.sum())} of {bad.numel()} off: {y[bad][:3].tolist()} for {ref[bad][:3].tolist()}"


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,rows,n", SHAPES)
def test_results_past_fp32s_largest_number(k3g, T, rows, n, fmt):
    """All products of one sign: past the largest number the sum is that infinity."""
    g, ac, asc, wc, wsc = operands(k3g, 3, T, rows, n, fmt)
    ac &= 0x77 if fmt == 0 else 0x7F
    wc &= 0x77
    wc[::2] |= 0x88  # every other row's weights negative
    asc[:], wsc[:] = 250, 130 if fmt == 0 else 124
    asc[0] = 127
    y, ref, nrm = product(k3g, ac, asc, wc, wsc, fmt)
    top = float(torch.finfo(torch.float32).max)
    over, under = ref.abs() > top * (1 + 2 * REL), ref.abs() < top * (1 - 2 * REL)
    assert bool(over.any()) and bool(under.any())
    assert bool((y[over].double() == torch.sign(ref[over]) * float("inf")).all())
    assert bool(((y.double() - ref).abs() <= REL * nrm)[under].all())


@pytest.mark.parametrize("T,rows,n", SHAPES)
def test_nan_codes(k3g, T, rows, n):
    """An e4m3 NaN code makes its token's results NaN, and none where its group's byte is 255."""
    g, ac, asc, wc, wsc = operands(k3g, 4, T, rows, n, 1)
    ac[0, 37], ac[1, n - 1], ac[2, 40] = 0x7F, 0xFF, 0x7F
    asc[2, 1] = 255
    y, _, _ = product(k3g, ac, asc, wc, wsc, 1)
    assert bool(torch.isnan(y[:2]).all())
    ac[2, 40] = 0
    want, ref, nrm = product(k3g, ac, asc, wc, wsc, 1)
    assert torch.equal(y[2:], want[2:]) and bool(((y.double() - ref).abs() <= REL * nrm)[2:].all())


@pytest.mark.parametrize("T,rows", [(3, 70), (40, 10240)])
@pytest.mark.parametrize("kind", ["large", "small", "both", "scales"])
def test_unlike_products_of_one_sum(k3g, T, rows, kind):
    """One product far above the others of its eight, of its group or of its step: the small ones still count. (Codes
    from 2 on beside 448, below 2 beside 2^-9, and groups 2^-14 apart.)"""
    n = 512
    g = torch.Generator(device="cuda").manual_seed(5)

    def pick(codes, share, *shape):
        i = torch.multinomial(torch.tensor(share, device="cuda"), shape[0] * shape[1], True, generator=g)
        return torch.tensor(codes, dtype=torch.uint8, device="cuda")[i].view(shape)
    # 0x7E 448, 0x41 2.25, 0x3F 1.875, 0x01 2^-9, 0x03 3 * 2^-9
    codes, share = {"large": ([0x7E, 0x41], [0.05, 0.95]), "small": ([0x3F, 0x01, 0x03], [0.05, 0.5, 0.45]),
                    "both": ([0x7E, 0x41, 0x3F, 0x01, 0x03], [0.02, 0.4, 0.08, 0.3, 0.2]),
                    "scales": ([0x7E], [1.0])}[kind]
    ac = pick(codes, share, T, n)
    asc = torch.full((T, n // 32), 127, dtype=torch.uint8, device="cuda")
    if kind == "scales":
        asc[:] = 113
        asc[:, 1::4] = 127
        ac.view(T, -1, 32)[:, 1::4, 1:] = 0
    wn = pick([1, 3, 7], [0.8, 0.1, 0.1], rows, n)
    wc = wn[:, 0::2] | (wn[:, 1::2] << 4)
    wsc = torch.full((rows, n // 32), 127, dtype=torch.uint8, device="cuda")
    y, ref, nrm = product(k3g, ac, asc, wc, wsc, 1)
    assert bool(((y.double() - ref).abs() <= REL * nrm).all())
