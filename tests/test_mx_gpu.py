"""The microscaled-activation operators on the GPU against 64-bit references.

Tolerances. The quantiser and the way back are exact (power-of-two scalings and
one rounding): codes, scale bytes and values are compared bit for bit. A product's
terms are exact in fp32 and its sum has at most K fp32 additions, but the bar is
the library's own 1e-5 * sum |a||w|, plus half a step of the output's type
(bf16 2^-9 of a value, doubled at a power of two: 2^-8; fp16 2^-11). The norm:
s and n take a rounding each, the mean's sum at most 8 * 8 + 6 + 16 fp32
additions of positive terms (half of that in its root), the root and the
division 2 ulp each: below 64 * 2^-24 of the value.
"""
import numpy as np
import pytest

from tests import mx_ref
from tests.helpers import REL, situ64, situ_tolerance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FMTS = [0, 1]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
NORM = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    t = t.detach().cpu()
    return t.float().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.numpy()


def strided(T, n, dtype, pad, fill=float("nan")):
    """Rows of n entries in a buffer n + pad wide, 1 entry in; the buffer, and the rows."""
    buf = torch.full((T, n + pad), fill, dtype=dtype, device="cuda")
    return buf, buf[:, min(1, pad):min(1, pad) + n]


# ---- quantiser and back ----------------------------------------------------------------

def quantiser_rows(T, n, seed):
    """Rows with every kind of group: normals at many magnitudes, zeros, signed zeros, ties, borders of the exponent,
    subnormals, the largest numbers, infinities and NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, n)) * 2.0 ** rng.integers(-30, 30, (T, n // 32)).repeat(32, 1)
    x = x.astype(np.float32).reshape(-1, 32)
    kinds = rng.integers(0, 14, len(x))
    for i, k in enumerate(kinds):
        s = np.float32(2.0 ** rng.integers(-20, 20))
        if k == 0:
            x[i] = 0.0
            x[i, ::3] = -0.0
        elif k == 1:  # ties of both formats
            x[i] = s * rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0], np.float32), 32)
            x[i, 0] = 6 * s
        elif k == 2:  # largest entry on the border, and one ulp above it
            x[i] *= 0
            x[i, 5] = s * np.float32(rng.choice([6, 448]))
            if rng.random() < 0.5:
                x[i, 5] = np.nextafter(x[i, 5], np.float32(np.inf))
        elif k == 3:
            x[i] = np.float32(1e-42) * rng.integers(-9, 9, 32)
        elif k == 4:
            x[i] = np.float32(3.4e38) * rng.uniform(-1, 1, 32).astype(np.float32)
        elif k == 5:
            x[i, 7] = rng.choice([np.inf, -np.inf, np.nan])
        elif k == 6:  # one large entry among small ones
            x[i, 9] *= 1000
        elif k == 7:  # near the floor of the exponent
            x[i] = (rng.standard_normal(32) * 2.0 ** -125).astype(np.float32)
    return x.reshape(T, n)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,n,pad", [(1, 32, 0), (3, 64, 5), (64, 96, 0), (7, 2080, 32), (130, 7168, 0), (2, 65536, 0)])
def test_quantize_bit_exact(k3g, T, n, pad, ty, fmt):
    print(f"quantize T={T} n={n} pad={pad} {ty} fmt={fmt}", flush=True)
    buf, x = strided(T, n, TYPES[ty], pad)
    with np.errstate(over="ignore"):
        x.copy_(torch.from_numpy(quantiser_rows(T, n, T + n)))
    q = k3g.mx_empty(T, n, fmt)
    k3g.k3g_mx_quantize(q, x)
    c, s = mx_ref.quantize(host(x).astype(np.float64), fmt)
    assert np.array_equal(host(q.scales), s)
    assert np.array_equal(mx_ref.unpack(host(q.codes), fmt), c)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_dequantize_bit_exact(k3g, ty, fmt, pad):
    # every code under every scale byte (fp32 holds each product exactly or overflows to infinity)
    n = 256 if fmt else 32
    codes = np.tile(np.arange(256 if fmt else 16, dtype=np.uint8), (256, 1 if fmt else 2))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], n // 32, 1)
    print(f"dequantize {ty} fmt={fmt} pad={pad}", flush=True)
    q = k3g.mx(dev(mx_ref.pack(codes, fmt)), dev(scales), fmt)
    buf, y = strided(256, n, TYPES[ty], pad, 7.0)
    k3g.k3g_mx_dequantize(y, q)
    with np.errstate(over="ignore"):
        ref = mx_ref.values(mx_ref.pack(codes, fmt), scales, fmt).astype(np.float32)
    ref = torch.from_numpy(ref).to(TYPES[ty])
    assert np.array_equal(host(y), host(ref), equal_nan=True)
    if pad:
        assert (host(buf)[:, n + 1:] == 7.0).all() and (host(buf)[:, 0] == 7.0).all()


# ---- residual + norm -----------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [None, 0, 1])
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,n,pad,res", [(1, 32, 0, True), (3, 96, 7, True), (64, 7168, 0, True), (5, 3584, 0, False),
                                         (2, 8224, 0, True), (2, 16416, 1, True), (1, 65536, 0, True), (300, 256, 0, False)])
def test_add_rmsnorm(k3g, T, n, pad, res, ty, fmt):
    print(f"norm T={T} n={n} pad={pad} res={res} {ty} fmt={fmt}", flush=True)
    rng = np.random.default_rng(n + T)
    _, x = strided(T, n, TYPES[ty], pad)
    _, r = strided(T, n, TYPES[ty], pad + 2 if pad else 0)
    x.copy_(torch.from_numpy(rng.standard_normal((T, n)).astype(np.float32)))
    r.copy_(torch.from_numpy((3 * rng.standard_normal((T, n))).astype(np.float32)))
    gamma = rng.uniform(0.5, 1.5, n).astype(np.float32)
    eps = 1e-5
    _, y = strided(T, n, TYPES[ty], pad)
    _, sm = strided(T, n, TYPES[ty], pad)
    q = k3g.mx_empty(T, n, fmt) if fmt is not None else None
    k3g.k3g_add_rmsnorm(x, dev(gamma), eps, r=r if res else None, sum=sm, y=y, q=q)
    s = host(x).astype(np.float64) + (host(r).astype(np.float64) if res else 0.0)
    ref = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * gamma
    assert np.all(np.abs(host(sm) - s) <= (HALF[ty] + 2.0 ** -24) * np.abs(s) + 1e-7)
    assert np.all(np.abs(host(y) - ref) <= (HALF[ty] + NORM) * np.abs(ref) + 2.0 ** -25)
    if fmt is not None:
        mx_ref.check_quantised(host(q.codes), host(q.scales), ref, NORM * np.abs(ref), fmt, "norm")


def test_add_rmsnorm_in_place_and_special_rows(k3g):
    rng = np.random.default_rng(3)
    n = 512
    x = rng.standard_normal((6, n)).astype(np.float32)
    r = rng.standard_normal((6, n)).astype(np.float32)
    x[1], r[1] = 0, 0            # zeros: n = 0
    x[2], r[2] = 1e-30, 0        # eps decides
    x[3, 5] = np.inf             # the row's infinity is a NaN, its other entries 0
    x[4, 7] = np.nan             # everything is a NaN
    g = np.ones(n, np.float32)
    xd, rd = dev(x), dev(r)
    q = k3g.mx_empty(6, n, k3g.MXFP8)
    k3g.k3g_add_rmsnorm(xd, dev(g), 1e-5, r=rd, sum=rd, y=xd, q=q)  # the sum over r, the norm over x
    with np.errstate(invalid="ignore"):
        s = x.astype(np.float64) + r
        ref = s / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5)
    assert np.array_equal(host(rd), (x + r), equal_nan=True)
    y = host(xd)
    ok = [0, 1, 2, 5]
    assert np.all(np.abs(y[ok] - ref[ok]) <= (NORM + 2.0 ** -24) * np.abs(ref[ok]))
    assert np.isnan(y[3, 5]) and np.all(np.delete(y[3], 5) == 0) and np.isnan(y[4]).all()
    sc = host(q.scales)
    assert sc[3, 0] == 255 and np.all(sc[3, 1:] == 1) and np.all(sc[4] == 255) and np.all(sc[1] == 1)
    assert np.all(host(q.codes)[4] == 0)


# ---- dense products ------------------------------------------------------------------------

def check_product(got, ref, nrm, ty, what):
    tol = REL * nrm + HALF[ty] * (np.abs(ref) + REL * nrm)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off; first {np.argwhere(bad)[:3].tolist()}: "
                           f"{got[bad][:3]} for {ref[bad][:3]}")
    assert np.all(got[nrm == 0] == 0), f"{what}: nonzero where every group is left out"


DENSE = [
    # T, rows, in, output columns beyond rows, share of 255 bytes
    (1, 1, 32, 0, 0.0),
    (1, 33, 96, 3, 0.1),
    (2, 64, 128, 0, 0.3),
    (15, 17, 160, 1, 0.05),
    (16, 256, 512, 0, 0.01),
    (17, 100, 224, 0, 0.05),
    (31, 3584, 7168, 0, 0.001),
    (33, 130, 1056, 4, 0.05),
    (64, 512, 992, 0, 0.01),
    (65, 257, 3584, 0, 0.01),
    (129, 384, 480, 0, 0.02),
    (256, 256, 256, 0, 0.01),
    (300, 515, 1184, 5, 0.01),
    (520, 1030, 320, 0, 0.01),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,rows,n,pad,p255", DENSE)
def test_matmul(k3g, T, rows, n, pad, p255, fmt):
    rng = np.random.default_rng(T * 1000 + rows)
    ac, asc = mx_ref.mx_bytes(rng, T, n, fmt, p255=p255)
    wc, wsc = mx_ref.mx_bytes(rng, rows, n, 0, p255=p255)
    if T > 3:
        asc[2] = 255  # a token of left-out groups
    if rows > 20:
        wsc[5] = 255
    ref, nrm = mx_ref.product(mx_ref.values(ac, asc, fmt), mx_ref.values(wc, wsc, 0))
    a, w = k3g.mx(dev(ac), dev(asc), fmt), k3g.mxfp4(dev(wc), dev(wsc))
    for ty in TYPES:
        if ty == "f16" and T != 33:
            continue
        print(f"matmul T={T} rows={rows} in={n} pad={pad} fmt={fmt} {ty}", flush=True)
        scale = 1.0
        buf, y = strided(T, rows, TYPES[ty], pad, 7.0)
        if ty == "f16":  # keep the values inside fp16's range
            wd = np.where(wsc == 255, 255, wsc.astype(int) - 12).astype(np.uint8)
            w16 = k3g.mxfp4(dev(wc), dev(wd))
            scale = 2.0 ** -12
        k3g.k3g_mx_matmul(y, a, w16 if ty == "f16" else w, )
        got = host(y).astype(np.float64)
        if ty == "f16":  # its subnormal step as well
            assert np.all(np.abs(got - ref * scale) <= scale * REL * nrm + HALF[ty] * np.abs(ref * scale) * 1.01 + 2.0 ** -25)
        else:
            check_product(got, ref, nrm, ty, f"matmul {T}x{rows}x{n}")
        if pad:
            b = host(buf)
            assert (b[:, rows + 1:] == 7.0).all() and (b[:, 0] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_full_range_of_scales(k3g, fmt):
    # bytes from 2^-127 to 2^127 on both sides wherever the product stays in fp32's normal range
    rng = np.random.default_rng(5)
    T, rows, n = 40, 48, 512
    ac, asc = mx_ref.mx_bytes(rng, T, n, fmt)
    wc, wsc = mx_ref.mx_bytes(rng, rows, n, 0)
    up = rng.integers(20, 235, (1, n // 32))
    asc[:], wsc[:] = up, 254 - up
    ref, nrm = mx_ref.product(mx_ref.values(ac, asc, fmt), mx_ref.values(wc, wsc, 0))
    y = torch.empty(T, rows, device="cuda")
    print(f"scales fmt={fmt}", flush=True)
    k3g.k3g_mx_matmul(y, k3g.mx(dev(ac), dev(asc), fmt), k3g.mxfp4(dev(wc), dev(wsc)))
    check_product(host(y).astype(np.float64), ref, nrm, "f32", "scales")


def test_matmul_scales_at_any_address(k3g):
    # scale tensors have no alignment: a weight's and an activation's at odd addresses
    rng = np.random.default_rng(6)
    for T, rows, n in ((3, 70, 384), (200, 300, 384)):
        ac, asc = mx_ref.mx_bytes(rng, T, n, 0, p255=0.02)
        wc, wsc = mx_ref.mx_bytes(rng, rows, n, 0, p255=0.02)
        place = lambda s, o: torch.cat([torch.zeros(o, dtype=torch.uint8), torch.from_numpy(s.ravel())]).cuda()[o:].view(s.shape)  # noqa: E731
        ref, nrm = mx_ref.product(mx_ref.values(ac, asc, 0), mx_ref.values(wc, wsc, 0))
        y = torch.empty(T, rows, device="cuda")
        print(f"odd addresses T={T}", flush=True)
        k3g.k3g_mx_matmul(y, k3g.mx(dev(ac), place(asc, 1), 0), k3g.mxfp4(dev(wc), place(wsc, 3)))
        check_product(host(y).astype(np.float64), ref, nrm, "f32", "odd addresses")


def test_empty_calls(k3g):
    n = 64
    for fmt in FMTS:
        q = k3g.mx_empty(0, n, fmt)
        x = torch.empty(0, n, device="cuda")
        k3g.k3g_mx_quantize(q, x)
        k3g.k3g_mx_dequantize(x, q)
        k3g.k3g_add_rmsnorm(x, torch.ones(n, device="cuda"), 1e-5, q=q)
        k3g.k3g_mx_matmul(torch.empty(0, 4, device="cuda"), q, k3g.mxfp4(torch.zeros(4, 32, dtype=torch.uint8, device="cuda"),
                                                                         torch.zeros(4, 2, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()


# ---- grouped products ------------------------------------------------------------------------

class Experts:
    """A bank of E experts of random bytes and their float64 values."""

    def __init__(self, k3g, rng, E, latent, inter, lo=118, hi=132, p255=0.01, tail=0):
        self.E, self.latent, self.inter = E, latent, inter
        off, stride = k3g.bank_layout(latent, inter)
        stride += tail
        bank = np.zeros((E, stride), np.uint8)
        self.w = []
        for t, (rows, cols) in enumerate(((inter, latent), (inter, latent), (latent, inter))):
            per = []
            for e in range(E):
                c, s = mx_ref.mx_bytes(rng, rows, cols, 0, lo, hi, p255)
                bank[e, off[2 * t]:off[2 * t] + c.size] = c.ravel()
                bank[e, off[2 * t + 1]:off[2 * t + 1] + s.size] = s.ravel()
                per.append(mx_ref.values(c, s, 0))
            self.w.append(per)
        self.bank = dev(bank.ravel())
        self.struct = k3g.bank_struct(self.bank, E, latent, inter, off, stride)


def ragged(rng, E, P, lead=0, behind=0, empty=0.3):
    """offsets of E groups over P rows, some empty, `lead` rows before the first and `behind` after the last."""
    p = rng.random(E) * (rng.random(E) > empty)
    p[rng.integers(0, E)] += 0.5
    counts = rng.multinomial(P - lead - behind, p / p.sum())
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)


GROUPED = [
    # E, latent, inter, tokens, top_k, rows before, rows behind
    (1, 32, 32, 1, 1, 0, 0),
    (3, 96, 64, 2, 2, 0, 0),
    (8, 256, 160, 5, 4, 1, 2),
    (70, 128, 96, 40, 3, 0, 5),
    (5, 544, 288, 100, 3, 3, 0),
    (130, 64, 128, 9, 8, 0, 0),
    (4, 512, 384, 300, 2, 0, 7),
    (2, 224, 1056, 500, 1, 2, 2),
    (2048, 32, 32, 64, 2, 0, 0),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,latent,inter,T,k,lead,behind", GROUPED)
def test_grouped_matmul(k3g, E, latent, inter, T, k, lead, behind, fmt):
    rng = np.random.default_rng(E * 100 + T)
    ex = Experts(k3g, rng, E, latent, inter, tail=256)
    P = T * k
    off = ragged(rng, E, P, lead, behind)
    for tensor, ty, gather in ((k3g.W2, "f32", False), (k3g.W1, "bf16", True), (k3g.W3, "f32", True)):
        rows, cols = (latent, inter) if tensor == k3g.W2 else (inter, latent)
        n_a = T if gather else P
        ac, asc = mx_ref.mx_bytes(rng, n_a, cols, fmt, p255=0.02)
        perm = rng.permutation(P).astype(np.int32)
        av = mx_ref.values(ac, asc, fmt)
        _, y = strided(P, rows, TYPES[ty], 0, 7.0)
        print(f"grouped E={E} {rows}x{cols} P={P} fmt={fmt} {ty} gather={gather}", flush=True)
        k3g.k3g_mx_grouped_matmul(y, k3g.mx(dev(ac), dev(asc), fmt), ex.struct, tensor, dev(off),
                                  perm=dev(perm) if gather else None, top_k=k)
        got = host(y).astype(np.float64)
        for e in range(E):
            p = np.arange(off[e], off[e + 1])
            if p.size:
                ref, nrm = mx_ref.product(av[perm[p] // k if gather else p], ex.w[tensor][e])
                check_product(got[p], ref, nrm, ty, f"expert {e}")
        left = np.r_[np.arange(off[0]), np.arange(off[-1], P)]
        assert np.all(got[left] == 7.0), "rows outside the groups were written"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hfmt", FMTS)
@pytest.mark.parametrize("E,latent,inter,T,k,lead,behind", GROUPED)
def test_grouped_glu(k3g, E, latent, inter, T, k, lead, behind, hfmt, fmt):
    rng = np.random.default_rng(E * 100 + T + 7)
    ex = Experts(k3g, rng, E, latent, inter, 110, 118)
    P = T * k
    off = ragged(rng, E, P, lead, behind)
    ac, asc = mx_ref.mx_bytes(rng, T, latent, fmt, 118 if fmt == 0 else 112, 126 if fmt == 0 else 118, p255=0.02)
    perm = rng.permutation(P).astype(np.int32)
    h = k3g.mx_empty(P, inter, hfmt)
    h.codes.fill_(77), h.scales.fill_(9)
    print(f"glu E={E} {inter}x{latent} P={P} fmt={fmt} h={hfmt}", flush=True)
    k3g.k3g_mx_grouped_glu(h, k3g.mx(dev(ac), dev(asc), fmt), ex.struct, dev(off), perm=dev(perm), top_k=k)
    av = mx_ref.values(ac, asc, fmt)
    hc, hs = host(h.codes), host(h.scales)
    for e in range(E):
        p = np.arange(off[e], off[e + 1])
        if p.size:
            g, ng = mx_ref.product(av[perm[p] // k], ex.w[0][e])
            u, nu = mx_ref.product(av[perm[p] // k], ex.w[1][e])
            mx_ref.check_quantised(hc[p], hs[p], situ64(g, u), situ_tolerance(g, u, ng, nu), hfmt, f"expert {e}")
    left = np.r_[np.arange(off[0]), np.arange(off[-1], P)]
    assert np.all(hc[left] == 77) and np.all(hs[left] == 9), "rows outside the groups were written"


def test_grouped_bad_tables_stay_in_range(k3g):
    # offsets and perm outside their ranges: nothing outside y is written, and rows of a wrong group hold some
    # expert's product or what they held (the preconditions are broken, the memory is not)
    rng = np.random.default_rng(11)
    E, latent, inter, P = 6, 64, 96, 40
    ex = Experts(k3g, rng, E, latent, inter)
    ac, asc = mx_ref.mx_bytes(rng, P, inter, 0)
    buf = torch.full((P + 64, latent), 7.0, device="cuda")
    y = buf[32:32 + P]
    for off in ([-9, 4, 8, 12, 16, 20, 400], [0, 30, 10, 40, 5, 41, 50], [50, 60, 70, 80, 90, 95, 99], [0] * 7,
                [-5, -4, -3, -2, -1, 0, 0], [0, 1 << 30, 1 << 30, 3, -(1 << 30), 2, 1]):
        for perm in (None, rng.integers(-(1 << 30), 1 << 30, P).astype(np.int32)):
            print(f"bad table {off} perm={perm is not None}", flush=True)
            k3g.k3g_mx_grouped_matmul(y, k3g.mx(dev(ac), dev(asc), 0), ex.struct, k3g.W2, dev(np.array(off, np.int32)),
                                      perm=None if perm is None else dev(perm), top_k=2)
    b = host(buf)
    assert (b[:32] == 7.0).all() and (b[32 + P:] == 7.0).all() and np.isfinite(b).all()


MANY = [
    # E, latent, inter, rows a group, rows before, rows behind: more tiles than workgroups that fit the chip, so that
    # each takes several in a row (inputs of whole 512 entries run on from tile to tile, others start anew)
    (300, 512, 512, 40, 0, 0),
    (300, 512, 544, 40, 2, 3),
    (40, 1024, 1536, 150, 0, 1),
    (600, 544, 96, 3, 0, 0),
    (24, 512, 2048, 700, 1, 0),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,latent,inter,per,lead,behind", MANY)
def test_grouped_many_tiles(k3g, E, latent, inter, per, lead, behind, fmt):
    """Every product of a large grouped call on the GPU in float64 (the device's own library) from the tests' values."""
    rng = np.random.default_rng(E + inter)
    P, k = E * per, 2
    ex = Experts(k3g, rng, E, latent, inter, 112, 118)
    off = ragged(rng, E, P, lead, behind, 0.2)
    perm = rng.permutation(P).astype(np.int32)
    ac, asc = mx_ref.mx_bytes(rng, (P + 1) // 2, latent, fmt, 118 if fmt == 0 else 112, 126 if fmt == 0 else 118, p255=0.01)
    hc, hs = mx_ref.mx_bytes(rng, P, inter, fmt, p255=0.01)
    print(f"many tiles E={E} latent={latent} inter={inter} P={P} fmt={fmt}", flush=True)
    y = torch.full((P, latent), 7.0, device="cuda")
    z = torch.full((P, inter), 7.0, device="cuda", dtype=torch.bfloat16)
    h = k3g.mx_empty(P, inter, k3g.MXFP8)
    h.codes.fill_(77), h.scales.fill_(9)
    a = k3g.mx(dev(ac), dev(asc), fmt)
    k3g.k3g_mx_grouped_matmul(y, k3g.mx(dev(hc), dev(hs), fmt), ex.struct, k3g.W2, dev(off))
    k3g.k3g_mx_grouped_matmul(z, a, ex.struct, k3g.W3, dev(off), perm=dev(perm), top_k=k)
    k3g.k3g_mx_grouped_glu(h, a, ex.struct, dev(off), perm=dev(perm), top_k=k)
    torch.cuda.synchronize()
    av, hv = dev(mx_ref.values(ac, asc, fmt)), dev(mx_ref.values(hc, hs, fmt))
    src = dev((perm // k).astype(np.int64))
    yc, zc, gc, gs = host(y).astype(np.float64), host(z).astype(np.float64), host(h.codes), host(h.scales)

    def product(x, w):
        w = dev(w).t().contiguous()
        return (x @ w).cpu().numpy(), (x.abs() @ w.abs()).cpu().numpy()
    for e in range(E):
        p0, p1 = int(off[e]), int(off[e + 1])
        if p1 > p0:
            check_product(yc[p0:p1], *product(hv[p0:p1], ex.w[2][e]), "f32", f"w2 of expert {e}")
            x = av[src[p0:p1]]
            g, ng = product(x, ex.w[0][e])
            u, nu = product(x, ex.w[1][e])
            check_product(zc[p0:p1], u, nu, "bf16", f"w3 of expert {e}")
            if e % 5 == 0:
                mx_ref.check_quantised(gc[p0:p1], gs[p0:p1], situ64(g, u), situ_tolerance(g, u, ng, nu), 1, f"h of expert {e}")
    left = np.r_[np.arange(off[0]), np.arange(off[-1], P)]
    assert np.all(yc[left] == 7.0) and np.all(zc[left] == 7.0) and np.all(gc[left] == 77) and np.all(gs[left] == 9)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,rows,n", [(2100, 4104, 1024), (1025, 8200, 544), (4096, 2304, 512), (700, 12800, 96)])
def test_matmul_many_tiles(k3g, T, rows, n, fmt):
    rng = np.random.default_rng(T)
    ac, asc = mx_ref.mx_bytes(rng, T, n, fmt, p255=0.01)
    wc, wsc = mx_ref.mx_bytes(rng, rows, n, 0, p255=0.01)
    print(f"many tiles T={T} rows={rows} in={n} fmt={fmt}", flush=True)
    y = torch.empty(T, rows, device="cuda")
    k3g.k3g_mx_matmul(y, k3g.mx(dev(ac), dev(asc), fmt), k3g.mxfp4(dev(wc), dev(wsc)))
    av, wv = dev(mx_ref.values(ac, asc, fmt)), dev(mx_ref.values(wc, wsc, 0)).t().contiguous()
    check_product(host(y).astype(np.float64), (av @ wv).cpu().numpy(), (av.abs() @ wv.abs()).cpu().numpy(), "f32", "many tiles")


# ---- together, on a side stream, and captured ----------------------------------------------------

def test_experts_from_route_to_combine(k3g):
    """The microscaled form of a layer as a program runs it: norm and quantised rows, the library's route, bucket and
    combine, the grouped GLU and down product; against the same steps in 64 bits from the kernel's own h."""
    import oracle
    import synth
    E, latent, inter, T, K, fmt = 24, 512, 256, 37, 4, k3g.MXFP8
    rng = np.random.default_rng(21)
    ex = Experts(k3g, rng, E, latent, inter, 112, 118)
    x = rng.standard_normal((T, latent)).astype(np.float32)
    r = rng.standard_normal((T, latent)).astype(np.float32)
    gamma = rng.uniform(0.5, 1.5, latent).astype(np.float32)
    W, b = synth.router(5, E, latent, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xd, rd, gd, Wd, bd = dev(x), dev(r), dev(gamma), dev(W), dev(b)
    mode = k3g.IDOT  # its bucket and combine stages; the products are the microscaled ones
    sh = k3g.shape(n_tokens=T, top_k=K, n_experts=E, latent=latent, inter=inter, mode=mode)
    ws, L = k3g.workspace(k3g.OP_MOE_LAYER, sh), k3g.workspace_layout(k3g.OP_MOE_LAYER, sh)
    ws_r = k3g.workspace(k3g.OP_MOE_ROUTE, k3g.shape(n_tokens=T, n_experts=E))
    region = lambda name, n, ty: ws[L[name]:L[name] + 4 * n].view(ty)  # noqa: E731
    P = T * K
    offsets, perm = region("offsets", E + 1, torch.int32), region("perm", P, torch.int32)
    ypair = region("ypair", P * latent, torch.float32).view(P, latent)
    y, nrm = torch.empty(T, latent, device="cuda"), torch.empty(T, latent, device="cuda")
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, K, device="cuda")
    q, h = k3g.mx_empty(T, latent, fmt), k3g.mx_empty(P, inter, fmt)
    torch.cuda.synchronize()
    print("route to combine", flush=True)
    with torch.cuda.stream(side):
        k3g.k3g_add_rmsnorm(xd, gd, 1e-5, r=rd, sum=xd, y=nrm, q=q)
        k3g.k3g_moe_route(idx, wts, nrm, Wd, bd, K, ws_r)
        k3g.k3g_moe_layer_stage(k3g.STAGE_BUCKET, y, nrm, idx, wts, ex.struct, mode, ws)
        k3g.k3g_mx_grouped_glu(h, q, ex.struct, offsets, perm=perm, top_k=K)
        k3g.k3g_mx_grouped_matmul(ypair, h, ex.struct, k3g.W2, offsets)
        k3g.k3g_moe_layer_stage(k3g.STAGE_COMBINE, y, nrm, idx, wts, ex.struct, mode, ws)
    side.synchronize()
    s = x.astype(np.float64) + r
    ref_n = s / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5) * gamma
    mx_ref.check_quantised(host(q.codes), host(q.scales), ref_n, NORM * np.abs(ref_n), fmt, "norm")
    io, wo, _ = oracle.route(host(nrm), W, b, K)
    assert np.array_equal(host(idx), io)
    qv, hv = mx_ref.values(host(q.codes), host(q.scales), fmt), mx_ref.values(host(h.codes), host(h.scales), fmt)
    order = np.argsort(io.ravel(), kind="stable")
    assert np.array_equal(host(perm), order)
    pos = np.empty(P, np.int64)
    pos[order] = np.arange(P)
    yr, yn = np.zeros((T, latent)), np.zeros((T, latent))
    for t in range(T):
        for k in range(K):
            e = io[t, k]
            g, ng = mx_ref.product(qv[t:t + 1], ex.w[0][e])
            u, nu = mx_ref.product(qv[t:t + 1], ex.w[1][e])
            p = pos[t * K + k]
            mx_ref.check_quantised(host(h.codes)[p:p + 1], host(h.scales)[p:p + 1], situ64(g, u),
                                   situ_tolerance(g, u, ng, nu), fmt, f"h of pair {t},{k}")
            d, dn = mx_ref.product(hv[p:p + 1], ex.w[2][e])
            yr[t] += wo[t, k] * d[0]
            yn[t] += wo[t, k] * dn[0]
    assert np.all(np.abs(host(y) - yr) <= 2 * REL * yn)


def test_capture_and_replay(k3g):
    """Every operator in one captured graph, replayed on new inputs with eager work between, against eager calls."""
    rng = np.random.default_rng(31)
    E, latent, inter, T, K = 6, 256, 128, 70, 2
    ex = Experts(k3g, rng, E, latent, inter, 112, 118)
    w = k3g.mxfp4(*[dev(b) for b in mx_ref.mx_bytes(rng, 300, latent, 0)])
    P = T * K
    gamma = torch.ones(latent, device="cuda")
    x, r = torch.zeros(T, latent, device="cuda", dtype=torch.bfloat16), torch.zeros(T, latent, device="cuda", dtype=torch.bfloat16)
    off, perm = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")

    def outputs():
        return dict(sum=torch.zeros_like(x), q=k3g.mx_empty(T, latent, 0), q8=k3g.mx_empty(T, latent, 1),
                    v=torch.zeros_like(x), y=torch.zeros(T, 300, device="cuda"), h=k3g.mx_empty(P, inter, 1),
                    z=torch.zeros(P, latent, device="cuda", dtype=torch.bfloat16))

    def step(o):
        k3g.k3g_add_rmsnorm(x, gamma, 1e-5, r=r, sum=o["sum"], q=o["q"])
        k3g.k3g_mx_quantize(o["q8"], o["sum"])
        k3g.k3g_mx_dequantize(o["v"], o["q8"])
        k3g.k3g_mx_matmul(o["y"], o["q"], w)
        k3g.k3g_mx_grouped_glu(o["h"], o["q"], ex.struct, off, perm=perm, top_k=K)
        k3g.k3g_mx_grouped_matmul(o["z"], o["h"], ex.struct, k3g.W2, off)

    def feed(seed):
        g = np.random.default_rng(seed)
        x.copy_(torch.from_numpy(g.standard_normal((T, latent)).astype(np.float32)))
        r.copy_(torch.from_numpy(g.standard_normal((T, latent)).astype(np.float32)))
        off.copy_(torch.from_numpy(ragged(g, E, P)))
        perm.copy_(torch.from_numpy(g.permutation(P).astype(np.int32)))

    captured, eager = outputs(), outputs()
    feed(0)
    step(captured)
    torch.cuda.synchronize()
    print("capture", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for seed in range(1, 5):
        feed(seed)
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for name in captured:
            a, b = captured[name], eager[name]
            for u, v in ((a.codes, b.codes), (a.scales, b.scales)) if isinstance(a, k3g.Mx) else ((a, b),):
                assert torch.equal(u, v), f"replay {seed}: {name}"


def test_results_repeat_and_do_not_depend_on_neighbours(k3g):
    """The same call twice gives the same bits, and a token's result does not change with the tokens beside it inside
    one form of the kernels."""
    rng = np.random.default_rng(41)
    n, rows = 1024, 600
    for fmt in FMTS:
        ac, asc = mx_ref.mx_bytes(rng, 700, n, fmt, p255=0.01)
        w = k3g.mxfp4(*[dev(b) for b in mx_ref.mx_bytes(rng, rows, n, 0, p255=0.01)])
        for T in (1, 9, 64, 200, 700):
            a = k3g.mx(dev(ac[:T]), dev(asc[:T]), fmt)
            y = [torch.empty(T, rows, device="cuda") for _ in range(2)]
            for o in y:
                k3g.k3g_mx_matmul(o, a, w)
            assert torch.equal(*y), f"T={T}"


@pytest.mark.parametrize("fmt", [None, 0, 1])
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,n", [(1024, 4096), (1025, 7168), (1031, 16416), (1024, 65536)])
def test_add_rmsnorm_many_rows(k3g, T, n, ty, fmt):
    """With 1024 rows or more a row gets fewer threads; the residual is the output's own place."""
    print(f"norm T={T} n={n} {ty} fmt={fmt}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(T, n, device="cuda", generator=g).to(TYPES[ty])
    r = torch.randn(T, n, device="cuda", generator=g).to(TYPES[ty])
    gamma = torch.rand(n, device="cuda", generator=g) + 0.5
    s = x.double() + r.double()
    ref = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5) * gamma.double()
    sm = torch.empty_like(x)
    q = k3g.mx_empty(T, n, fmt) if fmt is not None else None
    k3g.k3g_add_rmsnorm(x, gamma, 1e-5, r=r, sum=sm, y=r, q=q)
    assert bool(((sm.double() - s).abs() <= (HALF[ty] + 2.0 ** -24) * s.abs() + 1e-7).all())
    assert bool(((r.double() - ref).abs() <= (HALF[ty] + NORM) * ref.abs() + 2.0 ** -25).all())
    if fmt is not None:
        pick = [0, 1, T // 2, T - 1]
        part = host(ref[pick])
        mx_ref.check_quantised(host(q.codes[pick]), host(q.scales[pick]), part, NORM * np.abs(part), fmt, "norm")


def test_add_rmsnorm_more_rows_than_one_launch(k3g):
    """Past 2^25 rows of 64 threads the rows go out in several launches."""
    T, n = (1 << 26) + 5, 32
    print(f"norm T={T} n={n}", flush=True)
    x = torch.empty(T, n, device="cuda", dtype=torch.bfloat16).normal_()
    gamma = torch.ones(n, device="cuda")
    y = torch.full_like(x, 9.0)
    k3g.k3g_add_rmsnorm(x, gamma, 1e-5, y=y)
    for at in (0, (1 << 25) - 8, 1 << 25, T - 16):
        s = x[at:at + 16].double()
        ref = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5)
        assert bool(((y[at:at + 16].double() - ref).abs() <= (HALF["bf16"] + NORM) * ref.abs() + 2.0 ** -25).all()), at


def test_offsets_past_32_bits(k3g):
    """Rows so far apart that their offsets pass 32 bits, in every dense operand, and experts 5 GiB apart."""
    rng = np.random.default_rng(53)
    T, n, rows, ld = 200, 256, 264, 1 << 25  # 200 rows: 6.7e9 entries
    wide = torch.empty(T * ld, device="cuda", dtype=torch.bfloat16)
    far = wide.as_strided((T, n), (ld, 1))
    near = torch.from_numpy(rng.standard_normal((T, n)).astype(np.float32)).to("cuda", torch.bfloat16)
    far.copy_(near)
    gamma = torch.ones(n, device="cuda")
    w = k3g.mxfp4(*[dev(b) for b in mx_ref.mx_bytes(rng, rows, n, 0)])
    for fmt in FMTS:
        print(f"offsets fmt={fmt}", flush=True)
        q = [k3g.mx_empty(T, n, fmt) for _ in range(2)]
        for o, x in zip(q, (near, far)):
            k3g.k3g_mx_quantize(o, x)
        assert torch.equal(q[0].codes, q[1].codes) and torch.equal(q[0].scales, q[1].scales)
        z = [torch.empty_like(near), wide[n:].as_strided((T, n), (ld, 1))]
        for o in z:
            k3g.k3g_mx_dequantize(o, q[0])
        assert torch.equal(*z)
        for o, x in zip(z, (far, near)):  # (the gaps between far rows count as theirs: not both from one buffer)
            k3g.k3g_add_rmsnorm(x, gamma, 1e-5, y=o)
        assert torch.equal(*z)
        for t in (9, 60, T):  # streamed, and with more tokens
            a = k3g.mx(q[0].codes[:t], q[0].scales[:t], fmt)
            y = [torch.empty(t, rows, device="cuda", dtype=torch.bfloat16), wide[2 * n:].as_strided((t, rows), (ld, 1))]
            for o in y:
                k3g.k3g_mx_matmul(o, a, w)
            assert torch.equal(*y), t
    del wide, far, z, y, o, x
    torch.cuda.empty_cache()
    ex = Experts(k3g, rng, 2, 64, 96)
    stride = 5 << 30
    apart = torch.empty(2 * stride, dtype=torch.uint8, device="cuda")
    for e in range(2):
        apart[e * stride:e * stride + ex.struct.stride] = ex.bank[e * ex.struct.stride:(e + 1) * ex.struct.stride]
    b = k3g.bank_struct(apart, 2, 64, 96, list(ex.struct.off), stride)
    P = 40
    a = k3g.mx(*[dev(v) for v in mx_ref.mx_bytes(rng, P, 64, 1)], 1)
    off = dev(np.array([0, 7, P], np.int32))
    out = []
    for s in (ex.struct, b):
        h, y = k3g.mx_empty(P, 96, 1), torch.empty(P, 64, device="cuda")
        k3g.k3g_mx_grouped_glu(h, a, s, off)
        k3g.k3g_mx_grouped_matmul(y, h, s, k3g.W2, off)
        out.append((h, y))
    assert torch.equal(out[0][0].codes, out[1][0].codes) and torch.equal(out[0][0].scales, out[1][0].scales)
    assert torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("fmt", FMTS)
def test_two_streams_and_repeated_sources(k3g, fmt):
    """Calls on two streams at once share nothing; one source row may stand in many places of perm."""
    rng = np.random.default_rng(61)
    E, latent, inter, P = 5, 512, 288, 600
    ex = Experts(k3g, rng, E, latent, inter)
    off = dev(ragged(rng, E, P))
    a = [k3g.mx(*[dev(v) for v in mx_ref.mx_bytes(rng, 9, latent, fmt)], fmt) for _ in range(2)]
    perm = [dev(rng.integers(0, 9 * 2, P).astype(np.int32)) for _ in range(2)]

    def outputs():
        return k3g.mx_empty(P, inter, 1), torch.zeros(P, latent, device="cuda")

    def step(i, o):
        k3g.k3g_mx_grouped_glu(o[0], a[i], ex.struct, off, perm=perm[i], top_k=2)
        k3g.k3g_mx_grouped_matmul(o[1], o[0], ex.struct, k3g.W2, off)

    alone, both = [outputs() for _ in range(2)], [outputs() for _ in range(2)]
    for i in range(2):
        step(i, alone[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                step(i, both[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(alone[i][0].codes, both[i][0].codes) and torch.equal(alone[i][1], both[i][1])
    av = mx_ref.values(host(a[0].codes), host(a[0].scales), fmt)
    y = torch.zeros(P, inter, device="cuda")
    k3g.k3g_mx_grouped_matmul(y, a[0], ex.struct, k3g.W1, off, perm=perm[0], top_k=2)
    o, p = host(off), host(perm[0])
    for e in range(E):
        i = np.arange(o[e], o[e + 1])
        if i.size:
            ref, nrm = mx_ref.product(av[p[i] // 2], ex.w[k3g.W1][e])
            check_product(host(y)[i].astype(np.float64), ref, nrm, "f32", f"expert {e}")
