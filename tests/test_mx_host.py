"""The microscaled calls' refusals, before any launch (CPU), and the tests' own
64-bit reference against the formats' tables."""
import ctypes as C

import numpy as np
import pytest

from tests import mx_ref

EINVAL, EALIGN, UNSUPPORTED = -1, -2, -5


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


M = 1 << 20  # made-up addresses a MiB apart: never dereferenced, validation fails first


def mx(k3g, at, rows=4, n=64, fmt=0, scales=None):
    return k3g.MxStruct(at, at + M // 2 if scales is None else scales, rows, n, fmt)


def quantize(k3g, q, x=100 * M, t=0, ld=64):
    return k3g.lib().k3g_mx_quantize(C.byref(q) if q is not None else None, x, t, ld, None)


def test_quantize_refusals(k3g):
    ok = mx(k3g, M)
    assert quantize(k3g, None) == EINVAL
    assert quantize(k3g, mx(k3g, M, n=48)) == EINVAL
    assert quantize(k3g, mx(k3g, M, n=0)) == EINVAL
    assert quantize(k3g, mx(k3g, M, rows=-1)) == EINVAL
    assert quantize(k3g, mx(k3g, M, fmt=2)) == EINVAL
    assert quantize(k3g, mx(k3g, M, n=65536 + 32), ld=1 << 20) == UNSUPPORTED
    assert quantize(k3g, mx(k3g, M + 8)) == EALIGN
    assert quantize(k3g, ok, x=None) == EINVAL
    assert quantize(k3g, ok, x=100 * M + 2) == EALIGN  # fp32 off its four bytes
    assert quantize(k3g, ok, t=3) == EINVAL
    assert quantize(k3g, ok, ld=63) == EINVAL
    assert quantize(k3g, ok, x=M + 64) == EINVAL  # x over the codes
    assert quantize(k3g, ok, x=M // 2 + M - 1020) == EINVAL  # x's last row over the scales
    assert quantize(k3g, mx(k3g, M, scales=M + 16)) == EINVAL  # codes over scales
    assert quantize(k3g, mx(k3g, 0, rows=0, scales=0), x=None) == 0  # nothing to do, null pointers allowed
    assert quantize(k3g, mx(k3g, 0, rows=0, n=33, scales=0), x=None) == EINVAL
    L = k3g.lib()
    assert L.k3g_mx_dequantize(100 * M, 0, 63, C.byref(ok), None) == EINVAL
    assert L.k3g_mx_dequantize(100 * M, 4, 64, C.byref(ok), None) == EINVAL
    assert L.k3g_mx_dequantize(100 * M + 1, 1, 64, C.byref(ok), None) == EALIGN
    assert L.k3g_mx_dequantize(M + 16, 0, 64, C.byref(ok), None) == EINVAL
    assert L.k3g_mx_dequantize(None, 0, 64, C.byref(mx(k3g, 0, rows=0, scales=0)), None) == 0


def test_quantize_refuses_more_groups_than_a_launch_counts(k3g):
    for fn in (lambda q: quantize(k3g, q, x=1 << 46, t=1, ld=65536),
               lambda q: k3g.lib().k3g_mx_dequantize(1 << 46, 1, 65536, C.byref(q), None)):
        assert fn(mx(k3g, 1 << 40, rows=1 << 19, n=65536, scales=1 << 45)) == UNSUPPORTED


def test_norm_refusals(k3g):
    L = k3g.lib()

    def norm(y=M, ys=64, s=2 * M, ss=64, q=None, x=3 * M, xs=64, r=4 * M, rs=64, t=0, gamma=5 * M, eps=1e-5, n=4, w=64):
        return L.k3g_add_rmsnorm(y, ys, s, ss, C.byref(q) if q is not None else None, x, xs, r, rs, t, gamma, eps, n, w,
                                 None)
    for bad in ({"n": -1}, {"w": 33}, {"w": 0}, {"t": 3}, {"eps": -1e-5}, {"eps": float("nan")}, {"eps": float("inf")},
                {"x": None}, {"gamma": None}, {"y": None}, {"ys": 63}, {"ss": 63}, {"xs": 63}, {"rs": 63},
                {"q": mx(k3g, 6 * M, rows=3)}, {"q": mx(k3g, 6 * M, n=96)}, {"q": mx(k3g, M)},
                {"q": mx(k3g, 3 * M + 512)}, {"q": mx(k3g, 6 * M, scales=5 * M)},
                {"y": 3 * M, "ys": 65}, {"y": 3 * M + 256}, {"s": 4 * M + 256}, {"s": M}, {"y": 5 * M}, {"s": 5 * M}):
        assert norm(**bad) == EINVAL, bad
    assert norm(w=65536 + 32, xs=M, ys=M, ss=M, rs=M) == UNSUPPORTED
    assert norm(gamma=5 * M + 2) == EALIGN
    assert norm(x=3 * M + 2) == EALIGN
    assert norm(n=0, y=None, s=None, x=None, r=None, gamma=None) == 0


def test_product_refusals(k3g):
    L = k3g.lib()

    def mm(y=M, t=0, ld=8, a=None, w=None):
        a = mx(k3g, 2 * M) if a is None else a
        w = k3g.Mxfp4(3 * M, 4 * M, 8, 64) if w is None else w
        return L.k3g_mx_matmul(y, t, ld, C.byref(a), C.byref(w) if w != 0 else None, None)
    for bad in ({"y": None}, {"t": 3}, {"ld": 7}, {"w": 0}, {"w": k3g.Mxfp4(3 * M, 4 * M, 0, 64)},
                {"w": k3g.Mxfp4(3 * M, 4 * M, 8, 96)}, {"w": k3g.Mxfp4(None, 4 * M, 8, 64)},
                {"w": k3g.Mxfp4(3 * M, None, 8, 64)}, {"a": mx(k3g, 2 * M, fmt=5)}, {"y": 2 * M}, {"y": 3 * M},
                {"y": 4 * M - 64}, {"y": 2 * M + M // 2}):
        assert mm(**bad) == EINVAL, bad
    assert mm(a=mx(k3g, 1 << 40, rows=(1 << 30) + 1, scales=1 << 45)) == UNSUPPORTED
    assert mm(w=k3g.Mxfp4(1 << 40, 1 << 45, (1 << 30) + 1, 64), ld=1 << 31) == UNSUPPORTED
    assert mm(w=k3g.Mxfp4(3 * M + 4, 4 * M, 8, 64)) == EALIGN
    assert mm(y=M + 2) == EALIGN
    assert mm(a=mx(k3g, 0, rows=0, scales=0), y=None) == 0


def bank(k3g, E=8, latent=64, inter=96, base=16 * M, stride=None, off=None):
    o, st = k3g.bank_layout(64, 96)
    return k3g.ExpertBank(base, st if stride is None else stride, E, latent, inter, (C.c_int64 * 6)(*(off or o)))


def test_grouped_refusals(k3g):
    L = k3g.lib()

    def gm(y=M, t=0, ld=64, a=None, b=None, tensor=2, off=4 * M, perm=5 * M, k=2, n=8):
        a = mx(k3g, 2 * M, rows=4, n=96) if a is None else a
        b = bank(k3g) if b is None else b
        return L.k3g_mx_grouped_matmul(y, t, ld, C.byref(a), C.byref(b), tensor, off, perm, k, n, None)

    def glu(h=None, a=None, b=None, off=4 * M, perm=5 * M, k=2, n=8):
        h = mx(k3g, M, rows=8, n=96) if h is None else h
        a = mx(k3g, 2 * M, rows=4, n=64) if a is None else a
        b = bank(k3g) if b is None else b
        return L.k3g_mx_grouped_glu(C.byref(h), C.byref(a), C.byref(b), off, perm, k, n, None)
    for call in (gm, glu):
        for bad in ({"b": bank(k3g, E=0)}, {"b": bank(k3g, latent=33)}, {"b": bank(k3g, base=None)}, {"off": None},
                    {"k": 0}, {"n": -1}, {"perm": None}):  # no perm: a has fewer rows than the output
            assert call(**bad) == EINVAL, (call.__name__, bad)
        assert call(b=bank(k3g, E=2049)) == UNSUPPORTED
        assert call(b=bank(k3g, stride=-16384)) == EINVAL
        assert call(b=bank(k3g, stride=bank(k3g).stride + 8)) == EALIGN
        assert call(b=bank(k3g, base=16 * M + 8)) == EALIGN
        assert call(off=4 * M + 2) == EALIGN
        assert call(perm=5 * M + 2) == EALIGN
    assert gm(tensor=3) == EINVAL and gm(tensor=0) == EINVAL  # w1 takes rows of the latent width
    assert gm(ld=63) == EINVAL and gm(y=None) == EINVAL and gm(t=7) == EINVAL
    assert gm(y=2 * M) == EINVAL and gm(y=4 * M) == EINVAL and gm(y=5 * M) == EINVAL
    assert gm(y=16 * M + bank(k3g).off[4]) == EINVAL  # over the bank's w2
    assert gm(a=mx(k3g, 2 * M, rows=1 << 26, n=96, scales=1 << 50)) == UNSUPPORTED  # source offsets pass 32 bits
    assert gm(n=0, y=None, off=None, perm=None) == 0
    assert glu(h=mx(k3g, M, rows=7, n=96)) == EINVAL and glu(h=mx(k3g, M, rows=8, n=64)) == EINVAL
    assert glu(a=mx(k3g, 2 * M, rows=4, n=96)) == EINVAL
    assert glu(h=mx(k3g, 4 * M, rows=8, n=96)) == EINVAL and glu(h=mx(k3g, 16 * M, rows=8, n=96)) == EINVAL
    assert glu(h=mx(k3g, 2 * M, rows=8, n=96)) == EINVAL
    assert glu(n=0, off=None, perm=None, h=mx(k3g, 0, rows=0, n=96, scales=0)) == 0


def test_python_refusals_need_no_gpu(k3g):
    import torch
    cpu = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        k3g.mx_empty(4, 48, k3g.MXFP4, device="cpu")
    with pytest.raises(ValueError):
        k3g.mx_empty(4, 64, 2, device="cpu")
    with pytest.raises(ValueError):
        k3g.mx(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), k3g.MXFP4)  # on the host
    with pytest.raises(TypeError):
        k3g.k3g_mx_quantize(None, cpu)
    with pytest.raises(ValueError):
        k3g.k3g_add_rmsnorm(cpu, cpu[0], 1e-5)


def test_reference_formats():
    # every code is its own nearest, ties go to the even code, and the exponents fit
    for fmt in (0, 1):
        t = mx_ref.MAGS[fmt][: 8 if fmt == 0 else 127]
        assert np.array_equal(mx_ref.nearest_code(t, fmt), np.arange(len(t)))
        mid = (t[1:] + t[:-1]) / 2
        c = mx_ref.nearest_code(mid, fmt)
        assert np.all(c % 2 == 0) and np.all(np.abs(c - np.arange(len(mid)) - 0.5) == 0.5)
        m = np.array([mx_ref.MAX[fmt], np.nextafter(mx_ref.MAX[fmt], 1e9), 1.0, 1e-40, 0.0])
        assert mx_ref.exponent(m, fmt).tolist() == [0, 1, -2 if fmt == 0 else -8, -126, -126]
    assert mx_ref.MAGS[1][126] == 448 and mx_ref.MAGS[1][1] == 2.0 ** -9
