"""The refusals of the int4 products, before any launch (CPU)."""
import ctypes as C

import pytest

EINVAL, EALIGN, UNSUPPORTED = -1, -2, -5
M = 1 << 20  # made-up addresses a MiB apart: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def weights(k3g, at=M, E=1, rows=8, n=128, group=32, st=0, s=None, z=0):
    return k3g.Int4Struct(at, at + M if s is None else s, (at + 2 * M if z == 0 else z), E, rows, n, group, st)


BAD_WEIGHTS = [({"E": 0}, EINVAL), ({"rows": 0}, EINVAL), ({"n": 0}, EINVAL), ({"n": 112}, EINVAL), ({"group": 16}, EINVAL),
               ({"group": 96}, EINVAL), ({"group": 128, "n": 192}, EINVAL), ({"st": 3}, EINVAL), ({"at": 0, "s": M}, EINVAL),
               ({"s": 0}, EINVAL), ({"n": 65536 + 32}, UNSUPPORTED), ({"E": 2049}, UNSUPPORTED),
               ({"rows": (1 << 30) + 1}, UNSUPPORTED), ({"at": M + 8}, EALIGN), ({"s": 2 * M + 2}, EALIGN),
               ({"s": 2 * M + 1, "st": 1}, EALIGN)]


def test_matmul_refusals(k3g):
    L = k3g.lib()

    def mm(w=None, y=8 * M, yt=0, yl=8, x=9 * M, xt=0, xl=128, T=4, null=False):
        w = weights(k3g) if w is None else w
        return L.k3g_int4_matmul(y, yt, yl, x, xt, xl, T, None if null else C.byref(w), None)
    assert mm(null=True) == EINVAL
    for kw, rc in BAD_WEIGHTS:
        assert mm(weights(k3g, **kw), yl=1 << 31, xl=1 << 20) == rc, kw
    for bad in ({"T": -1}, {"yt": 3}, {"xt": -1}, {"yl": 7}, {"xl": 127}, {"y": None}, {"x": None}, {"y": M}, {"y": 2 * M},
                {"y": 3 * M}, {"y": 9 * M + 512 * 3}, {"y": 2 * M + 124}, {"y": 3 * M + 28}, {"w": weights(k3g, E=2)}):
        assert mm(**bad) == EINVAL, bad
    for bad in ({"y": 8 * M + 2}, {"x": 9 * M + 2}, {"x": 9 * M + 1, "xt": 2}):
        assert mm(**bad) == EALIGN, bad
    assert mm(T=(1 << 30) + 1) == UNSUPPORTED
    assert mm(T=0, x=None, y=None) == 0


@pytest.mark.parametrize("glu", [False, True])
def test_grouped_refusals(k3g, glu):
    L = k3g.lib()

    def call(w=None, y=16 * M, yt=0, yl=8, x=17 * M, xt=0, xl=128, xr=6, off=18 * M, perm=19 * M, k=2, R=6, null=False, w3=None):
        w = weights(k3g, E=3) if w is None else w
        r = None if null else C.byref(w)
        if glu:
            w3 = weights(k3g, at=5 * M, E=w.n_experts, rows=w.rows, n=w.in_, group=w.group, st=w.scale_type) if w3 is None else w3
            return L.k3g_int4_grouped_glu(y, yt, yl, x, xt, xl, xr, r, C.byref(w3), off, perm, k, R, None)
        return L.k3g_int4_grouped_matmul(y, yt, yl, x, xt, xl, xr, r, off, perm, k, R, None)
    assert call(null=True) == EINVAL
    for kw, rc in BAD_WEIGHTS:
        assert call(weights(k3g, **{"E": 3} | kw), yl=1 << 31, xl=1 << 20) == rc, kw
    for bad in ({"R": -1}, {"xr": -1}, {"xr": 0}, {"k": 0}, {"yt": 3}, {"xt": 3}, {"yl": 7}, {"xl": 127}, {"y": None},
                {"x": None}, {"off": None}, {"xr": 5, "perm": None}, {"y": M}, {"y": 2 * M + 4}, {"y": 3 * M},
                {"y": 17 * M}, {"y": 18 * M + 12}, {"y": 19 * M + 20}):
        assert call(**bad) == EINVAL, bad
    for bad in ({"y": 16 * M + 2}, {"x": 17 * M + 2}, {"off": 18 * M + 2}, {"perm": 19 * M + 1}):
        assert call(**bad) == EALIGN, bad
    for bad in ({"R": (1 << 30) + 1}, {"xr": (1 << 30) + 1}):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(R=0, x=None, y=None, off=None, perm=None, xr=0) == 0
    if glu:
        for kw in ({"E": 2}, {"rows": 9}, {"n": 256}, {"group": 64}, {"st": 1}):
            assert call(w3=weights(k3g, **{"at": 5 * M, "E": 3} | kw)) == EINVAL, kw
        assert call(y=5 * M) == EINVAL and call(y=6 * M) == EINVAL and call(y=7 * M) == EINVAL


def test_binding_refuses(k3g):
    import torch
    p, s = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4)
    for f in (lambda: k3g.int4(p, s), lambda: k3g.k3g_int4_matmul(s, s, s), lambda: k3g.k3g_int4_grouped_matmul(s, s, None, s),
              lambda: k3g.int4(p.int(), s), lambda: k3g.int4(p, s.double())):
        with pytest.raises((ValueError, TypeError)):
            f()


def test_form(k3g):
    """Which kernel a product runs on, and the refusals of the question."""
    import torch
    f32, b16, form = torch.float32, torch.bfloat16, k3g.k3g_probe_int4_form
    assert form(b16, 1, 3584, 7168) == (8, 1) and form(b16, 1, 8, 65536) == (16, 16)
    assert form(b16, 16, 3584, 7168) == (16, 16) and form(b16, 16, 7168, 3584) == (32, 16)
    assert form(b16, 64, 3584, 7168) == (32, 16) and form(b16, 65, 3584, 7168) == (64, 32)
    assert form(f32, 32, 8192, 64) == (32, 16) and form(f32, 32, 8193, 64) == (64, 32) == form(f32, 17, 16384, 64)
    assert form(b16, 1536, 3584, 7168) == (256, 128)
    assert form(b16, 1024, 3584, 7168, aligned=False) == (256, 64) and form(f32, 1024, 3584, 7168) == (256, 64)
    assert form(f32, 512, 3584, 7168) == (64, 32) and form(b16, 512, 3584, 7168) == (64, 64)
    assert form(b16, 128, 3584, 7168) == (64, 32) and form(b16, 129, 3584, 7168) == (64, 64)
    assert form(f32, 16, 3072, 3584, 896, glu=True) == (8, 1) and form(b16, 1024, 3072, 3584, 896, glu=True) == (32, 16)
    assert form(f32, 2, 3584, 7168) == (8, 1) and form(f32, 3, 3584, 7168) == (16, 16) == form(b16, 2, 3584, 7168)
    assert form(f32, 256, 3584, 512, 256) == (8, 1) and form(f32, 256, 3584, 512, 255) == (32, 16) == form(f32, 257, 64, 64, 896)
    assert form(f32, 4, 2**28, 32, 4, glu=True) == (8, 1) and form(f32, 4, 2**28 + 1, 32, 4, glu=True) == (32, 16)
    assert form(b16, 128, 3584, 512, 256) == (8, 1) and form(b16, 128, 3584, 512, 255) == (32, 16)
    assert form(b16, 12 * 896, 3584, 3072, 896) == (32, 16) and form(b16, 12 * 896 + 1, 3584, 3072, 896) == (64, 32)
    assert form(f32, 8 * 896, 3584, 3072, 896) == (32, 16) and form(f32, 8 * 896 + 1, 3584, 3072, 896) == (64, 32)
    assert form(b16, 16 * 896, 3584, 3072, 896) == (64, 32) and form(b16, 65536, 3584, 3072, 896) == (256, 128)
    L = k3g.lib()
    ok = [1, 1, 1, 64, 64, 64, 8]
    assert L.k3g_probe_int4_form(*ok) > 0
    for i, bad in ((0, 3), (2, 3), (2, -1), (3, 0), (4, 0), (5, 0), (5, 48), (5, 1 << 17), (6, 0), (6, 2049)):
        assert L.k3g_probe_int4_form(*[bad if j == i else v for j, v in enumerate(ok)]) == EINVAL, (i, bad)
