"""Products with int4 weights on the GPU: whole numbers to the bit, values against
64 bits, ragged groups, the gated up-product, and a layer's run of them."""
import numpy as np
import pytest
import torch

from tests import int4_ref as ref

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
name = lambda t: str(t)[6:] if isinstance(t, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def output(T, rows, t, pad=0):
    """A marked buffer of T rows and the view of its first `rows` columns."""
    b = torch.full((T + 2, rows + pad + 1), 7.0, device="cuda").to(t)
    return b, b[1:T + 1, :rows]


def untouched(b, T, rows):
    return bool((b[0] == 7).all() and (b[T + 1:] == 7).all() and (b[:, rows:] == 7).all())


# (tokens, columns, outputs, group): one token and one output, one group, ends inside a step of 128 columns and inside
# the 512 that a wavefront takes, more turns than wavefronts, ragged outputs and tokens, the largest row
DENSE = [(1, 32, 1, 32), (1, 64, 17, 64), (1, 128, 16, 128), (2, 96, 33, 32), (1, 7168, 3584, 64), (3, 320, 100, 64),
         (15, 544, 31, 32), (16, 640, 64, 128), (17, 1056, 48, 32), (31, 4224, 40, 128), (33, 3584, 129, 64),
         (61, 3584, 7168, 32), (64, 4160, 257, 32), (65, 512, 130, 128), (127, 1120, 77, 32), (200, 2048, 300, 64),
         (129, 352, 4200, 32), (141, 704, 4500, 64),
         (33, 704, 8300, 64), (2, 4224, 1030, 64), (24, 640, 8300, 128), (250, 1056, 500, 32), (70, 1088, 777, 64), (257, 2176, 70, 128),
         (4, 65536, 5, 32), (1000, 256, 512, 64), (300, 768, 4097, 128), (1, 34816, 40, 64),
         # tiles: ragged outputs and tokens, an odd number of 32-column blocks, ends inside a turn of 256 columns
         (300, 352, 11001, 32), (515, 704, 6700, 64), (500, 640, 11000, 128), (385, 32, 9700, 32)]


@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("T,n,rows,group", DENSE)
def test_whole_numbers_are_exact(k3g, T, n, rows, group, xt):
    """Small whole numbers and scales that are powers of two: sums of so few random terms stay far below 2^24 of their
    unit (65536 terms of at most 60 and scales of 1/8 to 2: about 2^15 of 1/8), so none is rounded."""
    g = gen(T + n + rows)
    for zeros in (False, True):
        for st in TYPES:
            w = ref.random_weights(g, (rows,), n, group, st, zeros, exact=True)
            x = ref.rows_of(g, T, n, xt, exact=True)
            want = x.double() @ ref.values(*w)[0].t().contiguous()
            for a in (x, x.clone()):  # rows off 16-byte addresses, and on them
                b, y = output(T, rows, torch.float32)
                k3g.k3g_int4_matmul(y, a, k3g.int4(*w))
                assert torch.equal(y.double(), want), (zeros, st)
                assert untouched(b, T, rows)


@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("yt", TYPES, ids=name)
@pytest.mark.parametrize("T,n,rows,group", DENSE)
def test_values(k3g, T, n, rows, group, xt, yt):
    g = gen(T * 3 + n + rows)
    for st, zeros in ((torch.bfloat16, False), (torch.float16, True), (torch.float32, True)):
        w = ref.random_weights(g, (rows,), n, group, st, zeros)
        x = ref.rows_of(g, T, n, xt, pad=5)
        if zeros:
            x = x.contiguous()
        b, y = output(T, rows, yt, pad=3)
        k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
        m, mag = ref.values(*w)
        ref.check(y, x.double() @ m.t().contiguous(), x.double().abs() @ mag.t().contiguous(), ref.roundings(n, group))
        assert untouched(b, T, rows)


def test_fp32_rows_go_in_whole(k3g):
    """A matrix of ones on the diagonal (code 1, zero 0, scale 1) gives x back bit for bit, all 24 bits of it, from
    2^-100 to 2^100; and of code 15 the rounding of 15 x (three parts, products exact, at most two sums)."""
    n = 256
    packed = torch.zeros(n, n // 2, dtype=torch.uint8, device="cuda")
    i = torch.arange(n, device="cuda")
    packed[i, i // 2] = torch.where(i % 2 == 0, 1, 16).to(torch.uint8)
    one, zero = torch.ones(n, n // 32, device="cuda"), torch.zeros(n, n // 32, dtype=torch.uint8, device="cuda")
    for T in (1, 3, 40, 300):
        g = gen(T)
        x = torch.randn(T, n, device="cuda", generator=g) * torch.exp2(torch.randint(-100, 100, (T, n), device="cuda", generator=g).float())
        # one entry a group keeps what it is: the others of its row are 0
        x = torch.where(i % 32 == 7 + T % 8, x, 0.0)
        y = torch.empty(T, n, device="cuda")
        k3g.k3g_int4_matmul(y, x, k3g.int4(packed, one, zero))
        assert torch.equal(y, x)
        k3g.k3g_int4_matmul(y, x, k3g.int4((packed * 15).to(torch.uint8), one, zero))
        assert bool(((y.double() - 15 * x.double()).abs() <= 2 * 2.0 ** -23 * 15 * x.double().abs()).all())


def test_weights_of_value_zero_next_to_large_entries(k3g):
    """Codes that equal their zero: the columns' sum and the codes' products cancel to nothing where x is whole numbers."""
    n, rows = 512, 64
    packed = torch.full((rows, n // 2), 0x88, dtype=torch.uint8, device="cuda")
    s = torch.ones(rows, n // 64, device="cuda", dtype=torch.bfloat16)
    for T in (1, 20, 100):
        x = torch.randint(-1000, 1000, (T, n), device="cuda").float()
        y = torch.empty(T, rows, device="cuda")
        k3g.k3g_int4_matmul(y, x, k3g.int4(packed, s))
        assert bool((y == 0).all())


def test_not_finite(k3g):
    """A token with an infinity or a NaN has no finite output; the tokens beside it keep theirs. So do rows with such
    a scale, and the rows beside them."""
    for T, n_out in ((1, 70), (5, 70), (40, 70), (300, 70), (300, 11000)):
        for xt in TYPES:
            g = gen(T)
            w = ref.random_weights(g, (n_out,), 384, 32, torch.float32, True)
            x = torch.randn(T, 384, device="cuda", generator=g).to(xt)
            good = torch.empty(T, n_out, device="cuda")
            k3g.k3g_int4_matmul(good, x, k3g.int4(*w))
            bad = sorted({T // 4, T // 2, T - 1})
            for t, c, v in zip(bad, (7, 380, 100), (float("inf"), float("nan"), -float("inf"))):
                x[t, c] = v
            y = torch.empty(T, n_out, device="cuda")
            k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
            hit = torch.zeros(T, dtype=torch.bool, device="cuda")
            hit[bad] = True
            assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], good[~hit])
            w[1][11, 4], w[1][n_out - 1, 0] = float("nan"), float("inf")
            k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
            rows = torch.ones(n_out, dtype=torch.bool, device="cuda")
            rows[[11, n_out - 1]] = False
            assert torch.equal(y[~hit][:, rows], good[~hit][:, rows]) and not torch.isfinite(y[:, ~rows]).any()


@pytest.mark.parametrize("xt,least", [(torch.float32, 2.0 ** -126), (torch.bfloat16, 2.0 ** -133), (torch.float16, 2.0 ** -24)], ids=name)
def test_the_smallest_entries(k3g, xt, least):
    """Whole multiples of the type's smallest step (of fp32's smallest normal number), subnormal numbers for the most
    part: products and sums are multiples of the same step below 2^24 of it, so nothing is rounded or lost."""
    for T, n_out in ((1, 40), (3, 40), (50, 40), (300, 11000)):
        g = gen(T)
        w = ref.random_weights(g, (n_out,), 96, 32, torch.float32, True)
        w[1].fill_(1.0)
        x = (torch.randint(-9, 10, (T, 96), device="cuda", generator=g).double() * least).to(xt)
        y = torch.empty(T, n_out, device="cuda")
        k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
        assert torch.equal(y.double(), x.double() @ ref.values(*w)[0].t().contiguous()), T


def test_rows_in_slices_of_one_buffer(k3g):
    """x and y beside each other in the rows of one buffer."""
    n, rows = 256, 72
    for T in (1, 9, 70):
        g = gen(T)
        w = ref.random_weights(g, (rows,), n, 64, torch.bfloat16, True, exact=True)
        b = torch.full((T, n + rows + 5), 7.0, device="cuda")
        b[:, :n] = torch.randint(-4, 5, (T, n), device="cuda", generator=g).float()
        x, y = b[:, :n], b[:, n + 2:n + 2 + rows]
        want = x.double() @ ref.values(*w)[0].t().contiguous()
        k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
        assert torch.equal(y.double(), want) and bool((b[:, n:n + 2] == 7).all() and (b[:, n + 2 + rows:] == 7).all())


def test_zeros_at_both_ends_and_tensors_off_their_alignment(k3g):
    """Zeros of 0, 15 and 128; scales and zeros that begin at any entry, next to marked ones."""
    for T, n, rows in ((1, 320, 50), (7, 320, 50), (40, 320, 50), (515, 320, 6700)):
        for xt in TYPES:
            g = gen(T)
            packed, s, _ = ref.random_weights(g, (rows,), n, 32, torch.bfloat16, False, exact=True)
            z = torch.tensor([0, 15, 128], dtype=torch.uint8, device="cuda")[torch.randint(0, 3, s.shape, device="cuda", generator=g)]
            sb = torch.full((s.numel() + 9,), float("nan"), dtype=s.dtype, device="cuda")
            zb = torch.full((z.numel() + 9,), 77, dtype=torch.uint8, device="cuda")
            s1, z1 = sb[3:3 + s.numel()].view(s.shape), zb[5:5 + z.numel()].view(z.shape)
            s1.copy_(s), z1.copy_(z)
            x = ref.rows_of(g, T, n, xt, exact=True).contiguous()
            y = torch.empty(T, rows, device="cuda")
            k3g.k3g_int4_matmul(y, x, k3g.int4(packed, s1, z1))
            assert torch.equal(y.double(), x.double() @ ref.values(packed, s, z)[0].t().contiguous()), (T, xt)


def test_the_sizes_above_reach_every_kernel(k3g):
    """The tiles (weight rows, tokens) that the tests' sizes run on, by kind and type of x."""
    form = k3g.k3g_probe_int4_form
    for xt in TYPES:
        wide = (256, 64) if xt == torch.float32 else (256, 128)
        dense = {form(xt, T, rows, n) for T, n, rows, _ in DENSE}
        assert dense == {(8, 1), (16, 16), (32, 16), (64, 32), wide} | ({(64, 64)} if xt != torch.float32 else set())
        if xt != torch.float32:
            assert (256, 64) in {form(xt, T, rows, n, aligned=False) for T, n, rows, _ in DENSE}
        for glu in (False, True):
            assert {form(xt, R, rows, n, E, glu) for E, R, n, rows, _, _ in GROUPED} == {(8, 1), (32, 16), (64, 32), wide}
            assert (256, 64) in {form(xt, R, rows, n, E, glu, aligned=False) for E, R, n, rows, _, _ in GROUPED}
        for group in (32, 64, 128):  # every group on tiles, dense and grouped
            assert any(form(xt, T, rows, n) == wide for T, n, rows, g in DENSE if g == group)
            assert xt == torch.float32 or any(form(xt, T, rows, n) == (64, 64) for T, n, rows, g in DENSE if g == group)
            for glu in (False, True):
                assert any(form(xt, R, rows, n, E, glu) == wide for E, R, n, rows, g, _ in GROUPED if g == group)


def test_no_tokens(k3g):
    w = ref.random_weights(gen(0), (8,), 64, 32, torch.float32, False)
    k3g.k3g_int4_matmul(torch.empty(0, 8, device="cuda"), torch.empty(0, 64, device="cuda"), k3g.int4(*w))


# ---- grouped -----------------------------------------------------------------------------

def ragged(g, E, n_rows, before=0, behind=0):
    """Offsets of E groups over rows before .. n_rows - behind, some of them empty."""
    cut = torch.sort(torch.randint(before, n_rows - behind + 1, (E - 1,), generator=g, device="cuda")).values
    if E > 4:
        cut[1] = cut[2]
    ends = torch.tensor([before], device="cuda"), torch.tensor([n_rows - behind], device="cuda")
    return torch.cat([ends[0], cut, ends[1]]).int()


# (experts, rows, columns, outputs, group, top_k): few and many rows an expert, one expert, more experts than rows
GROUPED = [(1, 5, 64, 16, 32, 1), (7, 40, 128, 48, 64, 2), (896, 64, 96, 33, 32, 16), (30, 700, 640, 100, 128, 4),
           (5, 400, 544, 257, 32, 3), (64, 1000, 1536, 128, 64, 8), (3, 1500, 256, 384, 128, 1), (2048, 300, 64, 8, 32, 6),
           # tiles
           (16, 1500, 352, 2000, 32, 1), (12, 1400, 448, 2600, 64, 4), (13, 1300, 640, 2401, 128, 2),
           # the vector kernel: rows of experts, more rows than an expert's share
           (896, 16, 3584, 100, 32, 16), (200, 64, 2112, 33, 64, 1), (130, 60, 6272, 70, 128, 7),
           (256, 250, 2080, 50, 32, 3), (600, 256, 1088, 33, 64, 4)]


@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("E,R,n,rows,group,k", GROUPED)
def test_grouped(k3g, E, R, n, rows, group, k, xt):
    g = gen(E + R)
    for zeros, st, yt in ((False, torch.bfloat16, torch.float32), (True, torch.float16, torch.bfloat16)):
        w = ref.random_weights(g, (E, rows), n, group, st, zeros)
        before, behind = (0, 0) if R < 10 else (3, 4)
        off = ragged(g, E, R, before, behind)
        perm = torch.randperm(R, generator=g, device="cuda").int()
        x = ref.rows_of(g, (R + k - 1) // k, n, xt, pad=1)
        straight = ref.rows_of(g, R, n, xt)
        if zeros:  # on 16-byte addresses, the other time off them
            x, straight = x.contiguous(), straight.clone()
        for source, p in ((x, perm), (straight, None)):
            b, y = output(R, rows, yt, pad=2)
            k3g.k3g_int4_grouped_matmul(y, source, k3g.int4(*w), off, perm=p, top_k=k)
            a = source.double() if p is None else source.double()[p.long() // k]
            want, mag = torch.full((R, rows), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(R, rows, dtype=torch.float64, device="cuda")
            o = off.tolist()
            for e in range(E):
                if o[e + 1] > o[e]:
                    v, m = ref.values(*[None if t is None else t[e] for t in w])
                    s = slice(o[e], o[e + 1])
                    want[s], mag[s] = a[s] @ v.t().contiguous(), a[s].abs() @ m.t().contiguous()
            ref.check(y, want, mag, ref.roundings(n, group))
            assert untouched(b, R, rows) and bool((y[:before] == 7).all() and (y[R - behind:] == 7).all())


@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("E,R,n,rows,group,k", GROUPED)
def test_glu(k3g, E, R, n, rows, group, k, xt):
    """h = f(g) U(u), f(g) = 4 tanh(g/4) sigmoid(g), U = 25 tanh(u/25): |f'| <= 1.1 and |U'| <= 1, and both in fp32 to
    a few steps (16 taken)."""
    g = gen(E + R + 1)
    steps = ref.roundings(n, group) * 2.0 ** -24
    for zeros, st, ht in ((False, torch.float32, torch.float32), (True, torch.bfloat16, torch.float16)):
        w1 = ref.random_weights(g, (E, rows), n, group, st, zeros)
        w3 = ref.random_weights(g, (E, rows), n, group, st, not zeros)
        off = ragged(g, E, R)
        perm = torch.randperm(R, generator=g, device="cuda").int()
        x = ref.rows_of(g, (R + k - 1) // k, n, xt)
        x = x.clone() if zeros else x
        b, h = output(R, rows, ht)
        k3g.k3g_int4_grouped_glu(h, x, k3g.int4(*w1), k3g.int4(*w3), off, perm=perm, top_k=k)
        a = x.double()[perm.long() // k]
        o = off.tolist()
        for e in range(E):
            if o[e + 1] == o[e]:
                continue
            s = slice(o[e], o[e + 1])
            (gate, eg), (up, eu) = [(a[s] @ v.t().contiguous(), steps * (a[s].abs() @ m.t().contiguous()))
                                    for v, m in (ref.values(*[None if t is None else t[e] for t in w]) for w in (w1, w3))]
            f, u = 4 * torch.tanh(gate / 4) / (1 + torch.exp(-gate)), 25 * torch.tanh(up / 25)
            fi = torch.finfo(ht)
            tol = (fi.eps / 2 + 16 * 2.0 ** -24) * (f * u).abs() + 1.01 * (1.1 * eg * (u.abs() + eu) + f.abs() * eu) + fi.smallest_normal * fi.eps / 2
            err = (h[s].double() - f * u).abs()
            assert bool((err <= tol).all()), (e, float((err / tol).max()))
        assert untouched(b, R, rows)


def test_groups_out_of_range_touch_nothing_outside(k3g):
    """Offsets beyond the rows and a perm beyond x: clipped, nothing outside is written (what is read is some row)."""
    E, R, n, rows = 4, 50, 128, 40
    w = ref.random_weights(gen(1), (E, rows), n, 32, torch.bfloat16, True)
    x = torch.randn(R, n, device="cuda")
    perm = torch.full((R,), 2**31 - 1, dtype=torch.int32, device="cuda")
    perm[::2] = -5
    for off in ([-7, 10, 20, 70, 90], [0, 0, 200, 300, 400], [50, 50, 50, 50, 50]):
        b, y = output(R, rows, torch.float32)
        k3g.k3g_int4_grouped_matmul(y, x, k3g.int4(*w), torch.tensor(off, dtype=torch.int32, device="cuda"), perm=perm, top_k=1)
        torch.cuda.synchronize()
        assert untouched(b, R, rows)


def test_far_experts_and_rows(k3g):
    """Codes past 2^32 bytes, rows of x and y past 2^31 entries."""
    E, rows, n = 520, 4096, 4096
    packed = torch.zeros(E, rows, n // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(E, rows, n // 128, dtype=torch.bfloat16, device="cuda")
    far = [0, 511, 512, 519]
    g = gen(5)
    for e in far:
        packed[e] = torch.randint(0, 256, (rows, n // 2), dtype=torch.uint8, device="cuda", generator=g)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for i, e in enumerate(far):
        off[e + 1:] = 2 * (i + 1)
    ld = (1 << 30) + 64
    xb = torch.zeros(7 * ld + n, dtype=torch.bfloat16, device="cuda")
    x = xb.as_strided((8, n), (ld, 1))
    x.copy_(torch.randint(-4, 5, (8, n), device="cuda", generator=g))
    yb = torch.zeros(7 * ld + rows, dtype=torch.bfloat16, device="cuda")
    y = yb.as_strided((8, rows), (ld, 1))
    k3g.k3g_int4_grouped_matmul(y, x, k3g.int4(packed, scales), off)
    for i, e in enumerate(far):
        v = ref.values(packed[e], scales[e], None)[0]
        assert torch.equal(y[2 * i:2 * i + 2], (x[2 * i:2 * i + 2].double() @ v.t().contiguous()).bfloat16())


# ---- together ----------------------------------------------------------------------------

def layer(k3g, b, x, idx, wts, w1, w3, w2, K):
    k3g.k3g_moe_sort(b["off"], b["perm"], b["inv"], idx, b["ws"])
    k3g.k3g_int4_grouped_glu(b["h"], x, w1, w3, b["off"], perm=b["perm"], top_k=K)
    k3g.k3g_int4_grouped_matmul(b["ys"], b["h"], w2, b["off"])
    return k3g.k3g_moe_combine(b["y"], b["ys"], b["inv"], wts=wts)


def layer_buffers(k3g, T, K, E, n, inter):
    ids = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(off=ids(E + 1), perm=ids(T * K), inv=ids(T, K), h=torch.empty(T * K, inter, device="cuda"),
                ys=torch.empty(T * K, n, device="cuda"), y=torch.empty(T, n, device="cuda"),
                ws=k3g.workspace(k3g.OP_MOE_SORT, k3g.shape(n_tokens=T, top_k=K, n_experts=E)))


@pytest.mark.parametrize("T", [1, 37, 600])
def test_a_layer_from_route_to_combine(k3g, T):
    """k3g_moe_route_topp, the sort, the experts' products and the combine, against 64 bits. The tolerance carries the
    up-products' errors through w2 and adds w2's own and the combine's."""
    E, K, n, inter, group = 48, 8, 512, 320, 64
    g = gen(T)
    ws = [ref.random_weights(g, (E, r), c, group, torch.bfloat16, z) for r, c, z in ((inter, n, True), (inter, n, False), (n, inter, True))]
    x = torch.randn(T, n, device="cuda", generator=g)
    router, bias = torch.randn(E, n, device="cuda", generator=g) * 0.05, torch.zeros(E, device="cuda")
    idx, wts = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    k3g.k3g_moe_route_topp(idx, wts, x, router, bias, K, 0.8, k3g.workspace(k3g.OP_MOE_ROUTE, k3g.shape(n_tokens=T, n_experts=E)))
    assert bool((idx == -1).any())
    y = layer(k3g, layer_buffers(k3g, T, K, E, n, inter), x, idx, wts, *[k3g.int4(*w) for w in ws], K)
    want, tol = torch.zeros(T, n, dtype=torch.float64, device="cuda"), torch.zeros(T, n, dtype=torch.float64, device="cuda")
    up, down = ref.roundings(n, group) * 2.0 ** -24, ref.roundings(inter, group) * 2.0 ** -24
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if e < 0:
                continue
            (v1, m1), (v3, m3), (v2, m2) = [ref.values(*[None if a is None else a[e] for a in w]) for w in ws]
            a = x[t].double()
            gate, u = v1 @ a, v3 @ a
            f, u25 = 4 * torch.tanh(gate / 4) / (1 + torch.exp(-gate)), 25 * torch.tanh(u / 25)
            h = f * u25
            eh = 17 * 2.0 ** -24 * h.abs() + 1.01 * (1.1 * up * (m1 @ a.abs()) * u25.abs() + f.abs() * up * (m3 @ a.abs()))
            w = float(wts[t, k])
            want[t] += w * (v2 @ h)
            tol[t] += w * (v2.abs() @ eh + down * (m2 @ h.abs())) + K * 2.0 ** -24 * w * (v2 @ h).abs()
        if t >= 60:
            break
    rows = min(T, 61)
    err = (y[:rows].double() - want[:rows]).abs()
    assert bool((err <= tol[:rows] + 2.0 ** -24 * want[:rows].abs()).all()), float((err / tol[:rows]).max())


def test_a_layer_captured_and_replayed_and_on_two_streams(k3g):
    T, K, E, n, inter = 50, 4, 24, 256, 192
    g = gen(9)
    ws = [k3g.int4(*ref.random_weights(g, (E, r), c, 32, torch.float16, True)) for r, c in ((inter, n), (inter, n), (n, inter))]
    x, wts = torch.zeros(T, n, device="cuda"), torch.zeros(T, K, device="cuda")
    idx = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    cap, eager = layer_buffers(k3g, T, K, E, n, inter), layer_buffers(k3g, T, K, E, n, inter)
    layer(k3g, eager, x, idx, wts, *ws, K)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        layer(k3g, cap, x, idx, wts, *ws, K)
    for i in range(3):
        x.copy_(torch.randn(T, n, device="cuda", generator=g))
        wts.copy_(torch.rand(T, K, device="cuda", generator=g))
        idx.copy_(torch.randint(0, E, (T, K), device="cuda", generator=g))
        graph.replay()
        layer(k3g, eager, x, idx, wts, *ws, K)
        torch.cuda.synchronize()
        assert torch.equal(cap["y"], eager["y"]), i
    want = eager["y"].clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, b in zip(streams, (cap, eager)):
        b["y"].zero_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer(k3g, b, x, idx, wts, *ws, K)
    torch.cuda.synchronize()
    assert torch.equal(cap["y"], want) and torch.equal(eager["y"], want)
    assert np.isfinite(float(want.sum()))
