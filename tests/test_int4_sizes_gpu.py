"""Launches of the int4 products that sizes select within a kernel: a wavefront to each item, more tiles than
workgroups, rows of two loads of the vector kernel; codes and rows past 32 bits in every kernel."""
import pytest
import torch

from tests import int4_ref as ref

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
F32, B16, F16 = TYPES
name = lambda t: str(t)[6:] if isinstance(t, torch.dtype) else None  # noqa: E731


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(w, e):
    return [None if t is None else t[e] for t in w]


def groups(g, E, T):
    """Ragged offsets that leave three rows at either end, an empty group among them, as a list too."""
    cut = torch.sort(torch.randint(3, T - 2, (E - 1,), generator=g, device="cuda")).values
    cut[1] = cut[2]
    off = torch.cat([torch.tensor([3], device="cuda"), cut, torch.tensor([T - 3], device="cuda")]).int()
    return off, off.tolist()


def items(o, tok):
    """The tiles of `tok` rows that the groups have."""
    return sum(-(-(b - a) // tok) for a, b in zip(o, o[1:]))


def check_dense(k3g, g, xt, T, n, rows, group, st, zeros, aligned=True):
    """Whole numbers, exact; the rows around y's stay."""
    w = ref.random_weights(g, (rows,), n, group, st, zeros, exact=True)
    x = torch.randint(-4, 5, (T, n + (0 if aligned else 1)), device="cuda", generator=g).to(xt)[:, :n]
    b = torch.full((T + 2, rows + 1), 7.0, device="cuda")
    k3g.k3g_int4_matmul(b[1:T + 1, :rows], x, k3g.int4(*w))
    assert torch.equal(b[1:T + 1, :rows], (x.double() @ ref.values(*w)[0].t().contiguous()).float()), (T, n, rows)
    assert bool((b[[0, -1]] == 7).all() and (b[:, rows] == 7).all())


def check_grouped(k3g, g, xt, E, T, n, rows, group, st, zeros, off, o, aligned=True):
    """Whole numbers through perm, exact; rows in no group stay."""
    w = ref.random_weights(g, (E, rows), n, group, st, zeros, exact=True)
    x = torch.randint(-4, 5, (T, n + (0 if aligned else 1)), device="cuda", generator=g).to(xt)[:, :n]
    perm = torch.randperm(T, generator=g, device="cuda").int()
    y = torch.full((T, rows), 7.0, device="cuda")
    k3g.k3g_int4_grouped_matmul(y, x, k3g.int4(*w), off, perm=perm)
    a, want = x.double()[perm.long()], torch.full((T, rows), 7.0, device="cuda")
    for e in range(E):
        if o[e + 1] > o[e]:
            want[o[e]:o[e + 1]] = (a[o[e]:o[e + 1]] @ ref.values(*matrix(w, e))[0].t().contiguous()).float()
    assert torch.equal(y, want), (E, T, n, rows)


def check_glu(k3g, g, xt, E, T, n, rows, group, st, off, o, aligned=True):
    """Exact sums (scales of 2^-13 to 2^-9), so h is off by the gate's functions alone (16 steps) and its rounding."""
    w1, w3 = [ref.random_weights(g, (E, rows), n, group, st, z, exact=True) for z in (True, False)]
    w1[1].mul_(2.0 ** -10), w3[1].mul_(2.0 ** -10)
    x = torch.randint(-4, 5, (T, n + (0 if aligned else 1)), device="cuda", generator=g).to(xt)[:, :n]
    h = torch.full((T, rows), 7.0, device="cuda")
    k3g.k3g_int4_grouped_glu(h, x, k3g.int4(*w1), k3g.int4(*w3), off)
    a, want = x.double(), torch.full((T, rows), 7.0, dtype=torch.float64, device="cuda")
    for e in range(E):
        if o[e + 1] > o[e]:
            s = slice(o[e], o[e + 1])
            gate, up = [a[s] @ ref.values(*matrix(w, e))[0].t().contiguous() for w in (w1, w3)]
            want[s] = 4 * torch.tanh(gate / 4) / (1 + torch.exp(-gate)) * 25 * torch.tanh(up / 25)
    assert bool(((h.double() - want).abs() <= 17 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all()), (E, T, n, rows)


# ---- a wavefront to each item -------------------------------------------------------------

# (form, aligned, tokens, outputs) of more than 4096 items
ALONE_DENSE = {F32: [((32, 16), True, 9, 131101), ((64, 32), True, 75, 87500)],
               B16: [((32, 16), True, 9, 131101), ((64, 64), True, 19, 262200), ((64, 64), False, 75, 131073)]}
ALONE_DENSE[F16] = ALONE_DENSE[B16]
# (form, experts, rows, outputs of the grouped and of the gated product)
ALONE_GROUPED = [((32, 16), 64, 500, 1400, 700), ((64, 32), 64, 900, 2850, 1430)]


@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("group,n", [(32, 32), (32, 352), (64, 192), (64, 1216), (128, 128), (128, 1408)])
def test_a_wavefront_to_each_item(k3g, xt, group, n):
    """Rows within one turn of 256 or 512 columns and over several with a ragged end."""
    g = gen(group + n)
    for form, aligned, T, rows in ALONE_DENSE[xt] if n < 1000 else ALONE_DENSE[xt][:1]:
        assert k3g.k3g_probe_int4_form(xt, T, rows, n, aligned=aligned) == form
        assert k3g.k3g_probe_int4_launch(xt, T, rows, n, group, aligned=aligned) == (4096, 1)
        check_dense(k3g, g, xt, T, n, rows, group, B16, group != 64, aligned)
    for form, E, T, rows, gated in ALONE_GROUPED:
        off, o = groups(g, E, T)
        for glu, r in ((False, rows), (True, gated)):
            assert k3g.k3g_probe_int4_form(xt, T, r, n, E, glu) == form
            assert k3g.k3g_probe_int4_launch(xt, T, r, n, group, E, glu) == (4096, 1)
            if glu:
                check_glu(k3g, g, xt, E, T, n, r, group, F16, off, o)
            else:
                assert items(o, form[1]) * -(-r // form[0]) > 1024  # (the groups' real ones; some wavefronts have none)
                check_grouped(k3g, g, xt, E, T, n, r, group, F32, group == 64, off, o)


# ---- more tiles than workgroups -----------------------------------------------------------

@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("group,n", [(32, 64), (32, 416), (64, 64), (64, 832), (128, 128), (128, 640)])
def test_more_tiles_than_workgroups(k3g, xt, group, n, aligned):
    """Workgroups go from tile to tile: the sources, the scales and the stages of one are used again by the next, rows of
    fewer groups than a turn has among them."""
    g = gen(group + n + 1)
    form = (256, 128) if aligned and xt != F32 else (256, 64)
    T, rows = 1029, 14851
    assert k3g.k3g_probe_int4_form(xt, T, rows, n, aligned=aligned) == form
    assert k3g.k3g_probe_int4_launch(xt, T, rows, n, group, aligned=aligned) == (512, 4)
    assert -(-T // form[1]) * -(-rows // 256) > 512
    check_dense(k3g, g, xt, T, n, rows, group, B16, group != 64, aligned)
    E, T = 9, 3000
    off, o = groups(g, E, T)
    for glu in (False, True):
        out = 128 if glu else 256
        rows = out * (540 // items(o, form[1])) + 70
        assert k3g.k3g_probe_int4_form(xt, T, rows, n, E, glu, aligned=aligned) == form
        assert items(o, form[1]) * -(-rows // out) > 512
        if glu:
            check_glu(k3g, g, xt, E, T, n, rows, group, F16, off, o, aligned)
        else:
            check_grouped(k3g, g, xt, E, T, n, rows, group, F32, group == 64, off, o, aligned)


# ---- rows of two loads of the vector kernel -------------------------------------------------

@pytest.mark.parametrize("st", TYPES, ids=name)
@pytest.mark.parametrize("xt", TYPES, ids=name)
@pytest.mark.parametrize("group,n", [(32, 16416), (64, 24704), (128, 32768), (32, 16384)])
def test_vector_kernel_of_long_rows(k3g, xt, st, group, n):
    """16416 to 32768 columns: a wavefront takes 4096 of them in two loads (16384: the last of one load)."""
    g = gen(group + n + 2)
    waves = -(-n // 2048) if n == 16384 else -(-n // 4096)
    for T in (1, 2) if xt == F32 else (1,):
        assert k3g.k3g_probe_int4_launch(xt, T, 37, n, group)[1] == 8 // waves * waves
        assert k3g.k3g_probe_int4_form(xt, T, 37, n) == (8, 1)
        check_dense(k3g, g, xt, T, n, 37, group, st, group == 64)
    E, T = 40, 20
    off, o = groups(g, E, T)
    for glu in (False, True):
        assert k3g.k3g_probe_int4_form(xt, T, 21, n, E, glu) == (8, 1)
    check_grouped(k3g, g, xt, E, T, n, 21, group, st, group != 64, off, o)
    check_glu(k3g, g, xt, E, T, n, 21, group, st, off, o)


# ---- past 32 bits ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def far_codes():
    """520 experts of 4096 x 4096: the codes pass 2^32 bytes at the 512th. All codes are 0 (of zeros 0) but three experts'."""
    E, m = 520, 4096
    packed = torch.zeros(E, m, m // 2, dtype=torch.uint8, device="cuda")
    g = gen(11)
    for e in (1, 512, 519):
        packed[e] = torch.randint(0, 256, (m, m // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.ones(E, m, m // 128, dtype=torch.bfloat16, device="cuda")
    yield packed, scales, torch.zeros_like(scales, dtype=torch.uint8)
    del packed, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("xt,form,aligned,T", [
    (t, f, a, T) for t in TYPES for f, a, T in
    [((8, 1), True, 200), ((32, 16), True, 700), ((64, 32), True, 6500)] +
    ([((256, 64), True, 42000)] if t == F32 else [((256, 128), True, 10500), ((256, 64), False, 42000)])], ids=str)
def test_codes_past_32_bits(k3g, far_codes, xt, form, aligned, T):
    """Nearly all rows belong to an expert before and two behind 2^32 bytes, the others to one of zeros only."""
    E, m = 520, 4096
    assert k3g.k3g_probe_int4_form(xt, T, m, m, E, aligned=aligned) == form
    own = min(T // 4, 150)
    ends = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ends[2:], ends[513:], ends[520:] = own, 2 * own, 3 * own  # experts 1, 512, 519
    if T > 3 * own:  # the rest lies in expert 0
        ends[1:] += T - 3 * own
    g = gen(T)
    x = torch.zeros(T, m + (0 if aligned else 1), dtype=xt, device="cuda")[:, :m]
    rest = T - 3 * own
    x[rest:] = torch.randint(-4, 5, (3 * own, m), device="cuda", generator=g).to(xt)
    y = torch.full((T, m), 7.0, dtype=torch.float32, device="cuda")
    k3g.k3g_int4_grouped_matmul(y, x, k3g.int4(*far_codes), ends)
    assert bool((y[:rest] == 0).all())
    for i, e in enumerate((1, 512, 519)):
        s = slice(rest + i * own, rest + (i + 1) * own)
        v = ref.values(far_codes[0][e], far_codes[1][e], far_codes[2][e])[0]
        assert torch.equal(y[s], (x[s].double() @ v.t().contiguous()).float()), e
    torch.cuda.empty_cache()


@pytest.mark.parametrize("xt,form,aligned,T,rows", [
    (t, f, a, T, rows) for t in TYPES for f, a, T, rows in
    [((16, 16), True, 12, 100), ((32, 16), True, 12, 4200), ((64, 32), True, 33, 7000)] +
    ([((8, 1), True, 2, 100), ((256, 64), True, 130, 14100)] if t == F32 else
     [((64, 64), True, 19, 16500), ((256, 128), True, 40, 32700), ((256, 64), False, 130, 14100)])], ids=str)
def test_rows_past_32_bits(k3g, xt, form, aligned, T, rows):
    """The last rows of x and y lie past 2^31 entries (and 2^32 bytes) of their buffers."""
    n = 128
    ld = ((1 << 31) // max(T - 3, 1) + rows) // 8 * 8 + (0 if aligned else 1)
    assert (T - 1) * ld > 1 << 31 and ld >= rows
    assert k3g.k3g_probe_int4_form(xt, T, rows, n, aligned=aligned) == form
    g = gen(T + rows)
    w = ref.random_weights(g, (rows,), n, 64, B16, True, exact=True)
    x = torch.empty((T - 1) * ld + n, dtype=xt, device="cuda").as_strided((T, n), (ld, 1))
    x.copy_(torch.randint(-4, 5, (T, n), device="cuda", generator=g))
    y = torch.empty((T - 1) * ld + rows, dtype=xt, device="cuda").as_strided((T, rows), (ld, 1))
    k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
    assert torch.equal(y, (x.double() @ ref.values(*w)[0].t().contiguous()).to(xt))
    del x, y
    torch.cuda.empty_cache()
