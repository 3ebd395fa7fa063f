"""Every kernel of the int4 products, by sizes that each asserts to select it: zeros of any byte, fp32's
smallest entries, codes that equal their zero, infinities, offsets and sources out of range."""
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


def rows_at(x, aligned):
    """x's rows on 16-byte addresses, or the same rows off them (fp32 rows are always on 4-byte ones)."""
    if aligned:
        return x.contiguous()
    b = torch.zeros(x.numel() + x.shape[0] + 1, dtype=x.dtype, device="cuda")
    v = b[1:].view(x.shape[0], -1)[:, :x.shape[1]]
    return v.copy_(x)


def forms(xt, n):
    """(form, aligned, experts (0: dense), rows of y, outputs) that reach every kernel with rows of n columns (n at most
    2048: the rule goes by other sizes), dense and grouped."""
    wide = [((256, 64), True)] if xt == F32 else [((256, 128), True), ((256, 64), False)]
    dense = [((8, 1), True, 1, 70), ((16, 16), True, 7, 130), ((32, 16), True, 9, 4200), ((64, 32), True, 33, 7000)]
    dense += [] if xt == F32 else [((64, 64), True, 141, 4500)]
    dense += [(f, a, 385, 10753) for f, a in wide]
    grouped = [((8, 1), True, 40, 20, 70), ((32, 16), True, 5, 37, 70), ((64, 32), True, 4, 70, 100)]
    grouped += [(f, a, 4, 1300, 2700) for f, a in wide]
    return [(f, a, 0, T, rows) for f, a, T, rows in dense] + grouped


def product(k3g, form, aligned, E, T, rows, n, x, *w, off=None, perm=None, top_k=1, mark=7.0):
    """The product's output in fp32, its kernel asserted; E = 0: dense."""
    assert k3g.k3g_probe_int4_form(x.dtype, T, rows, n, E, aligned=aligned) == form
    x = rows_at(x, aligned)
    assert (x.data_ptr() % 16 == 0 and (x.shape[0] == 1 or x.stride(0) * x.element_size() % 16 == 0)) == aligned
    b = torch.full((T + 2, rows + 3), mark, device="cuda")
    y = b[1:T + 1, 1:rows + 1]
    if E:
        k3g.k3g_int4_grouped_matmul(y, x, k3g.int4(*w), off, perm=perm, top_k=top_k)
    else:
        k3g.k3g_int4_matmul(y, x, k3g.int4(*w))
    assert bool((b[[0, -1]] == mark).all() and (b[:, [0, -1, -2]] == mark).all())
    return y


def even(E, T):
    """Offsets of E groups of about as many rows, and the expert of each row."""
    off = (torch.arange(E + 1, device="cuda") * T // E).int()
    return off, torch.bucketize(torch.arange(T, device="cuda"), off[1:].long(), right=True)


def expect(x, w, E, T, expert):
    """The product in 64 bits and its magnitudes."""
    if not E:
        v, m = ref.values(*w)
        return x.double() @ v.t().contiguous(), x.double().abs() @ m.t().contiguous()
    rows = w[0].shape[1]
    want, mag = [torch.empty(T, rows, dtype=torch.float64, device="cuda") for _ in range(2)]
    for e in range(E):
        s = expert == e
        v, m = ref.values(*[None if t is None else t[e] for t in w])
        want[s], mag[s] = x[s].double() @ v.t().contiguous(), x[s].double().abs() @ m.t().contiguous()
    return want, mag


def any_zeros(g, lead, n, group):
    """Weights with zeros of any byte, every range's ends among them, and scales that are powers of two."""
    packed, s, _ = ref.random_weights(g, lead, n, group, B16, False, exact=True)
    z = torch.randint(0, 256, s.shape, dtype=torch.uint8, device="cuda", generator=g)
    ends = torch.tensor([0, 15, 127, 128, 129, 143, 144, 255], dtype=torch.uint8, device="cuda")
    return packed, s, torch.where(torch.rand(s.shape, device="cuda", generator=g) < 0.3, ends[(z % 8).long()], z)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", TYPES, ids=name)
def test_zeros_of_any_byte(k3g, xt, group):
    """Zeros from 0 to 255, the codes' whole range and beyond it, rows of one group and of more: whole numbers, exact."""
    for n in (group, 384, 640):
        for form, aligned, E, T, rows in forms(xt, n):
            g = gen(T + rows + group)
            w = any_zeros(g, (E, rows) if E else (rows,), n, group)
            x = torch.randint(-4, 5, (T, n), device="cuda", generator=g).to(xt)
            off, expert = even(E, T) if E else (None, None)
            y = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
            assert bool((y.double() == expect(x, w, E, T, expert)[0]).all()), (form, E, n)


@pytest.mark.parametrize("xt", TYPES, ids=name)
def test_zeros_of_any_byte_in_gated_products(k3g, xt):
    """w1 with such zeros and w3 without any, and the other way round: both sums are exact, so h is off by the gate's
    functions alone (16 steps taken, and h's own rounding)."""
    n, group = 448, 64
    for form, aligned, E, R, rows in [f for f in forms(xt, n) if f[2]]:
        g = gen(R + rows)
        one, two = any_zeros(g, (E, rows), n, group), ref.random_weights(g, (E, rows), n, group, B16, False, exact=True)
        for w in (one, two):
            w[1].mul_(2.0 ** -10)
        x = rows_at(torch.randint(-4, 5, (R, n), device="cuda", generator=g).to(xt), aligned)
        off, expert = even(E, R)
        for w1, w3 in ((one, two), (two, one)):
            assert k3g.k3g_probe_int4_form(xt, R, rows, n, E, True, aligned=aligned) == form
            h = k3g.k3g_int4_grouped_glu(torch.empty(R, rows, device="cuda"), x, k3g.int4(*w1), k3g.int4(*w3), off)
            gate, up = [expect(x, w, E, R, expert)[0] for w in (w1, w3)]
            want = 4 * torch.tanh(gate / 4) / (1 + torch.exp(-gate)) * 25 * torch.tanh(up / 25)
            assert bool(((h.double() - want).abs() <= 17 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all()), form


def test_fp32_entries_down_to_the_smallest(k3g):
    """fp32 from its smallest step to 2^-110: the vector kernel takes them whole; the matrix cores' three bf16 parts
    end at 2^-133, so an entry loses less than that."""
    n, group = 256, 32
    for form, aligned, E, T, rows in forms(F32, n):
        g = gen(T + rows)
        w = ref.random_weights(g, (E, rows) if E else (rows,), n, group, F32, True)
        w[1].mul_(2.0 ** 20)
        e = torch.randint(-149, -109, (T, n), device="cuda", generator=g).double()
        x = (torch.randn(T, n, device="cuda", generator=g).double() * torch.exp2(e)).float()
        off, expert = even(E, T) if E else (None, None)
        y = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
        want, mag = expect(x, w, E, T, expert)
        lost = torch.zeros_like(want)
        if form != (8, 1):
            sums = ref.values(*w)[0].abs().sum(-1)  # of |scale * (code - zero)|
            lost += 2.0 ** -133 * (sums[expert] if E else sums)
        steps = ref.roundings(n, group)
        # products of codes and sums are multiples of 2^-149 as x is; once scaled they lose half of it an addition:
        # one a group, 8 wavefronts, the output
        tol = steps * 2.0 ** -24 * mag + lost + (n // group + 9) * 2.0 ** -150
        err = (y.double() - want).abs()
        assert bool((err <= tol).all()), (form, E, float((err / tol).max()))
        y3 = product(k3g, form, aligned, E, T, rows, n, x * 2.0 ** 40, *w, off=off)
        ref.check(y3, want * 2.0 ** 40, mag * 2.0 ** 40, steps)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", TYPES, ids=name)
def test_weights_of_value_zero_and_large_entries(k3g, xt, group):
    """Rows whose codes all equal their zero, between ordinary ones, and entries of any size: what is left is within
    the sums' roundings of scale * (code + zero) * |x|."""
    n = 1152
    for form, aligned, E, T, rows in forms(xt, n):
        g = gen(T + rows)
        w = ref.random_weights(g, (E, rows) if E else (rows,), n, group, F32, True)
        z = w[2].repeat_interleave(group, -1)
        w[0][..., ::3, :] = (z[..., 0::2] | z[..., 1::2] << 4)[..., ::3, :]
        x = torch.randn(T, n, device="cuda", generator=g)
        x = torch.where(torch.rand(T, n, device="cuda", generator=g) < 0.01, 1000 * x, x).to(xt)
        off, expert = even(E, T) if E else (None, None)
        y = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
        want, mag = expect(x, w, E, T, expert)
        assert bool((want[:, ::3] == 0).all())
        ref.check(y, want, mag, ref.roundings(n, group))


@pytest.mark.parametrize("xt", TYPES, ids=name)
def test_not_finite(k3g, xt):
    """A token with an infinity or a NaN has no finite output, the tokens beside it keep theirs; likewise a scale."""
    n = 384
    for form, aligned, E, T, rows in forms(xt, n):
        g = gen(T)
        w = ref.random_weights(g, (E, rows) if E else (rows,), n, 32, F32, True)
        x = torch.randn(T, n, device="cuda", generator=g).to(xt)
        off, expert = even(E, T) if E else (None, None)
        good = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
        bad = sorted({T // 4, T // 2, T - 1})
        for t, c, v in zip(bad, (7, 380, 100), (float("inf"), float("nan"), -float("inf"))):
            x[t, c] = v
        hit = torch.zeros(T, dtype=torch.bool, device="cuda")
        hit[bad] = True
        y = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
        assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], good[~hit]), (form, E)
        w[1][..., 11, 4], w[1][..., rows - 1, 0] = float("nan"), float("inf")
        y = product(k3g, form, aligned, E, T, rows, n, x, *w, off=off)
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[[11, rows - 1]] = False
        assert torch.equal(y[~hit][:, keep], good[~hit][:, keep]) and not torch.isfinite(y[:, ~keep]).any(), (form, E)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("xt", TYPES, ids=name)
def test_groups_and_sources_out_of_range(k3g, xt, glu):
    """Offsets outside the rows and a perm outside x's: clipped, in every kernel. Rows in no group stay as they were, and so
    does what lies around y."""
    n = 160
    for form, aligned, E, R, rows in [f for f in forms(xt, n) if f[2]]:
        g = gen(R)
        w = [k3g.int4(*ref.random_weights(g, (E, rows), n, 32, B16, True)) for _ in range(2)]
        x = rows_at(torch.randn(R, n, device="cuda", generator=g).to(xt), aligned)
        perm = torch.full((R,), 2**31 - 1, dtype=torch.int32, device="cuda")
        perm[::2], perm[1::4] = -5, -2**31
        inner = torch.sort(torch.randint(-R, 3 * R, (E - 1,), device="cuda", generator=g)).values
        for lo, hi in ((-7, R + 90), (0, 2**31 - 1), (-2**31, 3 * R), (R, R), (R + 9, R + 9), (5, R - 3)):
            off = torch.cat([torch.tensor([lo], device="cuda"), inner.clamp(lo, hi), torch.tensor([hi], device="cuda")]).int()
            assert k3g.k3g_probe_int4_form(xt, R, rows, n, E, glu, aligned=aligned) == form
            b = torch.full((R + 2, rows + 1), 7.0, device="cuda")
            y = b[1:R + 1, :rows]
            for p in (perm, None):
                if glu:
                    k3g.k3g_int4_grouped_glu(y, x, *w, off, perm=p, top_k=1)
                else:
                    k3g.k3g_int4_grouped_matmul(y, x, w[0], off, perm=p, top_k=1)
                assert bool((b[[0, -1]] == 7).all() and (b[:, -1] == 7).all()), form
                assert bool((y[:max(lo, 0)] == 7).all() and (y[max(min(hi, R), 0):] == 7).all()), form
