"""Every kernel that the microscaled products choose from, on the GPU against 64 bits. The sizes are picked by the tile
they select, which each test asserts, so that a change of the rules cannot leave one untested. Widths: 512 (rows of
whole four stages, whose workgroups run on from item to item, scale bytes on 16-byte addresses), 480 (the same with the
last group missing, so scale bytes anywhere), 544 (a fifth stage of one group: every item starts anew) and 2048.

The bar is the library's 1e-5 * sum |a||w|, and half a step of a bf16 output (2^-8).
"""
import numpy as np
import pytest

from tests import mx_dev, mx_ref
from tests.helpers import REL, situ64, situ_tolerance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def check(y, a, w, what):
    ref, nrm = a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()
    bad = ~((y.double() - ref).abs() <= REL * nrm + HALF[y.dtype] * (ref.abs() + REL * nrm))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:3].tolist()}"
    assert bool((y[nrm == 0] == 0).all()), f"{what}: nonzero where every group is left out"


DENSE = [
    # format, tokens, outputs, tile (outputs, tokens)
    (0, 3, 100, (16, 16)), (1, 3, 100, (16, 16)),
    (0, 9, 16401, (32, 16)), (1, 9, 16401, (32, 16)),
    (0, 31, 3000, (32, 32)), (1, 31, 3000, (32, 32)),
    (0, 63, 3000, (32, 64)), (1, 63, 3000, (32, 64)),
    (0, 250, 3584, (128, 32)), (1, 250, 3584, (128, 32)),
    (0, 505, 3579, (128, 64)), (1, 1020, 4472, (128, 64)),  # MXFP8: 560 items, more than run at once
    (0, 1010, 3584, (128, 128)),
    (0, 2500, 3570, (256, 128)), (1, 4090, 6136, (256, 128)),  # 280 and 768 items on 256 CUs
    (0, 4090, 6136, (256, 256)),  # 384
    (0, 20, 110005, (128, 32)), (1, 20, 110005, (128, 32)),  # few tokens, 860 items
    (0, 40, 70004, (128, 64)), (1, 40, 70004, (128, 64)),  # 547
]


@pytest.mark.parametrize("n", [512, 480, 544, 2048])
@pytest.mark.parametrize("fmt,T,rows,tile", DENSE)
def test_dense(k3g, fmt, T, rows, tile, n):
    assert k3g.k3g_probe_mx_form(fmt, T, rows) == tile
    g = torch.Generator(device="cuda").manual_seed(T + n)
    ac, asc = mx_dev.mx_bytes(g, T, n, fmt)
    wc, wsc = mx_dev.mx_bytes(g, rows, n, 0)
    asc[T // 2], wsc[rows // 3] = 255, 255
    a, w = k3g.mx(ac, asc, fmt), k3g.mxfp4(wc, wsc)
    av, wv = mx_dev.values(ac, asc, fmt), mx_dev.values(wc, wsc, 0)
    for ty, pad in ((torch.float32, 3), (torch.bfloat16, 8)):
        buf = torch.full((T + 2, rows + pad), 7.0, device="cuda", dtype=ty)
        y = buf[1:T + 1, :rows]
        print(f"dense fmt={fmt} T={T} rows={rows} n={n} {ty}", flush=True)
        k3g.k3g_mx_matmul(y, a, w)
        check(y, av, wv, str(ty))
        assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all()) and bool((buf[:, rows:] == 7).all())
    # the same bits again, in another order of the tokens, and with fewer of them
    y = y.contiguous()
    again = torch.empty_like(y)
    k3g.k3g_mx_matmul(again, a, w)
    assert torch.equal(again, y)
    order = torch.randperm(T, device="cuda", generator=g)
    k3g.k3g_mx_matmul(again, k3g.mx(ac[order].contiguous(), asc[order].contiguous(), fmt), w)
    assert torch.equal(again, y[order])
    t = T - 2
    if k3g.k3g_probe_mx_form(fmt, t, rows) == tile:
        k3g.k3g_mx_matmul(again[:t], k3g.mx(ac[:t], asc[:t], fmt), w)
        assert torch.equal(again[:t], y[:t])


GROUPED = [
    # format, experts, rows an expert on average, tile: more items than run at once
    (0, 300, 2, (128, 32)), (1, 300, 2, (128, 32)),
    (0, 120, 12, (128, 64)), (1, 120, 12, (128, 64)),
    (0, 80, 40, (256, 128)), (1, 80, 40, (256, 128)),
]


@pytest.mark.parametrize("latent", [512, 480, 544])
@pytest.mark.parametrize("fmt,E,per,tile", GROUPED)
def test_grouped(k3g, fmt, E, per, tile, latent):
    inter, P, k = 992, E * per, 2
    assert k3g.k3g_probe_mx_form(fmt, P, inter, E) == tile and k3g.k3g_probe_mx_form(fmt, P, inter, E, glu=True) == tile
    g = torch.Generator(device="cuda").manual_seed(E + latent)
    rng = np.random.default_rng(E + latent)
    share = rng.random(E) * (rng.random(E) > 0.1) + 1e-9
    counts = rng.multinomial(P - 4, share / share.sum())
    off = np.concatenate([[1], 1 + np.cumsum(counts)]).astype(np.int32)  # a row before the groups, three behind
    offd = torch.from_numpy(off).cuda()
    perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    o, stride = k3g.bank_layout(latent, inter)
    bank = torch.zeros(E, stride, dtype=torch.uint8, device="cuda")
    parts = []
    for t, (rows, cols) in enumerate(((inter, latent), (inter, latent), (latent, inter))):
        c, s = mx_dev.mx_bytes(g, E * rows, cols, 0, 112, 118)
        bank[:, o[2 * t]:o[2 * t] + rows * cols // 2] = c.view(E, -1)
        bank[:, o[2 * t + 1]:o[2 * t + 1] + rows * cols // 32] = s.view(E, -1)
        parts.append((c.view(E, rows, -1), s.view(E, rows, -1)))
    b = k3g.bank_struct(bank.view(-1), E, latent, inter)
    weights = lambda t, e: mx_dev.values(parts[t][0][e], parts[t][1][e], 0)  # noqa: E731
    lo, hi = (118, 126) if fmt == 0 else (112, 118)
    ac, asc = mx_dev.mx_bytes(g, P // k, latent, fmt, lo, hi)
    hc, hs = mx_dev.mx_bytes(g, P, inter, fmt)
    a, hin = k3g.mx(ac, asc, fmt), k3g.mx(hc, hs, fmt)
    av, hv = mx_dev.values(ac, asc, fmt), mx_dev.values(hc, hs, fmt)
    y = torch.full((P, inter), 7.0, device="cuda")
    z = torch.full((P, latent), 7.0, device="cuda", dtype=torch.bfloat16)
    h = [k3g.mx_empty(P, inter, f) for f in (0, 1)]
    print(f"grouped fmt={fmt} E={E} P={P} latent={latent}", flush=True)
    k3g.k3g_mx_grouped_matmul(y, a, b, k3g.W3, offd, perm=perm, top_k=k)
    k3g.k3g_mx_grouped_matmul(z, hin, b, k3g.W2, offd)
    for q in h:
        q.codes.fill_(77), q.scales.fill_(9)
        k3g.k3g_mx_grouped_glu(q, a, b, offd, perm=perm, top_k=k)
    src = (perm // k).long()
    picked = {int(counts.argmax()), *rng.integers(0, E, 12).tolist()}
    codes, scales = [q.codes.cpu().numpy() for q in h], [q.scales.cpu().numpy() for q in h]
    for e in range(E):
        p0, p1 = int(off[e]), int(off[e + 1])
        if p1 == p0:
            continue
        x = av[src[p0:p1]]
        check(y[p0:p1], x, weights(1, e), f"w3 of expert {e}")
        check(z[p0:p1], hv[p0:p1], weights(2, e), f"w2 of expert {e}")
        if e in picked:
            (gate, ng), (up, nu) = (((x @ w.t().contiguous()).cpu().numpy(), (x.abs() @ w.abs().t().contiguous()).cpu().numpy())
                                    for w in (weights(0, e), weights(1, e)))
            for f in (0, 1):
                mx_ref.check_quantised(codes[f][p0:p1], scales[f][p0:p1], situ64(gate, up), situ_tolerance(gate, up, ng, nu), f,
                                       f"h of expert {e}")
    left = [0, P - 3, P - 2, P - 1]
    assert bool((y[left] == 7).all()) and bool((z[left] == 7).all())
    assert all((c[left] == 77).all() and (s[left] == 9).all() for c, s in zip(codes, scales))
    # the rows of each group the other way round: the same bits, the other way round
    back = torch.cat([torch.arange(0, 1), *[torch.arange(int(off[e + 1]) - 1, int(off[e]) - 1, -1) for e in range(E)],
                      torch.arange(P - 3, P)]).cuda()
    y2, h2 = torch.full_like(y, 7.0), k3g.mx_empty(P, inter, 1)
    h2.codes.fill_(77), h2.scales.fill_(9)
    k3g.k3g_mx_grouped_matmul(y2, a, b, k3g.W3, offd, perm=perm[back].contiguous(), top_k=k)
    k3g.k3g_mx_grouped_glu(h2, a, b, offd, perm=perm[back].contiguous(), top_k=k)
    assert torch.equal(y2, y[back]) and torch.equal(h2.codes, h[1].codes[back]) and torch.equal(h2.scales, h[1].scales[back])


def test_every_tile_is_named_above(k3g):
    """Over many sizes the rules choose no tile that the tests above do not name."""
    named = {(f, t) for f, _, _, t in DENSE}
    rng = np.random.default_rng(1)
    for _ in range(20000):
        T, rows = (int(2 ** rng.uniform(0, 14)) for _ in range(2))
        f = int(rng.integers(0, 2))
        assert (f, k3g.k3g_probe_mx_form(f, T, rows)) in named, (f, T, rows)
        E = int(rng.integers(1, 2049))
        for glu in (False, True):
            assert (f, k3g.k3g_probe_mx_form(f, T, rows, E, glu)) in {(f, t) for f, _, _, t in GROUPED}
