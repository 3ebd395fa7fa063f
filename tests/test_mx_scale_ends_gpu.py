"""Scale tensors that begin and end anywhere, through the tiled kernels (GPU): the first and last rows, whose bytes
share a dword with what lies outside the tensor, hold the scales that the others hold. The library's bar,
1e-5 * sum |a||w|, as in the other product tests."""
import pytest

from tests import mx_dev
from tests.helpers import REL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def check(y, a, w, what):
    ref, nrm = a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()
    bad = ~((y.double() - ref).abs() <= REL * nrm)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:3].tolist()}"


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 15, 18])
def test_dense(k3g, G, fmt):
    n, T, rows = 32 * G, 63, 10241
    g = torch.Generator(device="cuda").manual_seed(G)
    ac, asc = mx_dev.mx_bytes(g, T, n, fmt)
    wc, wsc = mx_dev.mx_bytes(g, rows, n, 0)
    av, wv = mx_dev.values(ac, asc, fmt), mx_dev.values(wc, wsc, 0)
    for at in range(4):
        a = k3g.mx(ac, mx_dev.placed(asc, at), fmt)
        w = k3g.mxfp4(wc, mx_dev.placed(wsc, 3 - at))
        y = torch.empty(T, rows, device="cuda")
        print(f"dense G={G} fmt={fmt} at={at}", flush=True)
        k3g.k3g_mx_matmul(y, a, w)
        check(y, av, wv, f"at {at}")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("per", [1, 12, 40])
@pytest.mark.parametrize("G", [1, 3, 6, 17])
def test_grouped(k3g, G, per, fmt):
    E, n, inter = 5, 32 * G, 160
    g = torch.Generator(device="cuda").manual_seed(G + per)
    P = E * per
    off = torch.arange(0, P + 1, per, dtype=torch.int32, device="cuda")
    ac, asc = mx_dev.mx_bytes(g, P, n, fmt)
    perm = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    av = mx_dev.values(ac, asc, fmt)
    codes, scales = inter * n // 2, inter * G
    for at in range(4):
        # w1 and w3 only (w2's place is not read): codes at multiples of 16, scales `at` bytes behind one
        stride = 2 * (codes + scales + 64) // 16 * 16 + 256
        offs = [0, codes + at, codes + 16 * (scales // 16 + 2), 2 * codes + 16 * (scales // 16 + 2) + 3 - at, 0, 0]
        bank = torch.full((E, stride), 0x5A, dtype=torch.uint8, device="cuda")
        w = []
        for t in range(2):
            c, s = mx_dev.mx_bytes(g, E * inter, n, 0)
            bank[:, offs[2 * t]:offs[2 * t] + codes] = c.view(E, -1)
            bank[:, offs[2 * t + 1]:offs[2 * t + 1] + scales] = s.view(E, -1)
            w.append(mx_dev.values(c, s, 0).view(E, inter, n))
        b = k3g.bank_struct(bank.view(-1), E, n, inter, offs, stride)
        a = k3g.mx(ac, mx_dev.placed(asc, at), fmt)
        for tensor in (k3g.W1, k3g.W3):
            y = torch.empty(P, inter, device="cuda")
            print(f"grouped G={G} per={per} fmt={fmt} at={at} tensor={tensor}", flush=True)
            k3g.k3g_mx_grouped_matmul(y, a, b, tensor, off, perm=perm)
            for e in range(E):
                check(y[e * per:(e + 1) * per], av[perm[e * per:(e + 1) * per].long()], w[tensor][e], f"at {at}, expert {e}")
        h = [k3g.mx_empty(P, inter, 1) for _ in range(2)]
        k3g.k3g_mx_grouped_glu(h[0], a, b, off, perm=perm)
        # the same experts with every scale tensor at a multiple of 256
        o2, st2 = k3g.bank_layout(n, inter)
        bank2 = torch.zeros(E, st2, dtype=torch.uint8, device="cuda")
        for i, size in ((0, codes), (1, scales), (2, codes), (3, scales)):
            bank2[:, o2[i]:o2[i] + size] = bank[:, offs[i]:offs[i] + size]
        k3g.k3g_mx_grouped_glu(h[1], k3g.mx(ac, asc, fmt), k3g.bank_struct(bank2.view(-1), E, n, inter), off, perm=perm)
        assert torch.equal(h[0].codes, h[1].codes) and torch.equal(h[0].scales, h[1].scales)
