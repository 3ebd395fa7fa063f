"""SiTU of gates and up-products at and past the ends of fp32's range (GPU): the formula
4 tanh(g/4) sigmoid(g) 25 tanh(u/25) is bounded, so an infinite g or u has an ordinary value."""
import numpy as np
import pytest

from tests import mx_ref
from tests.helpers import REL, situ64, situ_tolerance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# The one nonzero weight of rows of w1 and w3 (e2m1 code, scale byte), with a = 1: g or u is +-6 2^(s-127) and, of a
# scaled a = 2^100, up to +-2^229, which fp32 holds as an infinity.
ENDS = [(c, s) for c in (7, 15, 1, 9) for s in (20, 126, 130, 151, 152, 154, 200, 254)]


def end_rows(rng, rows, n):
    """w1 or w3 [rows][n]: e2m1 codes one a byte, scale bytes; row r has ENDS[r] in column 0, or is random and small."""
    c, s = np.zeros((rows, n), np.uint8), np.full((rows, n // 32), 127, np.uint8)
    for r in range(rows):
        if r < len(ENDS):
            c[r, 0], s[r, 0] = ENDS[rng.integers(0, len(ENDS))] if r >= 32 else ENDS[r]
    return c, s


@pytest.mark.parametrize("hfmt", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T", [1, 70])
def test_glu_of_infinite_gates(k3g, T, fmt, hfmt):
    rng = np.random.default_rng(3)
    n, inter = 512, 64
    off, stride = k3g.bank_layout(n, inter)
    bank, per = np.zeros(stride, np.uint8), []
    for t in range(2):
        c, s = end_rows(rng, inter, n)
        order = rng.permutation(32)
        c[:32], s[:32] = c[order], s[order]  # gates and up-products of every kind side by side
        if t == 1:  # the second group: ordinary gates with infinite up-products, and the other way round
            c[32:], s[32:] = c[:32], s[:32]
        else:
            c[32:, 0] = 5
        p = mx_ref.pack(c, 0)
        bank[off[2 * t]:off[2 * t] + p.size], bank[off[2 * t + 1]:off[2 * t + 1] + s.size] = p.ravel(), s.ravel()
        per.append(mx_ref.values(p, s, 0))
    ac = np.zeros((T, n), np.uint8)
    ac[:, 0] = 2 if fmt == 0 else 0x38  # 1
    asc = np.full((T, n // 32), 127, np.uint8)
    asc[T // 2:] = 227
    h = k3g.mx_empty(T, inter, hfmt)
    print(f"infinite gates T={T} fmt={fmt} h={hfmt}", flush=True)
    k3g.k3g_mx_grouped_glu(h, k3g.mx(dev(mx_ref.pack(ac, fmt)), dev(asc), fmt), k3g.bank_struct(dev(bank), 1, n, inter),
                           dev(np.array([0, T], np.int32)))
    av = mx_ref.values(mx_ref.pack(ac, fmt), asc, fmt)
    g, ng = mx_ref.product(av, per[0])
    u, nu = mx_ref.product(av, per[1])
    assert (np.abs(g) > 2.0 ** 128).any() and (np.abs(u) > 2.0 ** 128).any()
    mx_ref.check_quantised(h.codes.cpu().numpy(), h.scales.cpu().numpy(), situ64(g, u), situ_tolerance(g, u, ng, nu), hfmt, "h")


@pytest.mark.parametrize("mode", ["exact", "lut"])
def test_expert_of_infinite_gates(k3g, mode):
    rng = np.random.default_rng(4)
    n, inter = 256, 64
    ex, val = {}, []
    for t, name in enumerate(("w1", "w3")):
        c, s = end_rows(rng, inter, n)
        order = rng.permutation(32)
        c[:32], s[:32] = c[order], s[order]
        p = mx_ref.pack(c, 0)
        ex[name + "p"], ex[name + "s"] = dev(p), dev(s)
        val.append(mx_ref.values(p, s, 0))
    w2c, w2s = mx_ref.mx_bytes(rng, n, inter, 0, 110, 118)
    ex["w2p"], ex["w2s"] = dev(w2c), dev(w2s)
    x = np.zeros((1, n), np.float32)
    x[0, 0] = 2.0 ** 100
    m = k3g.EXACT | (k3g.DECODE_LUT if mode == "lut" else 0)
    y = torch.empty(n, device="cuda")
    ws = k3g.workspace(k3g.OP_EXPERT_GLU, k3g.shape(n_tokens=1, latent=n, inter=inter, mode=m))
    print(f"expert of infinite gates {mode}", flush=True)
    k3g.k3g_expert_glu(y, dev(x[0]), ex, m, ws)
    g, ng = mx_ref.product(x.astype(np.float64), val[0])
    u, nu = mx_ref.product(x.astype(np.float64), val[1])
    h, th = situ64(g, u), situ_tolerance(g, u, ng, nu)
    w2 = mx_ref.values(w2c, w2s, 0)
    ref, nrm = mx_ref.product(h, w2)
    assert (np.abs(g) > 2.0 ** 128).any()
    assert np.all(np.abs(y.cpu().numpy() - ref) <= REL * nrm + th @ np.abs(w2).T)
