"""Routed pairs on the GPU: the sort against a count in plain numpy, the rows and
their gradients against the formulas in 64 bits, and the gradients against differences."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def order(idx, E):
    """offsets, perm, inv of idx [T][K] (numpy), by going through the experts."""
    flat = idx.reshape(-1)
    perm, offsets = [], [0]
    where = {}
    for q, e in enumerate(flat.tolist()):
        where.setdefault(e, []).append(q)
    for e in range(E):
        perm += where.get(e, [])
        offsets.append(len(perm))
    inv = np.full(flat.size, -1, np.int32)
    inv[perm] = np.arange(len(perm))
    return (np.array(offsets, np.int32), np.array(perm + [-1] * (flat.size - len(perm)), np.int32), inv.reshape(idx.shape))


def run_sort(k3g, idx, E, stream=None):
    T, K = idx.shape
    ws = k3g.workspace(k3g.OP_MOE_SORT, k3g.shape(n_tokens=T, top_k=K, n_experts=E))
    ws.fill_(0xA5)
    off = torch.full((E + 1,), 77, dtype=torch.int32, device="cuda")
    perm = torch.full((T * K,), 77, dtype=torch.int32, device="cuda")
    inv = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
    return k3g.k3g_moe_sort(off, perm, inv, idx, ws, stream=stream)


# one workgroup of 256 and of 1024 threads, its last pair, one more; several chunks, a ragged last one; ids at both
# ends, one expert for all, experts that nobody names, dropped pairs, the same expert twice in a token
SORTS = [(1, 1, 1, "flat"), (1, 16, 896, "flat"), (3, 5, 7, "twice"), (16, 16, 64, "flat"), (257, 1, 2, "flat"),
         (64, 16, 896, "drop"), (61, 17, 2048, "flat"), (256, 16, 896, "flat"), (257, 16, 896, "twice"),
         (4097, 1, 1, "flat"), (1000, 64, 33, "one"), (511, 8, 1025, "none"), (8191, 16, 896, "drop"), (40000, 30, 5, "drop"),
         (70001, 16, 300, "flat")]


@pytest.mark.parametrize("T,K,E,kind", SORTS)
def test_sort(k3g, T, K, E, kind):
    g = np.random.default_rng(T * 131 + K * 7 + E)
    idx = g.integers(0, E, (T, K)).astype(np.int32)
    if kind == "drop":
        bad = np.array([-1, E, E + 5, -2**31, 2**31 - 1], np.int64).astype(np.int32)
        idx = np.where(g.random((T, K)) < 0.3, bad[g.integers(0, 5, (T, K))], idx)
    elif kind == "one":
        idx[:] = E - 1
    elif kind == "none":
        idx[:] = -1
    elif kind == "twice":
        idx[:, K // 2:] = idx[:, :1]
    got = run_sort(k3g, torch.from_numpy(idx).cuda(), E)
    torch.cuda.synchronize()
    for a, b in zip(got, order(idx, E)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_sort_of_no_tokens_and_the_layer_bucket(k3g):
    """No tokens: offsets are zeros. And the pairs' order is the one that the layer's own bucket writes."""
    off = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    k3g.k3g_moe_sort(off, none, none.view(0, 4), none.view(0, 4), ws)
    assert off.tolist() == [0] * 9
    T, K, E, n = 40, 6, 24, 128
    idx = torch.randint(-1, E, (T, K), dtype=torch.int32, device="cuda")
    off, stride = k3g.bank_layout(n, n)
    bank = k3g.bank_struct(torch.zeros(E * stride, dtype=torch.uint8, device="cuda"), E, n, n)
    sh = k3g.shape(n_tokens=T, top_k=K, n_experts=E, latent=n, inter=n, mode=k3g.EXACT)
    ws = k3g.workspace(k3g.OP_MOE_LAYER, sh)
    x = torch.zeros(T, n, device="cuda")
    k3g.k3g_moe_layer_stage(k3g.STAGE_BUCKET, x.clone(), x, idx, torch.ones(T, K, device="cuda"), bank, k3g.EXACT, ws)
    L = k3g.workspace_layout(k3g.OP_MOE_LAYER, sh)
    at = lambda name, m: ws[L[name]:L[name] + 4 * m].view(torch.int32)  # noqa: E731
    o, p, i = run_sort(k3g, idx, E)
    kept = int(o[E])
    assert torch.equal(o, at("offsets", E + 1)) and torch.equal(i.view(-1), at("inv", T * K))
    assert torch.equal(p[:kept], at("perm", T * K)[:kept])


# ---- rows ------------------------------------------------------------------------------

def half_step(t):
    """A rounding is off by at most this much of the value, and by this much near zero."""
    f = torch.finfo(t)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def close(got, want, scale, steps):
    """got (its own type) is want (64 bits) rounded once, from fp32 sums of `steps` roundings relative to `scale`."""
    rel, least = half_step(got.dtype)
    err = (got.double() - want).abs()
    tol = rel * want.abs() + (steps * 2.0 ** -24 * (1 + rel)) * scale + least
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} entries off, worst {float((err / tol).nan_to_num(9e9).max()):.2f} of the tolerance"


def slab(g, rows, n, t, pad):
    """Rows `pad` columns apart in a buffer, behind an odd number of entries."""
    b = torch.randn(rows * (n + pad) + 3, generator=g, device="cuda", dtype=torch.float32).to(t)
    return b[3:].view(rows, n + pad)[:, :n] if pad else b[3:].view(rows, n)


def case(T, K, R, n, row_t, tok_t, pad, seed, drop=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    names = torch.randperm(max(R, T * K), generator=g, device="cuda")[:T * K]  # places beyond R: pairs without a row
    names = torch.where(torch.rand(T * K, generator=g, device="cuda") < drop, -1, names)
    inv = torch.where(names >= R, R + names % 7, names).to(torch.int32).view(T, K)
    w = torch.randn(T, K, generator=g, device="cuda")
    return inv, w, slab(g, T, n, tok_t, pad), slab(g, R, n, row_t, pad)


def maps(inv, R):
    t, k = torch.nonzero((inv >= 0) & (inv < R), as_tuple=True)
    return t, k, inv[t, k].long()


SHAPES = [(1, 1, 1, 1, 0), (1, 16, 16, 7168, 0), (5, 3, 9, 63, 5), (33, 4, 140, 512, 1), (7, 64, 448, 520, 0),
          (64, 16, 1024, 3584, 8), (61, 9, 300, 3585, 3), (3, 5, 15, 65536, 0), (9, 2, 0, 40, 0), (2, 7, 14, 8200, 2),
          (1500, 6, 9000, 96, 0), (4200, 3, 13000, 96, 1), (701, 5, 3000, 3003, 3)]
PAIRS = [(a, b) for a in TYPES for b in TYPES]


@pytest.mark.parametrize("row_t,tok_t", PAIRS, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,K,R,n,pad", SHAPES)
def test_rows_and_gradients(k3g, T, K, R, n, pad, row_t, tok_t):
    inv, w, tok, rows = case(T, K, R, n, row_t, tok_t, pad, T + K + n)
    t, k, p = maps(inv, R)
    T64, R64, W = tok.double(), rows.double(), w.double()
    for wts in (w, None):
        wv = W[t, k][:, None] if wts is not None else torch.ones(len(t), 1, dtype=torch.float64, device="cuda")
        # gather, and combine's dys: the same values, rows that no pair names left
        mark = torch.randn(R, n + pad, device="cuda").to(row_t)
        want = mark[:, :n].double()
        want[p] = T64[t] * wv
        named = torch.zeros(R, 1, dtype=torch.bool, device="cuda")
        named[p] = True
        out = mark.clone()
        k3g.k3g_moe_gather(out[:, :n], tok, inv, wts=wts)
        assert torch.equal(out[~named[:, 0]], mark[~named[:, 0]]) and torch.equal(out[:, n:], mark[:, n:])
        close(out[:, :n], want, want.abs(), 1)
        back = mark.clone()
        dw = torch.full((T, K), float("nan"), device="cuda")
        k3g.k3g_moe_combine_backward(back[:, :n], tok, inv, wts=wts, ys=rows, dwts=dw)
        assert torch.equal(back, out)
        # the weights' gradient: 8 products in a thread, 6 sums in a wavefront, up to 8 turns and 16 wavefronts
        want_dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        mag = want_dw.clone()
        want_dw[t, k] = (T64[t] * R64[p]).sum(1)
        mag[t, k] = (T64[t] * R64[p]).abs().sum(1)
        close(dw, want_dw, mag, 38)
        dx = torch.full((T, n + pad), 9.0, device="cuda").to(tok_t)
        dw2 = torch.full_like(dw, float("nan"))
        k3g.k3g_moe_gather_backward(dx[:, :n], rows, inv, wts=wts, x=tok, dwts=dw2)
        assert torch.equal(dw, dw2) and bool((dx[:, n:] == 9).all())
        # combine: K products and sums
        want_y = torch.zeros(T, n, dtype=torch.float64, device="cuda").index_add_(0, t, R64[p] * wv)
        mag = torch.zeros_like(want_y).index_add_(0, t, (R64[p] * wv).abs())
        close(dx[:, :n], want_y, mag, K)
        y = torch.full((T, n), 9.0, device="cuda").to(tok_t)
        k3g.k3g_moe_combine(y, rows, inv, wts=wts)
        assert torch.equal(y, dx[:, :n])
        # one result alone
        dx1 = torch.full_like(y, 3)
        k3g.k3g_moe_gather_backward(dx1, rows, inv, wts=wts)
        dw1 = torch.full_like(dw, 3)
        k3g.k3g_moe_gather_backward(None, rows, inv, wts=wts, x=tok, dwts=dw1)
        assert torch.equal(dx1, y) and torch.equal(dw1, dw)
        dw1.fill_(3)
        k3g.k3g_moe_combine_backward(None, tok, inv, wts=wts, ys=rows, dwts=dw1)
        back1 = mark.clone()
        k3g.k3g_moe_combine_backward(back1[:, :n], tok, inv, wts=wts)
        assert torch.equal(dw1, dw) and torch.equal(back1, out)
        # over the rows themselves
        over = rows.clone()
        dw1.fill_(3)
        k3g.k3g_moe_combine_backward(over, tok, inv, wts=wts, ys=over, dwts=dw1)
        assert torch.equal(dw1, dw) and torch.equal(over[named[:, 0]], out[:, :n][named[:, 0]])
        assert torch.equal(over[~named[:, 0]], rows[~named[:, 0]])


def test_left_out_pairs_bring_nothing_of_their_rows_or_weights(k3g):
    """NaN and infinities in rows that no pair names, and in the weights of dropped pairs, reach nothing."""
    T, K, n = 6, 4, 200
    inv = torch.arange(T * K, dtype=torch.int32, device="cuda").view(T, K).clone()
    inv[1, 2], inv[3, :], inv[4, 0] = -1, -1, T * K + 3
    rows, tok = torch.randn(T * K, n, device="cuda"), torch.randn(T, n, device="cuda")
    w = torch.rand(T, K, device="cuda")
    gone = (inv < 0) | (inv >= T * K)
    rows[gone.view(-1)] = float("nan")
    w[gone] = float("inf")
    y, dw = torch.empty(T, n, device="cuda"), torch.empty(T, K, device="cuda")
    k3g.k3g_moe_gather_backward(y, rows, inv, wts=w, x=tok, dwts=dw)
    assert torch.isfinite(y).all() and bool((y[3] == 0).all()) and torch.isfinite(dw).all() and bool((dw[gone] == 0).all())
    # and what is named carries them
    rows[5, 7], w[2, 0] = float("inf"), float("nan")
    k3g.k3g_moe_combine(y, rows, inv, wts=w)
    assert torch.isinf(y[1, 7]) and torch.isnan(y[2]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[4:]).all()


def test_gradients_by_differences(k3g):
    """L = <c, combine(ys, w)> and L = <c, gather(x, w)>: the gradients against central differences of the calls
    themselves. L is linear in each variable and all values are small whole numbers: nothing is rounded, they are equal."""
    T, K, n = 5, 4, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    inv = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32).view(T, K)
    rnd = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float()  # noqa: E731  (exact in every sum)
    w, ys, x, c, cs = rnd(T, K), rnd(T * K, n), rnd(T, n), rnd(T, n), rnd(T * K, n)

    def combine(w, ys):
        return float((k3g.k3g_moe_combine(torch.empty(T, n, device="cuda"), ys, inv, wts=w).double() * c).sum())

    def gather(w, x):
        return float((k3g.k3g_moe_gather(torch.zeros(T * K, n, device="cuda"), x, inv, wts=w).double() * cs).sum())
    dys, dw = torch.empty(T * K, n, device="cuda"), torch.empty(T, K, device="cuda")
    k3g.k3g_moe_combine_backward(dys, c, inv, wts=w, ys=ys, dwts=dw)
    dx, dw2 = torch.empty(T, n, device="cuda"), torch.empty(T, K, device="cuda")
    k3g.k3g_moe_gather_backward(dx, cs, inv, wts=w, x=x, dwts=dw2)
    for f, a, b, da, db in ((combine, w, ys, dw, dys), (gather, w, x, dw2, dx)):
        for v, d in ((a, da), (b, db)):
            for at in torch.randint(0, v.numel(), (12,), generator=g, device="cuda").tolist():
                old = float(v.view(-1)[at])
                v.view(-1)[at] = old + 1
                hi = f(a, b)
                v.view(-1)[at] = old - 1
                lo = f(a, b)
                v.view(-1)[at] = old
                assert (hi - lo) / 2 == float(d.view(-1)[at])  # whole numbers: exact


def test_rows_past_32_bits(k3g):
    """Sorted rows that lie past 2^32 bytes and 2^31 entries."""
    R, n = 70001, 32768
    rows = torch.zeros(R, n, dtype=torch.bfloat16, device="cuda")
    inv = torch.tensor([[R - 1, 0], [65537, R - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, n, device="cuda").bfloat16()
    k3g.k3g_moe_gather(rows, x, inv)
    assert torch.equal(rows[inv.long().view(-1)], x.repeat_interleave(2, 0))
    assert int((rows[[1, 65536, R - 3]] != 0).sum()) == 0
    y = torch.empty(2, n, device="cuda")
    k3g.k3g_moe_combine(y, rows, inv)
    assert torch.equal(y, 2 * x.float())


def test_captured_on_another_stream_and_replayed(k3g):
    """Sort, gather, combine and both gradients in a graph, replayed with other inputs between eager work."""
    T, K, E, n = 200, 8, 64, 264
    idx = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    x, w, dy = torch.zeros(T, n, device="cuda"), torch.zeros(T, K, device="cuda"), torch.zeros(T, n, device="cuda")
    ids = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731

    def buffers():
        return dict(off=ids(E + 1), perm=ids(T * K), inv=ids(T, K), rows=torch.empty(T * K, n, device="cuda").bfloat16(),
                    y=torch.empty(T, n, device="cuda"), dys=torch.empty(T * K, n, device="cuda").bfloat16(),
                    dw=torch.empty(T, K, device="cuda"), dx=torch.empty(T, n, device="cuda"),
                    ws=k3g.workspace(k3g.OP_MOE_SORT, k3g.shape(n_tokens=T, top_k=K, n_experts=E)))

    def step(b):
        k3g.k3g_moe_sort(b["off"], b["perm"], b["inv"], idx, b["ws"])
        k3g.k3g_moe_gather(b["rows"], x, b["inv"])
        k3g.k3g_moe_combine(b["y"], b["rows"], b["inv"], wts=w)
        k3g.k3g_moe_combine_backward(b["dys"], dy, b["inv"], wts=w, ys=b["rows"], dwts=b["dw"])
        k3g.k3g_moe_gather_backward(b["dx"], b["dys"], b["inv"])
    cap, eager = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(cap)
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        idx.copy_(torch.randint(-1 if i % 2 else 0, E, (T, K), generator=gen, device="cuda"))
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        for b in (cap, eager):
            b["rows"].zero_(), b["dys"].zero_()
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for name in cap:
            if name != "ws":
                assert torch.equal(cap[name], eager[name]), (i, name)


def test_two_streams(k3g):
    """Two calls at once, each with its own workspace and outputs."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    idx = [torch.randint(0, 896, (8191, 16), dtype=torch.int32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, i in zip(streams, idx):
        with torch.cuda.stream(s):
            got.append(run_sort(k3g, i, 896))
    torch.cuda.synchronize()
    for g, i in zip(got, idx):
        for a, b in zip(g, order(i.cpu().numpy(), 896)):
            assert np.array_equal(a.cpu().numpy(), b)
