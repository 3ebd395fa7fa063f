"""The refusals of the calls on routed pairs, before any launch (CPU)."""
import pytest

EINVAL, EALIGN, NOSPACE, UNSUPPORTED = -1, -2, -3, -5
M = 1 << 20  # made-up addresses a MiB apart: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def test_sort_refusals(k3g):
    L = k3g.lib()

    def sort(off=M, perm=2 * M, inv=3 * M, idx=4 * M, T=8, K=4, E=16, ws=5 * M, n=1 << 20):
        return L.k3g_moe_sort(off, perm, inv, idx, T, K, E, ws, n, None)
    for bad in ({"T": -1}, {"K": 0}, {"E": 0}, {"off": None}, {"perm": None}, {"inv": None}, {"idx": None}, {"ws": None},
                {"perm": M}, {"inv": 2 * M + 124}, {"idx": 3 * M}, {"idx": M + 64}, {"ws": 4 * M}, {"inv": M + 64}):
        assert sort(**bad) == EINVAL, bad
    for bad in ({"off": M + 2}, {"perm": 2 * M + 1}, {"inv": 3 * M + 2}, {"idx": 4 * M + 2}, {"ws": 5 * M + 128}):
        assert sort(**bad) == EALIGN, bad
    assert sort(E=2049) == UNSUPPORTED
    assert sort(T=1 << 26, K=17) == UNSUPPORTED
    assert sort(n=255) == NOSPACE
    need = k3g.workspace_bytes(k3g.OP_MOE_SORT, k3g.shape(n_tokens=4096, top_k=16, n_experts=896))
    assert need > 16 * 896 * 4
    assert sort(off=16 * M, perm=32 * M, inv=64 * M, idx=128 * M, T=4096, K=16, E=896, n=need - 1) == NOSPACE


def test_sort_workspace(k3g):
    b = lambda **kw: k3g.workspace_bytes(k3g.OP_MOE_SORT, k3g.shape(**kw))  # noqa: E731
    assert b(n_tokens=0, top_k=1, n_experts=1) > 0
    assert b(n_tokens=1 << 24, top_k=64, n_experts=2048) == 256 + 256 * 2048 * 4  # chunks stop growing in number
    for bad in ({"n_tokens": -1, "top_k": 1, "n_experts": 1}, {"n_tokens": 1, "top_k": 0, "n_experts": 1},
                {"n_tokens": 1, "top_k": 1, "n_experts": 0}, {"n_tokens": 1, "top_k": 1, "n_experts": 2049},
                {"n_tokens": 1 << 26, "top_k": 17, "n_experts": 8}):
        assert b(**bad) == 0, bad


def calls(L):
    """The four calls by one set of names: rows (sorted side), tok (token side), their strides and types."""
    def gather(tok=M, rows=2 * M, w=3 * M, inv=4 * M, tt=0, rt=0, tl=64, rl=64, T=4, K=2, R=8, n=64):
        return L.k3g_moe_gather(rows, rt, rl, tok, tt, tl, w, inv, T, K, R, n, None)

    def combine(tok=M, rows=2 * M, w=3 * M, inv=4 * M, tt=0, rt=0, tl=64, rl=64, T=4, K=2, R=8, n=64):
        return L.k3g_moe_combine(tok, tt, tl, rows, rt, rl, w, inv, T, K, R, n, None)

    def gather_backward(tok=M, rows=2 * M, w=3 * M, inv=4 * M, tt=0, rt=0, tl=64, rl=64, T=4, K=2, R=8, n=64, x=5 * M,
                        xl=64, dw=6 * M):
        return L.k3g_moe_gather_backward(tok, dw, rows, rt, rl, x, tt, xl, tl, w, inv, T, K, R, n, None)

    def combine_backward(tok=M, rows=2 * M, w=3 * M, inv=4 * M, tt=0, rt=0, tl=64, rl=64, T=4, K=2, R=8, n=64, ys=5 * M,
                         yl=64, dw=6 * M):
        return L.k3g_moe_combine_backward(rows, dw, tok, tt, tl, ys, rt, yl, rl, w, inv, T, K, R, n, None)
    return gather, combine, gather_backward, combine_backward


@pytest.mark.parametrize("which", range(4))
def test_row_refusals(k3g, which):
    call = calls(k3g.lib())[which]
    out = "rows" if which in (0, 3) else "tok"
    for bad in ({"T": -1}, {"K": 0}, {"R": -1}, {"n": 0}, {"tt": 3}, {"rt": -1}, {"tl": 63}, {"rl": 63}, {"inv": None},
                {"tok": 2 * M + 4 * 64}, {"rows": M + 4 * 64}, {out: 4 * M}, {out: 3 * M}, {out: 4 * M + 28}):
        assert call(**bad) == EINVAL, bad
    for bad in ({"tok": M + 2}, {"rows": 2 * M + 2}, {"inv": 4 * M + 2}, {"w": 3 * M + 2}, {"tok": M + 1, "tt": 1, "rt": 1}):
        assert call(**bad) == EALIGN, bad
    for bad in ({"K": 65}, {"n": 65537, "tl": M, "rl": M}, {"T": 1 << 25, "K": 64}, {"R": (1 << 30) + 1}):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, inv=None, w=None, tok=None, **({"x": None, "dw": None} if which == 2 else
                                                    {"dw": None} if which == 3 else {})) == 0
    if which < 2:
        assert call(tok=None) == EINVAL and call(rows=None) == EINVAL


def test_gradient_refusals(k3g):
    _, _, gb, cb = calls(k3g.lib())
    for bad in ({"tok": None, "dw": None}, {"x": None}, {"dw": M}, {"dw": 2 * M}, {"dw": 3 * M}, {"dw": 4 * M},
                {"dw": 5 * M}, {"x": M}, {"xl": 63}):
        assert gb(**bad) == EINVAL, bad
    for bad in ({"rows": None, "dw": None}, {"ys": None}, {"dw": M}, {"dw": 2 * M}, {"dw": 3 * M}, {"dw": 5 * M},
                {"ys": 2 * M, "yl": 65}, {"ys": 2 * M + 256}, {"yl": 63}):
        assert cb(**bad) == EINVAL, bad
    assert gb(dw=6 * M + 2) == EALIGN and cb(ys=5 * M + 2) == EALIGN
    assert gb(x=5 * M + 2) == EALIGN and cb(dw=6 * M + 1) == EALIGN


def test_binding_refuses_host_tensors_and_wrong_shapes(k3g):
    import torch
    i = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError)):
        k3g.k3g_moe_sort(torch.zeros(5, dtype=torch.int32), i.view(-1), i, i, torch.zeros(256, dtype=torch.uint8))
    x = torch.zeros(2, 8)
    for f in (lambda: k3g.k3g_moe_gather(x, x, i), lambda: k3g.k3g_moe_combine(x, x, i),
              lambda: k3g.k3g_moe_gather_backward(None, x, i), lambda: k3g.k3g_moe_combine_backward(None, x, i),
              lambda: k3g.k3g_moe_gather_backward(x.double(), x, i)):
        with pytest.raises((ValueError, TypeError)):
            f()
