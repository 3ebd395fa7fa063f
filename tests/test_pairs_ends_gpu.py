"""Weights' gradients of dropped pairs next to rows of tokens that are not finite."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


# (tokens, pairs a token, columns): four pairs of a token and more in workgroups of their own, and a token's all in
# one; a ragged last four; one column and more than a wavefront's
@pytest.mark.parametrize("T,K,n", [(5, 1, 1), (12, 4, 200), (9, 7, 1030), (40, 64, 72), (4200, 5, 96)])
@pytest.mark.parametrize("t", TYPES, ids=lambda t: str(t)[6:])
def test_dropped_pairs_of_tokens_that_are_not_finite(k3g, T, K, n, t):
    """dwts of a pair without a row is 0, whatever its token's row holds and whichever pairs stand beside it; of the
    others what the same call gives where nothing is dropped."""
    g = torch.Generator(device="cuda").manual_seed(T * K + n)
    R = T * K
    whole = torch.randperm(R, generator=g, device="cuda").to(torch.int32).view(T, K)
    gone = torch.rand(T, K, generator=g, device="cuda") < 0.4
    gone[0], gone[1 % T, :K // 2] = False, True
    inv = torch.where(gone, torch.where(torch.rand(T, K, generator=g, device="cuda") < 0.5, -1, R + 3), whole).to(torch.int32)
    tok, rows = torch.randn(T, n, generator=g, device="cuda").to(t), torch.randn(R, n, generator=g, device="cuda")
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        tok[i::4, (7 * i) % n] = v
    w = torch.rand(T, K, generator=g, device="cuda")

    def dw(inv, call):
        d = torch.full((T, K), 5.0, device="cuda")
        call(inv, d)
        return d
    calls = [lambda i, d: k3g.k3g_moe_gather_backward(None, rows, i, wts=w, x=tok, dwts=d),
             lambda i, d: k3g.k3g_moe_gather_backward(torch.empty_like(tok), rows, i, wts=w, x=tok, dwts=d),
             lambda i, d: k3g.k3g_moe_combine_backward(None, tok, i, wts=w, ys=rows, dwts=d),
             lambda i, d: k3g.k3g_moe_combine_backward(torch.empty_like(rows), tok, i, wts=w, ys=rows, dwts=d)]
    for call in calls:
        want, got = dw(whole, call), dw(inv, call)
        assert bool((got[gone] == 0).all())
        assert torch.equal(torch.nan_to_num(got[~gone], 3e38, 2e38, 1e38), torch.nan_to_num(want[~gone], 3e38, 2e38, 1e38))
        assert not torch.isfinite(want[0]).any() and bool(torch.isfinite(want[3::4]).all())
