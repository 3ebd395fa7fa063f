"""The residual + RMS norm to the last bit, on the GPU against 64 bits.

Tolerances. The mean is summed in 64 bits and each n kept to 2^-46 of itself, so an output of 8 or 11 bits, or a code,
is the rounding of the 64-bit n (a tie closer than 2^-46 has a chance under 1e-3 in the largest test here); an fp32
output is within half a step and 2^-20 of one.
"""
import pytest

from tests import mx_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 2.0 ** -17


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


def norm64(x, r, gamma, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * gamma.double()


def check_rounded(y, ref, what):
    want = mx_dev.rounded(ref, y.dtype)
    if y.dtype == torch.float32:
        ulp = mx_dev.pow2((torch.frexp(ref)[1] - 24).clamp(min=-149))
        bad = ~((y.double() - ref).abs() <= 0.5 * (1 + 2.0 ** -20) * ulp)
    else:
        bad = ~(y.double() == want)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off; first {bad.nonzero()[:3].tolist()}: "
                                 f"{y[bad][:3].tolist()} for {want[bad][:3].tolist()}")


@pytest.mark.parametrize("ty", TYPES)
def test_norm_is_rounded_once(k3g, ty):
    """Every output of 29 million is the rounding of the 64-bit norm, and every code that of its group."""
    T, n = 4096, 7168
    g = torch.Generator(device="cuda").manual_seed(71)
    x = torch.randn(T, n, device="cuda", generator=g).to(TYPES[ty])
    r = torch.randn(T, n, device="cuda", generator=g).to(TYPES[ty])
    gamma = torch.rand(n, device="cuda", generator=g) + 0.5
    for fmt in (0, 1):
        y, q = torch.empty_like(x), k3g.mx_empty(T, n, fmt)
        print(f"norm rounded once {ty} fmt={fmt}", flush=True)
        k3g.k3g_add_rmsnorm(x, gamma, EPS, r=r, y=y, q=q)
        for t in range(0, T, 512):
            s = x[t:t + 512].float() + r[t:t + 512].float()
            ref = norm64(s, None, gamma, EPS)
            check_rounded(y[t:t + 512], ref, f"y from row {t}")
            got = mx_dev.values(q.codes[t:t + 512], q.scales[t:t + 512], fmt)
            bad = got != mx_dev.grid(ref, fmt)
            assert not bool(bad.any()), f"{int(bad.sum())} codes off from row {t}"
