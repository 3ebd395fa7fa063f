"""The residual + RMS norm at the ends of its range and to the last bit, on the GPU against 64 bits.

Tolerances. The mean is summed in 64 bits and each n kept to 2^-46 of itself, so an output of 8 or 11 bits, or a code,
is the rounding of the 64-bit n (a tie closer than 2^-46 has a chance under 1e-3 in the largest test here); an fp32
output is within half a step and 2^-20 of one.
"""
import numpy as np
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


# ---- the norm at the ends of its range ----------------------------------------------------

# (fp32's and bf16's smallest rows are subnormal numbers; the squares of all but the third leave fp32's range)
MAGNITUDES = {"f32": [2.0 ** -146, 1e-38, 1.0, 1e-25, 1e-20, 1e18, 1e20, 5e37],
              "bf16": [2.0 ** -130, 1e-38, 1.0, 1e-25, 1e-20, 1e18, 1e20, 5e37],
              "f16": [2.0 ** -21, 1e-6, 1.0, 1e-3, 1e2, 1e4]}


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("n", [32, 2080, 7168, 65536])
def test_norm_of_tiny_and_huge_rows_without_eps(k3g, n, ty, fmt):
    mags = torch.tensor(MAGNITUDES[ty], device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = (torch.randn(len(mags), n, device="cuda", generator=g, dtype=torch.float64).clamp(-6, 6) * mags[:, None]).to(TYPES[ty])
    gamma = torch.rand(n, device="cuda", generator=g) + 0.5
    y, q = torch.empty_like(x), k3g.mx_empty(len(mags), n, fmt)
    print(f"norm of tiny and huge rows n={n} {ty} fmt={fmt}", flush=True)
    k3g.k3g_add_rmsnorm(x, gamma, 0.0, y=y, q=q)
    ref = norm64(x, None, gamma, 0.0)
    check_rounded(y, ref, "y")
    assert torch.equal(mx_dev.values(q.codes, q.scales, fmt), mx_dev.grid(ref, fmt)), "q"


def test_norm_whose_scale_times_gamma_passes_fp32(k3g):
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 256
    x = torch.randn(4, n, device="cuda", generator=g) * torch.tensor([[1e-20], [1e-30], [1e15], [1e30]], device="cuda")
    for scale in (1e30, 1e-30):
        gamma = (torch.rand(n, device="cuda", generator=g) + 0.5) * scale
        y, q = torch.empty_like(x), k3g.mx_empty(4, n, k3g.MXFP8)
        print(f"gamma {scale}", flush=True)
        k3g.k3g_add_rmsnorm(x, gamma, 0.0, y=y, q=q)
        ref = norm64(x, None, gamma, 0.0)
        check_rounded(y, ref, "y")
        assert torch.equal(mx_dev.values(q.codes, q.scales, 1), mx_dev.grid(ref, 1)), "q"


def test_norm_of_a_row_of_zeros(k3g):
    # n = 0 / sqrt(0 + eps) * gamma: zeros with an eps, no value without
    x = torch.zeros(3, 64, device="cuda")
    x[1] = 1e-30
    for eps in (2.0 ** -17, 1e-38, 0.0):
        y, q = torch.empty_like(x), k3g.mx_empty(3, 64, k3g.MXFP4)
        k3g.k3g_add_rmsnorm(x, torch.ones(64, device="cuda"), eps, y=y, q=q)
        ref = norm64(x, None, torch.ones(64, device="cuda"), eps if eps == 0 else float(np.float32(eps)))
        assert torch.equal(torch.isnan(y), torch.isnan(ref)) and bool(torch.isnan(ref)[0].all()) == (eps == 0)
        check_rounded(y[1:2], ref[1:2], "y")
        assert q.scales.tolist()[0] == ([255, 255] if eps == 0 else [1, 1])


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
