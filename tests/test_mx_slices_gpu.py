"""Norm operands that are column slices of one buffer: their rows lie between each other's and share no entry (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    k.lib()
    return k


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("T,n", [(1, 32), (2, 96), (70, 256), (1100, 64)])
def test_norm_between_column_slices(k3g, T, n, ty):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, r = (torch.randn(T, n, device="cuda", generator=g).to(TYPES[ty]) for _ in range(2))
    gamma = torch.rand(n, device="cuda", generator=g) + 0.5
    alone = [torch.empty_like(x) for _ in range(2)]
    k3g.k3g_add_rmsnorm(x, gamma, 1e-5, r=r, sum=alone[0], y=alone[1])
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 3, 0, 2)):
        buf = torch.full((T, 4 * n + 1), 7.0, device="cuda", dtype=TYPES[ty])
        xs, rs, sm, y = (buf[:, i * n:(i + 1) * n] for i in order)
        xs.copy_(x), rs.copy_(r)
        print(f"column slices T={T} n={n} {ty} {order}", flush=True)
        k3g.k3g_add_rmsnorm(xs, gamma, 1e-5, r=rs, sum=sm, y=y)
        assert torch.equal(sm, alone[0]) and torch.equal(y, alone[1])
        assert torch.equal(xs, x) and torch.equal(rs, r) and bool((buf[:, 4 * n] == 7.0).all())
