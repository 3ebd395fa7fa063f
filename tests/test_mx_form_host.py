"""The kernel that a microscaled product runs on, as the host chooses it (CPU)."""
import pytest

EINVAL = -1


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def test_refusals(k3g):
    f = k3g.lib().k3g_probe_mx_form
    for bad in ((2, 0, 1, 1, 0), (-1, 0, 1, 1, 0), (0, 3, 1, 1, 1), (0, -1, 1, 1, 1), (0, 0, 0, 1, 0), (0, 0, 1, 0, 0),
                (0, 1, 1, 1, 0), (0, 2, 1, 1, 2049), (0, 0, (1 << 30) + 1, 1, 0), (0, 0, 1, (1 << 30) + 1, 0)):
        assert f(*bad) == EINVAL, bad
    with pytest.raises(k3g.K3GError):
        k3g.k3g_probe_mx_form(0, 0, 1)


def test_forms(k3g):
    form = k3g.k3g_probe_mx_form
    assert form(k3g.MXFP8, 1, 3584) == (16, 16) and form(k3g.MXFP4, 61, 7168) == (32, 64)
    assert form(k3g.MXFP4, 4096, 6144) == (256, 256) and form(k3g.MXFP8, 4096, 6144) == (256, 128)
    assert form(k3g.MXFP8, 1024, 3584, 896) == (128, 32) and form(k3g.MXFP4, 65536, 3584, 896, glu=True) == (256, 128)


@pytest.mark.parametrize("fmt", [0, 1])
def test_few_tokens_take_no_wide_tile(k3g, fmt):
    """However many outputs: a tile of the tokens' width, or the streaming kernel."""
    for rows in (3584, 16384, 20480, 40960, 65536, 131072, 1 << 20):
        for T in (1, 2, 8, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128):
            outputs, tokens = k3g.k3g_probe_mx_form(fmt, T, rows)
            assert tokens <= 32 or tokens < 2 * T, (rows, T, outputs, tokens)
    assert k3g.k3g_probe_mx_form(fmt, 1, 131072) == (128, 32)
    assert k3g.k3g_probe_mx_form(fmt, 129, 131072)[1] == (256 if fmt == 0 else 128)


@pytest.mark.parametrize("fmt", [0, 1])
def test_one_token_takes_sixteen_outputs_while_each_has_a_cu(k3g, fmt):
    for T in (1, 16):
        assert k3g.k3g_probe_mx_form(fmt, T, 4096) == (16, 16)
        for rows in (4097, 7168, 16384, 20000):
            assert k3g.k3g_probe_mx_form(fmt, T, rows) == (32, 16)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
def test_grouped_borders(k3g, fmt, glu):
    for E in (1, 8, 896):
        for per, tile in ((1, (128, 32)), (2, (128, 32)), (3, (128, 64)), (16, (128, 64)), (17, (256, 128))):
            assert k3g.k3g_probe_mx_form(fmt, E * per, 3584, E, glu) == tile
