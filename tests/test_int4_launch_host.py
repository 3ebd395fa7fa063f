"""The launches of the int4 products (CPU): the vector kernel's limit of threads, items of their own, the questions' refusals."""
import pytest

EINVAL = -1


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def test_the_vector_kernel_stays_below_2_to_32_threads(k3g):
    """Rows of more than 8192 columns take a wavefront's worth of outputs a workgroup: rows * T alone does not bound the
    grid. One more output than fits is streamed, on a grid that does not grow."""
    import torch
    b16, form, launch = torch.bfloat16, k3g.k3g_probe_int4_form, k3g.k3g_probe_int4_launch
    # (tokens, columns, experts, glu, outputs of a workgroup: 16 turns of 4 or 2 for each wavefront along them)
    for T, n, E, glu, out in ((1, 16384, 0, False, 64), (1, 32768, 0, False, 64), (1, 8192, 0, False, 128),
                              (1, 16384, 3, True, 32), (4, 8224, 8, True, 32), (4, 4096, 8, False, 256)):
        waves = 8 if n != 8224 else 5
        groups = (2**32 - 1) // (64 * waves) // T  # workgroups a row of y
        rows = min(groups * out, 2**30 // T)
        assert form(b16, T, rows, n, E, glu) == (8, 1)
        got = launch(b16, T, rows, n, 32, E, glu)
        assert got == (-(-rows // out) * T, waves) and got[0] * waves * 64 < 2**32
        if rows < 2**30 // T:
            assert form(b16, T, rows + 1, n, E, glu)[0] != 8
            assert launch(b16, T, rows + 1, n, 32, E, glu)[0] <= 4096


def test_items_of_their_own(k3g):
    """A wavefront takes an item to itself from 4096 items on; fewer are split over the row's length."""
    import torch
    b16, launch = torch.bfloat16, k3g.k3g_probe_int4_launch
    assert launch(b16, 1024, 3584, 3072, 64, 896) == (4096, 1) == launch(b16, 1024, 3072, 3584, 64, 896, True)
    assert launch(b16, 16, 32 * 4095, 4096, 64) == (1024, 8) and launch(b16, 16, 32 * 4095 + 1, 4096, 64) == (4096, 1)
    assert launch(b16, 16, 3584, 512, 64) == (224, 1) and launch(b16, 16, 3584, 544, 32) == (224, 2)
    assert launch(b16, 4096, 6144, 7168, 128) == (512, 4) and launch(b16, 1024, 4096, 7168, 128) == (128, 4)


def test_refusals(k3g):
    L = k3g.lib()
    ok = [1, 1, 1, 64, 64, 128, 8, 64]
    assert L.k3g_probe_int4_launch(*ok) > 0
    for i, bad in ((0, 3), (2, 3), (3, 0), (4, 0), (5, 0), (5, 48), (6, 0), (6, 2049), (7, 16), (7, 96), (5, 96)):
        assert L.k3g_probe_int4_launch(*[bad if j == i else v for j, v in enumerate(ok)]) == EINVAL, (i, bad)
