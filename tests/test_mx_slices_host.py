"""Norm operands in one buffer that share entries are refused, also where their rows lie between each other's (CPU;
nothing is launched)."""
import pytest

EINVAL = -1
M = 1 << 20  # made-up addresses: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def k3g():
    import mxfp4_moe_expert_amd as k
    return k


def norm(k3g, y, x, ys=256, xs=256, n=4, w=64, sm=None):
    return k3g.lib().k3g_add_rmsnorm(y, ys, sm, ys, None, x, xs, None, 0, 0, 100 * M, 1e-5, n, w, None)


def test_slices_that_share_entries(k3g):
    at = M + 4 * 64  # columns 64 .. 127 of rows of 256 floats
    for y in (at, at + 4 * 63, at - 4 * 63, at + 4 * 256 - 4, at + 4 * (256 + 60), at - 4 * (256 - 60), at + 4 * (3 * 256 + 63)):
        if y != at:
            assert norm(k3g, y, at) == EINVAL, y
    assert norm(k3g, at + 4 * 64, at, ys=260) == EINVAL  # rows of unlike distances: the gaps count
    assert norm(k3g, 50 * M, at, sm=50 * M + 4 * 32) == EINVAL  # the two outputs


def test_slices_that_share_none_are_not_refused(k3g):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would be launched")
    at = M + 4 * 64
    for y in (at + 4 * 64, at - 4 * 64, at + 4 * 128, at + 4 * 192, at + 4 * (256 - 64), at + 4 * (3 * 256 + 64)):
        assert norm(k3g, y, at) != EINVAL, y
