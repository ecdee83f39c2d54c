"""A workspace of the delta rule's or the norms' calls that is large enough for
one batch and length is so for every smaller one (CPU)."""
import pytest

from test_regression_amd import mesa

F32, BF16 = mesa.MESA_DTYPE_F32, mesa.MESA_DTYPE_BF16


def never_less(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (16, 16), (128, 16), (16, 256), (32, 128)])
def test_delta_forward_workspace_grows_with_length_and_heads(dk, dv, dtype):
    f = mesa.mesa_delta_workspace_bytes
    for H in (1, 2, 3, 5, 8, 16, 24, 33, 64):
        assert never_less([f(1, H, 64 * n - 3, dk, dv, dtype) for n in range(1, 300)]), H
    for n in (1, 12, 13, 16, 17, 31, 33, 40, 64, 100, 256, 1000):
        assert never_less([f(1, H, 64 * n, dk, dv, dtype) for H in range(1, 140)]), n
    assert f(4, 4, 4096, dk, dv, dtype) == f(1, 16, 4096, dk, dv, dtype)


@pytest.mark.parametrize("H", [1, 3, 16, 40, 1500])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
def test_gate_norm_backward_workspace_grows_with_rows_and_heads(d, H):
    g = mesa.lib().mesa_gate_norm_backward_workspace_bytes
    assert never_less([g(1, H, T, d) for T in range(1, 3000, 7)])
    assert never_less([g(2, h, 700, d) for h in range(1, 1100)])


def test_residual_norm_backward_workspace_grows_with_rows_and_width():
    r = mesa.lib().mesa_residual_norm_backward_workspace_bytes
    for D in (1, 100, 2048, 2049, 4096, 16384):
        assert never_less([r(R, D) for R in range(1, 4000, 3)])
    for R in (1, 5, 1000, 1500, 100000):
        assert never_less([r(R, D) for D in range(1, 16384, 5)])


def test_workspaces_hold_what_the_calls_take():
    """A call with the size of the largest of a run of shapes is not refused for
    its workspace (it is refused for an alias, the check after that one)."""
    from tests.test_abi_delta import call
    for H, top in ((2, 4160), (16, 2112), (16, 4096), (32, 4096)):
        size = mesa.mesa_delta_workspace_bytes(1, H, top, 128, 128, BF16)
        for T in range(64, top + 1, 64):
            _, msg = call("mesa_delta_forward", dtype=BF16, Hk=H, H=H, T=T, dk=128, dv=128, workspace_bytes=size)
            assert "alias" in msg, (H, T, msg)
    r = mesa.lib().mesa_gate_norm_backward_workspace_bytes
    for T in range(1, 4000, 13):
        _, msg = call("mesa_gate_norm_backward", T=T, workspace_bytes=r(1, 2, 4000, 64))
        assert "alias" in msg, (T, msg)
