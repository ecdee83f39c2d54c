"""More of what the state space layer's and the rotation's entry points refuse before they
touch the device (CPU, fake pointers as in tests/test_abi_ssm.py): strides whose
extent leaves the address space, and backward workspaces where the heads of shared b
and c are split over odd numbers of chunks."""
import pytest

from test_regression_amd import mesa
from tests.test_abi_ssm import BF16, ENTRIES, INVALID, P, call, refused


@pytest.mark.parametrize("name", ["mesa_qk_rotate", "mesa_qk_rotate_backward"])
def test_position_strides(name):
    refused(name, INVALID, "positions_stride must not be negative", pos_stride=-1)
    for stride, B in ((1 << 61, 3), (1 << 62, 2), ((1 << 63) - 1, 3), ((1 << 61) + 5, 9)):
        refused(name, INVALID, "strides of positions are too large", pos_stride=stride, B=B)
    # a batch that the positions reach into an output with
    out = "yq" if name == "mesa_qk_rotate" else "grad_q"
    gap = (ENTRIES[name][out] - ENTRIES[name]["positions"]) // 8
    refused(name, INVALID, f"{out} must not alias positions", pos_stride=gap, B=2)
    refused(name, INVALID, f"{out} must not alias positions", **{out: P(ENTRIES[name]["positions"])})


def test_backward_workspaces_of_split_heads():
    """A workspace for the largest of a run of batches and lengths serves all of them."""
    A = ENTRIES["mesa_ssm_backward"]["A"]
    size = mesa.mesa_ssm_backward_workspace_bytes
    for Hk, H in ((1, 32), (1, 7), (4, 24), (1, 300)):
        for T in (64, 130, 700, 4096):
            sizes = [size(B, Hk, H, T, 64, 16, BF16) for B in range(1, 90)]
            assert sizes == sorted(sizes)
            for B in range(1, 90, 4):
                _, msg = call("mesa_ssm_backward", B=B, Hk=Hk, H=H, T=T, dv=16, grad_A=A, workspace_bytes=sizes[-1], dtype=BF16)
                assert "alias" in msg, msg
                _, msg = call("mesa_ssm_backward", B=B, Hk=Hk, H=H, T=T, dv=16, grad_A=A, workspace_bytes=size(B, Hk, H, T, 64, 16, BF16),
                              dtype=BF16)
                assert "alias" in msg, msg
        for B in (1, 3, 5):
            sizes = [size(B, Hk, H, 64 * n, 64, 16, BF16) for n in range(1, 200)]
            assert sizes == sorted(sizes)
            for n in range(1, 200, 7):
                _, msg = call("mesa_ssm_backward", B=B, Hk=Hk, H=H, T=64 * n, dv=16, grad_A=A, workspace_bytes=sizes[-1], dtype=BF16)
                assert "alias" in msg, msg
