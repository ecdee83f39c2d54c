"""Which batches the delta rule's entry points refuse as too large for a launch of
fewer than 2^32 threads (CPU): those that are, and no smaller ones."""
import pytest

from test_regression_amd import mesa
from tests.test_abi_delta import BF16, call

SIZES = dict(dtype=BF16, Hk=16, H=16, dk=128, dv=128)


@pytest.mark.parametrize("name,kw", [
    ("mesa_delta_step", dict(N=32768)), ("mesa_delta_step", dict(N=1 << 17)),
    ("mesa_delta_step", dict(N=200000, dk=16, dv=16)),
    ("mesa_delta_forward", dict(B=40000, T=1)), ("mesa_delta_forward", dict(B=60000, T=64)),
    ("mesa_delta_backward", dict(B=40000, T=1)),
])
def test_large_batches_that_fit_a_launch(name, kw):
    """Refused for an alias only, the check after that of the grid."""
    _, msg = call(name, **{**SIZES, **kw, **({} if "step" in name else dict(workspace_bytes=1 << 46)),
                           **(dict(out=0x10000) if "step" in name else {})})
    assert "alias" in msg, msg


@pytest.mark.parametrize("name,kw", [
    ("mesa_delta_step", dict(N=1 << 18)), ("mesa_delta_forward", dict(B=90000, T=1)),
    ("mesa_delta_forward", dict(B=16384, T=4096)), ("mesa_delta_backward", dict(B=90000, T=1)),
])
def test_batches_that_do_not(name, kw):
    _, msg = call(name, **{**SIZES, **kw})
    assert "grid too large" in msg, msg
