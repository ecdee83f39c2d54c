"""The gradients of gates near and below the smallest normal float, whose
products with other decays leave float's range, against the float64 form."""
import numpy as np
import pytest

from tests.delta_helpers import delta_inputs, rel
from tests.test_gpu_delta import GRAD_F32, backward_errors, grad_tol, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("bf16", 64, 32), ("bf16", 128, 128), ("f32", 128, 64), ("f32", 16, 16)])
@pytest.mark.parametrize("lo", [0.8, 0.1])
def test_tiny_gates(dtype, dk, dv, lo):
    say("case delta tiny gates", (dtype, dk, dv, lo))
    t, f = delta_inputs(501, 1, 2, 4, 200, dk, dv, dtype, lo=lo)
    at = [0, 3, 40, 64, 70, 71, 127, 128, 190, 199]
    for i, size in zip(at, [1e-40, 2.0 ** -126, 1e-44, 2.0 ** -110, 1e-40, 1e-38, 2.0 ** -100, 2.0 ** -63, 2.0 ** -65, 1e-30]):
        t["gamma"][:, :, i] = size
    f["gamma"] = t["gamma"].double().numpy()
    assert (f["gamma"] > 0).all()
    errs, got, ref = backward_errors(t, f, dtype, 501)
    e = rel(got["grad_gamma"][:, :, at], ref["grad_gamma"][:, :, at])
    say(f"  at them {e:.1e}  " + " ".join(f"{n[5:]}={x:.1e}" for n, x in errs.items()))
    assert e <= GRAD_F32
    for n, x in errs.items():
        if np.abs(ref[n]).max() < 2.0 ** -126:
            # the state's, past the first token's gate of 1e-40: decays below the
            # smallest normal float are taken as 0, off by less than that
            assert n == "grad_state" and np.abs(got[n]).max() < 2.0 ** -126
        else:
            assert x <= grad_tol(n, dtype), n


def test_a_gate_of_zero_beside_tiny_ones():
    """A reset is not differentiated; the gates around it are."""
    t, f = delta_inputs(511, 1, 2, 2, 130, 64, 64, "f32")
    say("case delta reset beside tiny gates")
    t["gamma"][:, :, 20], t["gamma"][:, :, 30], t["gamma"][:, :, 31] = 1e-40, 0.0, 1e-39
    f["gamma"] = t["gamma"].double().numpy()
    errs, got, ref = backward_errors(t, f, "f32", 511)
    assert (got["grad_gamma"][:, :, 30] == 0).all()
    ref["grad_gamma"][:, :, 30] = 0
    for i in ([20, 31], slice(0, 130)):
        assert rel(got["grad_gamma"][:, :, i], ref["grad_gamma"][:, :, i]) <= GRAD_F32
    assert all(x <= grad_tol(n, "f32") for n, x in errs.items() if n != "grad_gamma"), errs
