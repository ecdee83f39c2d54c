"""The gate of the gate norm far from zero, element by element.

silu(g) = g / (1 + e^-g).  An exponential within 2 2^-24 of its value, the sum,
the division (at most 2.5 2^-24) and three products leave 12 2^-24 of the
result; the row's norm, exact here up to its root and product, 4 more.  An
exponential taken as 2^(g log2 e) with a rounded exponent is off by |g| 2^-24.
"""
import numpy as np
import pytest

from tests.delta_helpers import store

pytestmark = pytest.mark.gpu
BOUND = 16 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def test_gates_far_from_zero():
    import torch
    from test_regression_amd import mesa
    print("case gate accuracy", flush=True)
    rng = np.random.default_rng(9)
    x, xf = store(np.where(rng.random((1, 4, 64, 32)) < 0.5, -1.0, 1.0), "f32")   # rows of mean square 1
    g, gf = store(rng.uniform(-80, 20, (1, 64, 4, 32)), "f32")
    w, _ = store(np.ones((4, 32)), "f32")
    dy, dyf = store(np.ones((1, 64, 4, 32)), "f32")
    y = mesa.mesa_gate_norm(x.cuda(), g.cuda(), w.cuda(), 1e-20)
    r = mesa.mesa_gate_norm_backward(x.cuda(), g.cuda(), w.cuda(), dy.cuda(), 1e-20)
    torch.cuda.synchronize()
    u, s = xf.transpose(0, 2, 1, 3), 1.0 / (1.0 + np.exp(-gf))
    for got, ref, terms in ((y, u * gf * s, np.abs(gf * s)),
                            (r["grad_gate"], u * s * (1.0 + gf * (1.0 - s)), s * (1.0 + np.abs(gf * (1.0 - s))))):
        e = np.abs(got.double().cpu().numpy() - ref) / terms
        print(f"  largest {e.max():.1e}", flush=True)
        assert e.max() <= BOUND
