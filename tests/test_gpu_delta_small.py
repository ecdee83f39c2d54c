"""The gated delta rule on values and gradients far below unit size: from no
state at all, onto a state that a gate has forgotten, and in segments.  The
scale of a chunk's writes must follow the writes themselves wherever no larger
state is left beside them.  Bounds as in tests/test_gpu_delta.py; scalings are
powers of two, so the float64 form sees the same significands at every size.
"""
import numpy as np
import pytest

from tests.delta_helpers import F32, delta_inputs, delta_ref, rel, tol
from tests.test_gpu_delta import GRAD_F32, check_grads, dev, forward, grad_tol, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def scaled(t, f, name, by):
    t[name] = t[name] * by
    f[name] = t[name].double().numpy()


# every kernel of the passes: twelve waves in both types, four waves (float, dk = 128)
WIDTHS = [("f32", 64, 64), ("bf16", 64, 64), ("f32", 16, 32), ("bf16", 128, 128), ("f32", 128, 64)]


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 64, 200])
@pytest.mark.parametrize("e", [36, 44, 60])
def test_small_values_onto_no_state(dtype, dk, dv, T, e):
    say("case delta small values", (dtype, dk, dv, T, e))
    t, f = delta_inputs(201 + T + e, 1, 2, 2, T, dk, dv, dtype, start=False)
    scaled(t, f, "v", 2.0 ** -e)
    o, S = forward(t)
    ro, rS = delta_ref(f)
    assert rel(o, ro) <= tol(dtype) and rel(S, rS) <= F32, (rel(o, ro), rel(S, rS))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("start,e,lo", [(False, 60, 0.999), (True, 40, 0.99)])
def test_small_values_in_segments(dtype, start, e, lo):
    """Each segment's end is formed from nothing, also where the sequence has a
    start state of unit size."""
    say("case delta small values, segments", dtype, start)
    t, f = delta_inputs(211, 1, 1, 1, 4100, 64, 64, dtype, start=start, lo=lo)
    scaled(t, f, "v", 2.0 ** -e)
    o, S = forward(t)
    ro, rS = delta_ref(f)
    # a token forgets about 1/128 of the state by its write and 1/200 by its
    # gate: after 4000 tokens 2^-70 of the start is left
    assert rel(S, rS) <= F32, rel(S, rS)
    assert rel(o[:, :, 4000:], ro[:, :, 4000:]) <= tol(dtype), rel(o[:, :, 4000:], ro[:, :, 4000:])


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
def test_small_values_after_a_reset(dtype, dk, dv):
    """A sequence of unit size, then, from a gate of 0 on, one of 2^-40."""
    say("case delta small values after a reset", (dtype, dk, dv))
    t, f = delta_inputs(221, 1, 2, 2, 200, dk, dv, dtype)
    t["gamma"][:, :, 128] = 0.0
    t["v"][:, :, 128:] *= 2.0 ** -40
    f["gamma"], f["v"] = t["gamma"].double().numpy(), t["v"].double().numpy()
    o, S = forward(t)
    ro, rS = delta_ref(f)
    assert rel(S, rS) <= F32, rel(S, rS)
    assert rel(o[:, :, 128:], ro[:, :, 128:]) <= tol(dtype) and rel(o[:, :, :128], ro[:, :, :128]) <= tol(dtype)


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("bf16", 128, 128), ("f32", 128, 64)])
def test_small_values_beside_a_decaying_state(dtype, dk, dv):
    """A state (and a gradient of the final one) of unit size over features the
    keys and queries never touch, halved by every token; what is written
    meanwhile is 2^-60, and so are the outputs' gradients."""
    import torch
    from test_regression_amd import mesa
    say("case delta small values, decaying state", (dtype, dk, dv))
    t, f = delta_inputs(231, 1, 2, 2, 64, dk, dv, dtype)
    half = dk // 2
    for n in ("q", "k"):
        t[n][..., half:] = 0
    t["state"][..., :half] = 0
    t["gamma"].fill_(0.5)
    t["v"] *= 2.0 ** -60
    f.update({n: t[n].double().numpy() for n in ("q", "k", "state", "gamma", "v")})
    o, S = forward(t)
    ro, rS = delta_ref(f)
    assert rel(S[..., :half], rS[..., :half]) <= F32, rel(S[..., :half], rS[..., :half])
    assert rel(S[..., half:], rS[..., half:]) <= F32
    assert rel(o, ro) <= tol(dtype)
    go = torch.randn(t["v"].shape, generator=torch.Generator().manual_seed(1)).mul(2.0 ** -60).to(t["v"].dtype)
    d = dev(t)
    g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go.cuda(), grad_final=d["state"],
                                 state=torch.zeros_like(d["state"]))
    f["state"], gf = np.zeros_like(f["state"]), f["state"]
    ref = delta_ref(f, go.double().numpy(), gf)[2]["grad_state"]
    got = g["grad_state"].double().cpu().numpy()
    for part in (slice(0, half), slice(half, dk)):
        assert rel(got[..., part], ref[..., part]) <= GRAD_F32, rel(got[..., part], ref[..., part])


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
@pytest.mark.parametrize("T", [64, 200])
@pytest.mark.parametrize("e", [36, 44, 60])
def test_small_gradients_from_nothing(dtype, dk, dv, T, e):
    """grad_out as of a mean over many tokens, no gradient of the final state."""
    import torch
    from test_regression_amd import mesa
    say("case delta small gradients", (dtype, dk, dv, T, e))
    t, f = delta_inputs(241 + T, 1, 2, 2, T, dk, dv, dtype)
    go = (torch.from_numpy(np.random.default_rng(e).standard_normal(t["v"].shape)) * 2.0 ** -e).to(t["v"].dtype)
    d = dev(t)
    g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go.cuda(), d["state"])
    _, _, ref = delta_ref(f, go.double().numpy())
    for n, x in g.items():
        assert rel(x.double().cpu().numpy(), ref[n]) <= grad_tol(n, dtype), (n, rel(x.double().cpu().numpy(), ref[n]))


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
def test_gradients_of_small_values_from_no_state(dtype, dk, dv):
    say("case delta gradients of small values", (dtype, dk, dv))
    t, f = delta_inputs(251, 1, 2, 2, 200, dk, dv, dtype, start=False)
    scaled(t, f, "v", 2.0 ** -50)
    check_grads(t, f, dtype, 251, with_final=False)


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
def test_small_values_with_small_gradients(dtype, dk, dv):
    """Products of 2^-110."""
    import torch
    from test_regression_amd import mesa
    say("case delta small values, small gradients", (dtype, dk, dv))
    t, f = delta_inputs(255, 1, 2, 2, 200, dk, dv, dtype)
    for n in ("v", "state"):
        scaled(t, f, n, 2.0 ** -55)
    go = (torch.from_numpy(np.random.default_rng(255).standard_normal(t["v"].shape)) * 2.0 ** -55).to(t["v"].dtype)
    d = dev(t)
    g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go.cuda(), d["state"])
    _, _, ref = delta_ref(f, go.double().numpy())
    for n, x in g.items():
        assert rel(x.double().cpu().numpy(), ref[n]) <= grad_tol(n, dtype), (n, rel(x.double().cpu().numpy(), ref[n]))


@pytest.mark.parametrize("dtype,dk,dv", WIDTHS)
def test_small_gradients_before_a_reset(dtype, dk, dv):
    """Gradients of unit size behind a gate of 0, of 2^-40 before it."""
    import torch
    from test_regression_amd import mesa
    say("case delta small gradients before a reset", (dtype, dk, dv))
    t, f = delta_inputs(261, 1, 2, 2, 200, dk, dv, dtype)
    t["gamma"][:, :, 128] = 0.0
    f["gamma"] = t["gamma"].double().numpy()
    rng = np.random.default_rng(261)
    go = torch.from_numpy(rng.standard_normal(t["v"].shape))
    go[:, :, :128] *= 2.0 ** -40
    go = go.to(t["v"].dtype)
    gf = torch.from_numpy(rng.standard_normal(f["state"].shape)).float()
    d = dev(t)
    g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go.cuda(), d["state"], grad_final=gf.cuda())
    _, _, ref = delta_ref(f, go.double().numpy(), gf.double().numpy())
    got = {n: x.double().cpu().numpy() for n, x in g.items()}
    assert rel(got["grad_state"], ref["grad_state"]) <= GRAD_F32, rel(got["grad_state"], ref["grad_state"])
    for n in ("grad_q", "grad_k", "grad_v", "grad_beta", "grad_gamma"):
        for part in (slice(0, 128), slice(129, 200)):
            e = rel(got[n][:, :, part], ref[n][:, :, part])
            assert e <= grad_tol(n, dtype), (n, part, e)
