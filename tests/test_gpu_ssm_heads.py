"""Gradients of the state space scan where a workgroup goes over several heads, where
segments see one another, and without the operands that may be absent; the layer's
gradients of b and c at the plain bound.

The reference is the definition a token at a time, in float64 on the device, so that
many rows and heads stay cheap; it is checked here against the one in
tests/ssm_helpers.py, whose bounds these tests share.  Every head is held to the bound
by itself, so that one head's error does not vanish in the others' size."""
import sys

import numpy as np
import pytest

from tests import test_gpu_ssm as scan
from tests import test_gpu_ssm_layer as layer
from tests.ssm_helpers import near, ssm_inputs, ssm_ref, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def device_ref(g, lens, go=None, gf=None, plus=True):
    """As ssm_ref (tests/ssm_helpers.py), of tensors where they are."""
    import torch
    x, b, c, dt, A = (g[n].double() for n in ("x", "b", "c", "dt", "A"))
    B, H, T, dv = x.shape
    Hk, dk = b.shape[1], b.shape[3]
    r = H // Hk
    zero = torch.zeros(H, dtype=torch.float64, device=x.device)
    skip, bias = (zero if g[n] is None else g[n].double() for n in ("D", "dt_bias"))
    live = torch.arange(T, device=x.device)[None] < torch.tensor(list(lens), device=x.device)[:, None]
    on = live[:, None]
    raw = dt + bias[:, None]
    step = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs())) if plus else raw
    step = torch.where(on, step, 0.0)
    decay = torch.exp(step * A[:, None])
    x, b, c = (torch.where(on[..., None], y, 0.0) for y in (x, b.repeat_interleave(r, 1), c.repeat_interleave(r, 1)))
    S = torch.zeros((B, H, dv, dk), dtype=torch.float64, device=x.device) if g["state"] is None else g["state"].double()
    out, before = torch.zeros_like(x), []
    for t in range(T):
        if go is not None:
            before.append(S)
        S = decay[:, :, t, None, None] * S + (step[:, :, t, None] * x[:, :, t])[..., None] * b[:, :, t, None]
        out[:, :, t] = (S * c[:, :, t, None]).sum(-1) + skip[:, None] * x[:, :, t]
    out = torch.where(on[..., None], out, 0.0)
    if go is None:
        return out, S
    gx, gb, gc, dstep, dlog, tdt = (torch.zeros_like(y) for y in (x, b, c, step, step, step))
    R, after, go = torch.zeros_like(S) if gf is None else gf.double(), S, torch.where(on[..., None], go.double(), 0.0)
    for t in reversed(range(T)):
        do, bt, ct, xt, st = go[:, :, t], b[:, :, t], c[:, :, t], x[:, :, t], step[:, :, t, None]
        gc[:, :, t] = (after * do[..., None]).sum(2)
        R = R + do[..., None] * ct[:, :, None]
        Rb = (R * bt[:, :, None]).sum(-1)
        gx[:, :, t] = st * Rb + skip[:, None] * do
        gb[:, :, t] = st * (R * xt[..., None]).sum(2)
        mix = R * before[t]
        dstep[:, :, t] = (Rb * xt).sum(-1)
        dlog[:, :, t] = mix.sum((2, 3)) * decay[:, :, t]
        tdt[:, :, t] = (Rb * xt).abs().sum(-1) + A.abs() * mix.abs().sum((2, 3)) * decay[:, :, t]
        R = R * decay[:, :, t, None, None]
        after = before[t]
    slope = torch.sigmoid(raw) if plus else torch.ones_like(raw)
    graw, tdt = (torch.where(on, y, 0.0) for y in ((dstep + A[:, None] * dlog) * slope, tdt))
    fold = lambda y: y.reshape(B, Hk, r, T, dk).sum(2)  # noqa: E731
    grads = dict(grad_x=torch.where(on[..., None], gx, 0.0), grad_b=fold(gb), grad_c=fold(gc), grad_dt=graw,
                 grad_A=(step * dlog).sum((0, 2)), grad_D=(go * x).sum((0, 2, 3)), grad_dt_bias=graw.sum((0, 2)), grad_state=R)
    # what the step sizes' and the parameters' gradients are sums of
    terms = dict(grad_dt=tdt * slope, grad_dt_bias=(tdt * slope).sum((0, 2)), grad_A=(tdt * step / A.abs()[:, None]).sum((0, 2)),
                 grad_D=(go * x).abs().sum((0, 2, 3)))
    return out, S, grads, terms


# the axis of heads in each result
HEADS = dict(out=1, final=1, grad_x=1, grad_b=1, grad_c=1, grad_dt=1, grad_state=1, grad_A=0, grad_D=0, grad_dt_bias=0)


def held(name, got, ref, terms=None, bound=None):
    """Head by head."""
    axis = HEADS[name]
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    for h in range(ref.shape[axis]):
        size = 0.0 if terms is None else float(terms.select(axis, h).norm())
        near(got.select(axis, h), ref.select(axis, h).cpu().numpy(), bound, terms=size, what=(name, h))


def all_held(got, ref, terms):
    for n, y in ref.items():
        if got[n] is not None:
            held(n, got[n], y, terms.get(n))


def run(t, lens, dtype, seed, final=True, plus=True):
    """Forward and gradients held to the reference, head by head; returns the gradients."""
    import torch
    from test_regression_amd import mesa
    B, H, T, dv = t["x"].shape
    dk = t["b"].shape[3]
    rng = np.random.default_rng(seed)
    go, gf = store(rng.standard_normal((B, H, T, dv)), dtype)[0].cuda(), store(rng.standard_normal((B, H, dv, dk)), "f32")[0].cuda()
    gf = gf if final else None
    g = scan.dev(t)
    out, state = scan.forward(mesa, g, softplus=plus)
    r = scan.backward(mesa, g, go, gf, softplus=plus)
    torch.cuda.synchronize()
    ro, rs, rg, terms = device_ref(g, [min(max(n, 0), T) for n in lens], go, gf, plus)
    held("out", out, ro)
    held("final", state, rs)
    all_held(r, rg, terms)
    for n in ("D", "dt_bias", "state"):
        assert (r["grad_" + n] is None) == (t[n] is None)
    return r


def test_the_reference_is_the_definition():
    import torch
    t, f = ssm_inputs(1, 2, 2, 4, 70, 32, 16, "f32", True, (70, 33))
    go = np.random.default_rng(2).standard_normal((2, 4, 70, 16))
    gf = np.random.default_rng(3).standard_normal((2, 4, 16, 32))
    ro, rs, rg, terms = ssm_ref(f, go, gf)
    o, s, g, tm = device_ref(scan.dev(t), (70, 33), torch.from_numpy(go).cuda(), torch.from_numpy(gf).cuda())
    # both sum at most 2^12 terms in float64, each in its own order
    near(o, ro, 2.0 ** -40)
    near(s, rs, 2.0 ** -40)
    for n, y in rg.items():
        near(g[n], y, 2.0 ** -40, terms=terms.get(n, 0.0), what=n)


# (B, Hk, H, T, dk, dv): with the 256 workgroups that the gradients take, the heads of one
# b and c go to a workgroup by three or more
MANY = [(43, 1, 3, 130, 128, 64),    # 129 chunks: 3 heads, dB and dC stored directly
        (40, 1, 9, 130, 32, 64),     # 120 chunks: two parts, of 4 and 5 heads
        (64, 1, 7, 130, 16, 16),     # 192 chunks, 7 heads
        (22, 2, 8, 130, 64, 128),    # two groups of 4 heads, two pieces of dv each
        (65, 1, 3, 66, 128, 128)]    # 3 heads in two pieces each


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", MANY)
def test_several_heads_a_workgroup(size, dtype):
    B, Hk, H, T, dk, dv = size
    say("case heads", size, dtype)
    rng = np.random.default_rng(B)
    for lens in ([T] * B, [(0, 1, 64, 65, T)[i % 5] if i < 5 else int(rng.integers(0, T + 1)) for i in range(B)]):
        t, _ = ssm_inputs(B + H, B, Hk, H, T, dk, dv, dtype, True, lens)
        run(t, lens, dtype, H)


# chunks that do not divide the card: parts of two to eight heads in several turns
TURNS = [(64, 1, 32, 130, 16, 16), (107, 1, 8, 130, 32, 32), (20, 4, 24, 200, 64, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", TURNS)
def test_parts_in_several_turns(size, dtype):
    B, Hk, H, T, dk, dv = size
    say("case turns", size, dtype)
    rng = np.random.default_rng(B)
    lens = [int(rng.integers(0, T + 1)) for _ in range(B)]
    t, _ = ssm_inputs(B + H, B, Hk, H, T, dk, dv, dtype, True, lens)
    run(t, lens, dtype, H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 2, 1100, 32, 16), (1, 2, 2, 2111, 64, 128), (3, 1, 1, 1537, 128, 64), (1, 1, 3, 700, 128, 128)])
def test_gradients_of_segments_that_see_one_another(size, dtype):
    B, Hk, H, T, dk, dv = size
    say("case gradients of segments", size, dtype)
    for lens in ([T] * B, [T - 300 * (i + 1) for i in range(B)] if B == 1 else [T, 600, 63]):
        t, f = ssm_inputs(T + 1, B, Hk, H, T, dk, dv, dtype, True, lens)
        t["A"] = store(f["A"] * 0.02, "f32")[0]
        run(t, lens, dtype, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("absent", [("D",), ("dt_bias",), ("D", "dt_bias", "state")])
def test_absent_operands(absent, dtype):
    """Without the skip, the steps' bias, a start: sequences, gradients and tokens."""
    import torch
    from test_regression_amd import mesa
    say("case absent", absent, dtype)
    t, _ = ssm_inputs(7, 2, 2, 6, 150, 64, 64, dtype)
    for n in absent:
        t[n] = None
    run(t, [150] * 2, dtype, 3, final="state" not in absent)
    if "state" in absent:
        return
    g = scan.dev(t)
    state, outs = g["state"].clone(), []
    for i in range(3):
        outs.append(mesa.mesa_ssm_step(*(g[n][:, :, i] for n in ("x", "b", "c", "dt")), g["A"], state, g["D"], g["dt_bias"]))
    torch.cuda.synchronize()
    ro, rs = device_ref({n: y[:, :, :3] if n in ("x", "b", "c", "dt") else y for n, y in g.items()}, [3, 3])
    held("out", torch.stack(outs, 2), ro)
    held("final", state, rs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,lens", [(2, 150, 1, 3, 32, 64, (150, 41)), (1, 1290, 1, 2, 64, 32, None)])
def test_layer_gradients_of_b_and_c(B, T, Hk, H, dk, dv, lens, dtype):
    """In a layer of more tokens than one the gradients of b and c hold the plain bound."""
    import torch
    from test_regression_amd import mesa
    say("case layer b and c", (B, T, Hk, H, dk, dv, lens, dtype))
    L = layer.Layer(mesa, 3, B, Hk, H, dk, dv, dtype)
    rows, dt, gate, grad = layer.inputs(5, L, B, T)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    r = L.forward(rows, dt, gate, lens=n)
    g = L.backward(r, rows, dt, gate, grad, lens=n)
    torch.cuda.synchronize()
    given = dict(x=r["x"], b=r["rb"], c=r["rc"], dt=dt.transpose(1, 2), A=L.p["A"], D=L.p["skip"], dt_bias=L.p["dt_bias"], state=None)
    _, _, ref, _ = device_ref(given, lens or [T] * B, g["gate"]["grad_x"])
    for name in ("grad_b", "grad_c"):
        held(name, g["ssm"][name], ref[name])
