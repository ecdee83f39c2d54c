"""The state space scan on the GPU (mesa_ssm_forward, mesa_ssm_backward, mesa_ssm_step)
against its definition in float64 (tests/ssm_helpers.py, with the bounds)."""
import sys

import numpy as np
import pytest

from tests.ssm_helpers import F32, near, rel, ssm_inputs, ssm_ref, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def dev(t):
    return {n: None if y is None else y.cuda() for n, y in t.items()}


def forward(mesa, g, **kw):
    return mesa.mesa_ssm_forward(g["x"], g["b"], g["c"], g["dt"], g["A"], g["D"], g["dt_bias"], g["state"], lens=g["lens"],
                                 return_final=True, **kw)


def backward(mesa, g, go, gf, **kw):
    return mesa.mesa_ssm_backward(g["x"], g["b"], g["c"], g["dt"], g["A"], go, g["D"], g["dt_bias"], g["state"], lens=g["lens"],
                                  grad_final=gf, **kw)


def grads_near(r, ref, terms, start=True):
    for n, y in ref.items():
        if n == "grad_state" and not start:
            assert r[n] is None
            continue
        near(r[n], y, terms=terms.get(n, 0.0), what=n)


# (B, Hk, H, T, dk, dv, start, lens)
SIZES = [(1, 1, 1, 1, 16, 16, True, None), (2, 1, 3, 5, 32, 16, False, None), (1, 2, 4, 64, 16, 32, True, None),
         (2, 2, 2, 65, 64, 64, True, None), (1, 1, 5, 127, 128, 64, False, None), (1, 2, 6, 130, 64, 128, True, None),
         (1, 1, 2, 200, 128, 128, True, None), (3, 1, 2, 100, 32, 64, True, (0, 1, 100)), (4, 2, 2, 193, 64, 16, True, (64, 193, 128, 65)),
         (2, 1, 7, 70, 16, 128, False, (3, 70)), (2, 1, 2, 150, 128, 32, True, (-4, 400))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_gradients(size, dtype):
    import torch
    from test_regression_amd import mesa
    B, Hk, H, T, dk, dv, start, lens = size
    say("case ssm", size, dtype)
    t, f = ssm_inputs(T + dk + dv, B, Hk, H, T, dk, dv, dtype, start, lens)
    f["lens"] = [min(max(n, 0), T) for n in f["lens"]]
    rng = np.random.default_rng(T)
    go, gof = store(rng.standard_normal((B, H, T, dv)), dtype)
    gf, gff = store(rng.standard_normal((B, H, dv, dk)), "f32")
    g = dev(t)
    out, final = forward(mesa, g)
    r = backward(mesa, g, go.cuda(), gf.cuda())
    torch.cuda.synchronize()
    ro, rf, rg, terms = ssm_ref(f, gof, gff)
    near(out, ro, what="out")
    near(final, rf, what="final")
    grads_near(r, rg, terms, start)
    for b, n in enumerate(f["lens"]):
        assert bool((out[b, :, n:] == 0).all()) and bool((r["grad_x"][b, :, n:] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 2, 1100, 32, 16), (1, 2, 2, 2111, 64, 128), (3, 1, 1, 1537, 128, 64)])
def test_segments(size, dtype):
    """Lengths that are passed over in segments, whole and with lengths that end in each of them."""
    import torch
    from test_regression_amd import mesa
    B, Hk, H, T, dk, dv = size
    say("case segments", size, dtype)
    for lens in (None, [T - 700 * (i + 1) for i in range(B)] if B == 1 else [T, 600, 63]):
        t, f = ssm_inputs(T, B, Hk, H, T, dk, dv, dtype, True, lens)
        f["A"] *= 0.02   # so that segments see one another
        t["A"], f["A"] = store(f["A"], "f32")
        out, final = forward(mesa, dev(t))
        torch.cuda.synchronize()
        ro, rf = ssm_ref(f)
        near(out, ro, what="out")
        near(final, rf, what="final")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_of_all_sizes(dtype):
    """Tokens that forget all among tokens that forget nearly nothing, padded and masked
    ones, and raw steps that need no softplus."""
    import torch
    from test_regression_amd import mesa
    say("case decays", dtype)
    t, f = ssm_inputs(5, 2, 1, 4, 150, 64, 64, dtype, True, None, "f32", fast=True)
    raw = f["dt"].copy()
    raw[:, :, ::7] = 30.0
    raw[:, :, 3::11] = -40.0
    raw[:, :, 5::13] = -np.inf
    raw[:, :, 9::17] = np.finfo(np.float32).min
    t["dt"], f["dt"] = store(raw, "f32")
    f["dt"][~np.isfinite(f["dt"])] = -1e300
    g = dev(t)
    go, gof = store(np.random.default_rng(1).standard_normal((2, 4, 150, 64)), dtype)
    out, final = forward(mesa, g)
    r = backward(mesa, g, go.cuda(), None)
    torch.cuda.synchronize()
    ro, rf, rg, terms = ssm_ref(f, gof)
    near(out, ro, what="out")
    near(final, rf, what="final")
    grads_near(r, rg, terms)
    steps = np.abs(f["dt"]) % 3.0
    t["dt"], f["dt"] = store(steps, "f32")
    t["dt_bias"], f["dt_bias"] = None, np.zeros(4)
    g = dev(t)
    out, final = forward(mesa, g, softplus=False)
    r = backward(mesa, g, go.cuda(), None, softplus=False)
    torch.cuda.synchronize()
    ro, rf, rg, terms = ssm_ref(f, gof, plus=False)
    near(out, ro, what="out")
    near(final, rf, what="final")
    assert r.pop("grad_dt_bias") is None and rg.pop("grad_dt_bias") is not None
    grads_near(r, rg, terms)


@pytest.mark.parametrize("dtype,other", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_views_of_projection_rows(dtype, other):
    """x, b, c and dt as slices of rows, the gradients into slices of rows, at an odd row length."""
    import torch
    from test_regression_amd import mesa
    say("case views", dtype, other)
    B, Hk, H, T, dk, dv = 2, 2, 4, 90, 32, 64
    t, f = ssm_inputs(8, B, Hk, H, T, dk, dv, dtype, True, None, other)
    width = H * dv + 2 * Hk * dk + 3
    ty = t["x"].dtype

    def split(rows):
        a, n = 1 + H * dv, Hk * dk
        return [rows[..., i:j].unflatten(-1, (h, -1)).transpose(1, 2) for i, j, h in ((1, a, H), (a, a + n, Hk), (a + n, a + 2 * n, Hk))]
    rows = torch.full((B, T, width), float("nan"), dtype=ty, device="cuda")
    for v, n in zip(split(rows), "xbc"):
        v.copy_(t[n].cuda())
    gates = torch.full((B, T, H + 5), float("nan"), dtype=t["dt"].dtype, device="cuda")
    gates[..., 2:2 + H] = t["dt"].cuda().transpose(1, 2)
    g = dev(t)
    whole, final = forward(mesa, g)
    go = torch.randn((B, H, T, dv), device="cuda").to(ty)
    ref = backward(mesa, g, go, None)
    g["x"], g["b"], g["c"] = split(rows)
    g["dt"] = gates[..., 2:2 + H].transpose(1, 2)
    out, fin = forward(mesa, g)
    grows, ggates = torch.full_like(rows, 7.0), torch.full_like(gates, 7.0)
    gx, gb, gc = split(grows)
    r = backward(mesa, g, go, None, grad_x=gx, grad_b=gb, grad_c=gc, grad_dt=ggates[..., 2:2 + H].transpose(1, 2))
    torch.cuda.synchronize()
    assert torch.equal(out, whole) and torch.equal(fin, final)
    for n in ref:
        assert torch.equal(r[n], ref[n]), n
    assert bool((grows[..., 0] == 7).all()) and bool((grows[..., -2:] == 7).all())
    assert bool((ggates[..., :2] == 7).all()) and bool((ggates[..., 2 + H:] == 7).all())


def test_broadcast_inputs():
    """b and c that all rows of the batch share (stride 0)."""
    import torch
    from test_regression_amd import mesa
    say("case broadcast")
    t, f = ssm_inputs(4, 3, 1, 2, 70, 64, 32, "f32")
    for n in "bc":
        t[n], f[n] = t[n][:1].expand(3, -1, -1, -1), np.repeat(f[n][:1], 3, 0)
    g = {n: None if y is None else y.cuda() for n, y in t.items() if n not in "bc"}
    g["b"], g["c"] = (t[n][:1].cuda().expand(3, -1, -1, -1) for n in "bc")
    assert g["b"].stride(0) == 0
    out, final = forward(mesa, g)
    torch.cuda.synchronize()
    ro, rf = ssm_ref(f)
    near(out, ro)
    near(final, rf)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,Hk,H,dk,dv", [(1, 1, 1, 16, 16), (3, 2, 4, 32, 128), (2, 1, 5, 64, 64), (5, 3, 3, 128, 16), (1, 1, 2, 128, 128)])
def test_step(N, Hk, H, dk, dv, dtype):
    import torch
    from test_regression_amd import mesa
    say("case step", (N, Hk, H, dk, dv, dtype))
    t, f = ssm_inputs(dk + dv, N, Hk, H, 3, dk, dv, dtype)
    g = dev(t)
    state, outs = g["state"], []
    for i in range(3):
        rows = torch.cat([g[n][:, :, i].flatten(1) for n in "xbc"], 1)   # views of one row, as a convolution leaves them
        a, n = H * dv, Hk * dk
        x, b, c = rows[:, :a].unflatten(1, (H, dv)), rows[:, a:a + n].unflatten(1, (Hk, dk)), rows[:, a + n:].unflatten(1, (Hk, dk))
        outs.append(mesa.mesa_ssm_step(x, b, c, g["dt"][:, :, i], g["A"], state, g["D"], g["dt_bias"]))
    torch.cuda.synchronize()
    ro, rf = ssm_ref(f)
    near(torch.stack(outs, 2), ro)
    near(state, rf)


def test_pieces_and_tokens_join():
    """A sequence in one call, in pieces with the state carried in place, and its last tokens by steps."""
    import torch
    from test_regression_amd import mesa
    say("case pieces")
    t, f = ssm_inputs(21, 2, 1, 2, 140, 64, 64, "f32")
    g = dev(t)
    whole, final = forward(mesa, g)
    state, outs = g["state"].clone(), []
    for a, b in ((0, 64), (64, 65), (65, 65), (65, 137)):
        p = {n: g[n][:, :, a:b] for n in ("x", "b", "c", "dt")}
        o, s = mesa.mesa_ssm_forward(p["x"], p["b"], p["c"], p["dt"], g["A"], g["D"], g["dt_bias"], state, final_state=state)
        assert s is state
        outs.append(o)
    for i in range(137, 140):
        outs.append(mesa.mesa_ssm_step(g["x"][:, :, i], g["b"][:, :, i], g["c"][:, :, i], g["dt"][:, :, i], g["A"], state, g["D"],
                                       g["dt_bias"])[:, :, None])
    torch.cuda.synchronize()
    ref, rs = whole.double().cpu().numpy(), final.double().cpu().numpy()
    near(torch.cat(outs, 2), ref, 2 * F32)
    near(state, rs, 2 * F32)


def test_no_tokens():
    import torch
    from test_regression_amd import mesa
    say("case no tokens")
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    S = torch.randn((2, 3, 16, 32), device="cuda")
    a = (z(2, 3, 0, 16), z(2, 1, 0, 32), z(2, 1, 0, 32), z(2, 3, 0), -torch.ones(3, device="cuda"))
    out, final = mesa.mesa_ssm_forward(*a, torch.ones(3, device="cuda"), None, S, return_final=True)
    r = mesa.mesa_ssm_backward(*a, z(2, 3, 0, 16), torch.ones(3, device="cuda"), None, S, grad_final=2 * S)
    torch.cuda.synchronize()
    assert out.shape == (2, 3, 0, 16) and torch.equal(final, S) and torch.equal(r["grad_state"], 2 * S)
    assert bool((r["grad_A"] == 0).all()) and bool((r["grad_D"] == 0).all())


def test_runs_repeat_bit_for_bit_and_heads_are_apart():
    """The same twice; a NaN in one head's values stays in that head."""
    import torch
    from test_regression_amd import mesa
    say("case repeat")
    t, _ = ssm_inputs(2, 2, 1, 4, 300, 64, 64, "bf16")
    g = dev(t)
    go = torch.randn((2, 4, 300, 64), device="cuda").to(torch.bfloat16)
    a, b = forward(mesa, g), forward(mesa, g)
    ga, gb = backward(mesa, g, go, None), backward(mesa, g, go, None)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    g["x"] = g["x"].clone()
    g["x"][1, 2, 70] = float("nan")
    c, s = forward(mesa, g)
    torch.cuda.synchronize()
    apart = torch.ones((2, 4), dtype=torch.bool)
    apart[1, 2] = False
    assert torch.equal(c[apart], a[0][apart]) and torch.equal(s[apart], a[1][apart])
    assert torch.equal(c[1, 2, :64], a[0][1, 2, :64]) and bool(c[1, 2, 70:].isnan().all())


def test_gradients_against_differences():
    """The float32 gradients against central differences of the definition."""
    import torch
    from test_regression_amd import mesa
    say("case differences")
    t, f = ssm_inputs(3, 1, 1, 2, 9, 16, 16, "f32")
    rng = np.random.default_rng(0)
    go, gof = store(rng.standard_normal((1, 2, 9, 16)), "f32")
    gf, gff = store(rng.standard_normal((1, 2, 16, 16)), "f32")
    r = backward(mesa, dev(t), go.cuda(), gf.cuda())
    torch.cuda.synchronize()

    def loss(f):
        o, s = ssm_ref(f)
        return (o * gof).sum() + (s * gff).sum()
    for n in ("x", "b", "c", "dt", "A", "D", "dt_bias", "state"):
        g = r["grad_" + n].double().cpu().numpy()
        for _ in range(4):
            at = tuple(rng.integers(0, k) for k in f[n].shape)
            h = 1e-4
            up, down = ({**f, n: f[n].copy()} for _ in range(2))
            up[n][at] += h
            down[n][at] -= h
            d = (loss(up) - loss(down)) / (2 * h)
            # the difference is off by h^2 / 6 of the third derivative: below 1e-6 of the gradient's size here
            assert abs(g[at] - d) <= 1e-4 * max(np.abs(g).max(), 1.0), (n, at, g[at], d)


def test_long_offsets():
    """Rows that lie past 2^31 elements from the tensor's start."""
    import torch
    from test_regression_amd import mesa
    say("case long offsets")
    B, H, T, d = 2, 1, 66, 16
    big = torch.zeros((B, (1 << 31) + 64), dtype=torch.bfloat16, device="cuda")
    t, f = ssm_inputs(6, B, 1, H, T, d, d, "bf16")
    g = dev(t)
    x = big[:, -T * d:].unflatten(1, (1, T, d))
    x.copy_(g["x"])
    g["x"] = x
    out, final = forward(mesa, g)
    torch.cuda.synchronize()
    ro, rf = ssm_ref(f)
    near(out, ro)
    assert rel(final.double().cpu().numpy(), rf) <= F32
