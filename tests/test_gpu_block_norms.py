"""The norms around a layer on the GPU (mesa_gate_norm, mesa_residual_norm and
their gradients) against float64 forms.

Bounds, relative L2.  A float32 result is a row's sum of up to 16384 squares
(pairwise over lanes: 2 log2 of the lanes plus the few terms a lane adds in
turn, below 64 roundings of 2^-24), a division, a square root, an exponential
of error 2^-21 at the gates' size and a dozen products: below 96 2^-24 = 5.8e-6.
Parameter gradients sum up to 2^15 rows, at most 512 in turn in one register
and 512 parts: (512 + 512) 2^-24 / sqrt(1024) for roundings of random sign, and
terms of random sign can cancel to sqrt(rows) of their size, which the roundings
do too; with the terms' own error 96 2^-24 they stay below 1.2e-5.  bfloat16
results add their rounding, 2^-8.

The gradient of a norm is a difference, rsqrt(..) (d_u - u mean(d_u u)), which
vanishes where d_u lies along u: always for rows of one feature, where it is
d_u eps / (z^2 + eps) of two terms near d_u.  Each term carries the relative
error above, so the difference is held to that error of the terms, not of what
is left of them: the residual norm's row gradients are measured against
|rsqrt(..) d_u| + |dh'| where that is more than the gradient itself."""
import sys

import numpy as np
import pytest

from tests.delta_helpers import rel, store

pytestmark = pytest.mark.gpu
F32, SUMS, BF16 = 96 * 2.0 ** -24, 1.2e-5, 2.0 ** -8 + 96 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tol(dtype):
    return BF16 if dtype == "bf16" else F32


def name(t):
    import torch
    return "bf16" if t.dtype == torch.bfloat16 else "f32"


def near(got, ref, bound=None, terms=0.0):
    """`terms`: the norm of what the result is a difference of."""
    e = rel(got.double().cpu().numpy(), ref)
    size = np.linalg.norm(ref)
    e *= size / max(size, terms) if size else 1.0
    assert e <= (tol(name(got)) if bound is None else bound), e


def gate_ref(x, g, w, eps, dy=None):
    xt = x.transpose(0, 2, 1, 3)
    rs = 1.0 / np.sqrt((xt * xt).mean(-1, keepdims=True) + eps)
    u = xt * rs
    sig = np.ones_like(u) if g is None else 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    a = np.ones_like(u) if g is None else g * sig
    if dy is None:
        return u * w * a
    du = dy * w * a
    dx = rs * (du - u * (du * u).mean(-1, keepdims=True))
    return dict(grad_x=dx.transpose(0, 2, 1, 3), grad_w=(dy * u * a).sum((0, 1)),
                grad_gate=None if g is None else dy * u * w * sig * (1.0 + g * (1.0 - sig)))


@pytest.mark.parametrize("xt,gt", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1, 16), (2, 3, 9, 32), (1, 16, 1, 128), (3, 5, 17, 64), (2, 2, 100, 256),
                                     (1, 7, 300, 16), (5, 1, 8, 128)])
@pytest.mark.parametrize("gated", [True, False])
def test_gate_norm(B, H, T, d, xt, gt, gated):
    import torch
    from test_regression_amd import mesa
    say("case gate norm", (B, H, T, d, xt, gt, gated))
    rng = np.random.default_rng(B + H + T + d)
    x, xf = store(rng.standard_normal((B, H, T, d)), xt)
    g, gf = store(rng.standard_normal((B, T, H, d)) * 2, gt) if gated else (None, None)
    w, wf = store(1 + 0.2 * rng.standard_normal((H, d)), "f32")
    dy, dyf = store(rng.standard_normal((B, T, H, d)), gt)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = mesa.mesa_gate_norm(c(x), c(g), c(w), 1e-5, out_dtype=None if gated else dy.dtype)
    r = mesa.mesa_gate_norm_backward(c(x), c(g), c(w), c(dy), 1e-5)
    torch.cuda.synchronize()
    near(y, gate_ref(xf, gf, wf, 1e-5))
    ref = gate_ref(xf, gf, wf, 1e-5, dyf)
    assert y.shape == (B, T, H, d) and y.dtype == dy.dtype
    for n in ("grad_x", "grad_gate"):
        if ref[n] is not None:
            near(r[n], ref[n])
    assert gated or r["grad_gate"] is None
    near(r["grad_w"], ref["grad_w"], SUMS)


def test_gate_norm_rows_of_zeros_and_wide_gates():
    import torch
    from test_regression_amd import mesa
    say("case gate norm zeros")
    x, xf = store(np.random.default_rng(3).standard_normal((1, 2, 40, 64)), "f32")
    x[:, :, ::2] = 0
    xf[:, :, ::2] = 0
    g, gf = store(np.linspace(-200, 200, 40 * 2 * 64).reshape(1, 40, 2, 64), "f32")
    w, wf = store(np.ones((2, 64)), "f32")
    dy, dyf = store(np.ones((1, 40, 2, 64)), "f32")
    y = mesa.mesa_gate_norm(x.cuda(), g.cuda(), w.cuda(), 1e-6)
    r = mesa.mesa_gate_norm_backward(x.cuda(), g.cuda(), w.cuda(), dy.cuda(), 1e-6)
    torch.cuda.synchronize()
    assert bool((y[:, ::2] == 0).all()) and bool(torch.isfinite(y).all())
    near(y, gate_ref(xf, gf, wf, 1e-6))
    ref = gate_ref(xf, gf, wf, 1e-6, dyf)
    for n in ("grad_x", "grad_gate", "grad_w"):
        assert bool(torch.isfinite(r[n]).all())
        near(r[n], ref[n], SUMS)


def residual_ref(h, y, s, w, eps, dn=None, dh=None):
    z = h if y is None else h + (1.0 if s is None else s) * y
    rs = 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    u = z * rs
    if dn is None:
        return z, u * w
    d = dn * w
    dz = rs * (d - u * (d * u).mean(-1, keepdims=True)) + (0.0 if dh is None else dh)
    terms = np.linalg.norm(rs * d) + (0.0 if dh is None else np.linalg.norm(dh))
    return dict(terms=terms, grad_h=dz, grad_y=None if y is None else (1.0 if s is None else s) * dz, grad_w=(dn * u).sum(0),
                grad_scale=None if s is None else (dz * y).sum(0))


@pytest.mark.parametrize("ht,yt", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("R,D", [(1, 1), (3, 7), (5, 512), (1, 513), (257, 520), (1025, 1237), (1030, 2048), (2, 2056), (9, 1000), (2100, 640), (300, 8191), (260, 8200),
                                 (9, 4099), (3, 8192), (2, 9001), (1, 16384)])
def test_residual_norm(R, D, ht, yt):
    import torch
    from test_regression_amd import mesa
    rng = np.random.default_rng(R + D)
    h, hf = store(rng.standard_normal((R, D)) * 2, ht)
    y, yf = store(rng.standard_normal((R, D)), yt)
    s, sf = store(0.3 + 0.1 * rng.standard_normal(D), "f32")
    w, wf = store(1 + 0.2 * rng.standard_normal(D), "f32")
    dn, dnf = store(rng.standard_normal((R, D)), yt)
    dh, dhf = store(rng.standard_normal((R, D)), ht)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    for with_y, with_s, with_dh in ((True, True, True), (True, False, False), (False, False, True)):
        say("case residual norm", (R, D, ht, yt, with_y, with_s, with_dh))
        a = (y, yf) if with_y else (None, None)
        b = (s, sf) if with_s else (None, None)
        e = (dh, dhf) if with_dh else (None, None)
        hd = c(h)
        z, n = mesa.mesa_residual_norm(hd, c(a[0]), c(w), c(b[0]), 1e-5, out_dtype=None if with_y else dn.dtype)
        r = mesa.mesa_residual_norm_backward(hd, c(a[0]), c(w), c(dn), c(b[0]), 1e-5, grad_h_out=c(e[0]))
        torch.cuda.synchronize()
        rz, rn = residual_ref(hf, a[1], b[1], wf, 1e-5)
        near(z, rz)
        near(n, rn)
        assert n.dtype == dn.dtype and (with_y or z is hd)
        ref = residual_ref(hf, a[1], b[1], wf, 1e-5, dnf, e[1])
        # what dz's terms become in the results formed from dz
        scale_of = dict(grad_h=1.0, grad_y=np.abs(sf).max() if with_s else 1.0,
                        grad_scale=np.abs(yf).max() if R == 1 else 0.0)
        for k in ("grad_h", "grad_y", "grad_w", "grad_scale"):
            assert (r[k] is None) == (ref[k] is None)
            if ref[k] is not None:
                near(r[k], ref[k], SUMS if k in ("grad_w", "grad_scale") else None, ref["terms"] * scale_of.get(k, 0.0))
        if with_y:   # in place over the residual
            mesa.mesa_residual_norm(hd, c(a[0]), c(w), c(b[0]), 1e-5, h_out=hd)
            assert torch.equal(hd, z)


def test_parameter_gradients_over_many_rows_and_every_run_the_same():
    import torch
    from test_regression_amd import mesa
    say("case sums over many rows")
    torch.manual_seed(5)
    h, y, dn = (torch.randn(20011, 136, device="cuda") for _ in range(3))
    w, s = torch.ones(136, device="cuda"), torch.full((136,), 0.5, device="cuda")
    a = mesa.mesa_residual_norm_backward(h, y, w, dn, s)
    b = mesa.mesa_residual_norm_backward(h, y, w, dn, s)
    ref = residual_ref(*(t.double().cpu().numpy() for t in (h, y, s, w)), 1e-6, dn.double().cpu().numpy())
    for n in ("grad_w", "grad_scale"):
        assert torch.equal(a[n], b[n])
        near(a[n], ref[n], SUMS)
    x, g, dy = torch.randn(2, 3, 5001, 64, device="cuda"), *(torch.randn(2, 5001, 3, 64, device="cuda") for _ in range(2))
    w = torch.ones(3, 64, device="cuda")
    a, b = (mesa.mesa_gate_norm_backward(x, g, w, dy) for _ in range(2))
    assert torch.equal(a["grad_w"], b["grad_w"])
    near(a["grad_w"], gate_ref(*(t.double().cpu().numpy() for t in (x, g, w)), 1e-6, dy.double().cpu().numpy())["grad_w"],
         SUMS)


def test_no_rows():
    import torch
    from test_regression_amd import mesa
    say("case no rows")
    w = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    z, n = mesa.mesa_residual_norm(e, e, w, w)
    assert z.shape == n.shape == (0, 8)
    r = mesa.mesa_residual_norm_backward(e, e, w, e, w)
    assert bool((r["grad_w"] == 0).all()) and bool((r["grad_scale"] == 0).all())
    x, g, w = torch.empty(2, 3, 0, 16, device="cuda"), torch.empty(2, 0, 3, 16, device="cuda"), torch.ones(3, 16, device="cuda")
    assert mesa.mesa_gate_norm(x, g, w).shape == (2, 0, 3, 16)
    assert bool((mesa.mesa_gate_norm_backward(x, g, w, g)["grad_w"] == 0).all())
