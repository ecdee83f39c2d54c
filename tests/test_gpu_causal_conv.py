"""The causal convolution over rows on the GPU (mesa_causal_conv and its gradients)
against float64 (tests/ssm_helpers.py).

Bounds, relative L2.  A float32 output is a sum of at most five products, an
exponential whose argument is off by that sum's rounding, a reciprocal and a product:
below 32 roundings of 2^-24.  The gradients of x sum four such terms more: 48.  The
weights' gradients are sums over up to 2^13 rows in runs of 32, eight runs and the
parts in turn, held to 96 2^-24 of the terms they sum.  bfloat16 results add 2^-8; the
fast exponential they take is off by |z| 2^-24 more, below 64 2^-24 at these sizes."""
import sys

import numpy as np
import pytest

from tests.ssm_helpers import conv_ref, near, store

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
OUT = {"f32": 32 * U, "bf16": 2.0 ** -8 + 96 * U}
GRAD = {"f32": 48 * U, "bf16": 2.0 ** -8 + 112 * U}
SUMS = 96 * U


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def c(t):
    return None if t is None else t.cuda()


CASES = [(1, 1, 8, None), (2, 3, 1, None), (3, 31, 16, None), (2, 32, 7, None), (2, 33, 300, None), (1, 257, 264, None),
         (2, 600, 20, None), (4, 40, 24, (0, 1, 2, 40)), (3, 100, 9, (33, 100, 64)), (2, 300, 8, (-3, 900))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("B,T,D,lens", CASES)
def test_conv(B, T, D, lens, W, dtype):
    import torch
    from test_regression_amd import mesa
    say("case conv", (B, T, D, lens, W, dtype))
    rng = np.random.default_rng(T + D + W)
    x, xf = store(rng.standard_normal((B, T, D)), dtype)
    w, wf = store(rng.standard_normal((W, D)) / W, "f32")
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    ln = None if lens is None else [min(max(k, 0), T) for k in lens]
    for full in (False, True):
        bias, bf = store(rng.standard_normal(D), "f32") if full else (None, None)
        hist, hf = store(rng.standard_normal((B, W - 1, D)), dtype) if full else (None, None)
        dy, dyf = store(rng.standard_normal((B, T, D)), dtype)
        y, h = mesa.mesa_causal_conv(c(x), c(w), c(bias), c(hist), silu=full, lens=n, return_hist=True)
        r = mesa.mesa_causal_conv_backward(c(x), c(w), c(dy), c(bias), c(hist), silu=full, lens=n)
        torch.cuda.synchronize()
        ry, rh, rg, terms = conv_ref(xf, wf, bf, hf, ln, full, dyf)
        near(y, ry, OUT[dtype], what="y")
        assert np.array_equal(h.double().cpu().numpy(), rh)
        near(r["grad_x"], rg["grad_x"], GRAD[dtype], what="grad_x")
        near(r["grad_w"], rg["grad_w"], SUMS, terms["grad_w"], what="grad_w")
        if full:
            near(r["grad_bias"], rg["grad_bias"], SUMS, terms["grad_bias"], what="grad_bias")
            near(r["grad_hist"], rg["grad_hist"], GRAD[dtype], what="grad_hist")
        else:
            assert r["grad_bias"] is None and r["grad_hist"] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_in_place(dtype):
    """Pieces of 0 to 70 tokens with the carried rows updated in place are one sequence, bit for bit."""
    import torch
    from test_regression_amd import mesa
    say("case conv pieces", dtype)
    torch.manual_seed(0)
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    for D in (24, 13):
        x, w, bias = torch.randn((3, 130, D), device="cuda").to(ty), torch.randn((4, D), device="cuda"), torch.randn(D, device="cuda")
        hist = torch.randn((3, 3, D), device="cuda").to(ty)
        whole, last = mesa.mesa_causal_conv(x, w, bias, hist, return_hist=True)
        cuts, ys = (0, 1, 2, 3, 3, 50, 120, 121, 130), []
        for a, b in zip(cuts, cuts[1:]):
            ys.append(mesa.mesa_causal_conv(x[:, a:b], w, bias, hist, hist_out=hist))
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(ys, 1), whole) and torch.equal(hist, last)


def test_views_and_no_tokens():
    import torch
    from test_regression_amd import mesa
    say("case conv views")
    torch.manual_seed(1)
    rows = torch.randn((2, 77, 50), device="cuda").to(torch.bfloat16)
    w, bias, dy = torch.randn((4, 19), device="cuda"), torch.randn(19, device="cuda"), torch.randn((2, 77, 19), device="cuda").to(torch.bfloat16)
    x = rows[..., 5:24]
    grows = torch.full_like(rows, 3.0)
    y = mesa.mesa_causal_conv(x, w, bias)
    r = mesa.mesa_causal_conv_backward(x, w, dy, bias, grad_x=grows[..., 5:24])
    xc = x.contiguous()
    y2, r2 = mesa.mesa_causal_conv(xc, w, bias), mesa.mesa_causal_conv_backward(xc, w, dy, bias)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(r[n], r2[n]) for n in r if r[n] is not None)
    assert bool((grows[..., :5] == 3).all()) and bool((grows[..., 24:] == 3).all())
    hist = torch.randn((2, 3, 19), device="cuda").to(torch.bfloat16)
    y, h = mesa.mesa_causal_conv(xc[:, :0], w, bias, hist, return_hist=True)
    r = mesa.mesa_causal_conv_backward(xc[:, :0], w, dy[:, :0].contiguous(), bias, hist)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 19) and torch.equal(h, hist)
    assert all(bool((r[n] == 0).all()) for n in ("grad_w", "grad_bias", "grad_hist"))


def test_wide_values():
    """Values whose exponentials leave float32's range."""
    import torch
    from test_regression_amd import mesa
    say("case conv wide")
    x, xf = store(np.linspace(-300, 300, 2 * 40 * 8).reshape(2, 40, 8), "f32")
    w, wf = store(np.ones((2, 8)), "f32")
    dy, dyf = store(np.ones((2, 40, 8)), "f32")
    y = mesa.mesa_causal_conv(x.cuda(), w.cuda())
    r = mesa.mesa_causal_conv_backward(x.cuda(), w.cuda(), dy.cuda())
    torch.cuda.synchronize()
    ry, _, rg, terms = conv_ref(xf, wf, dy=dyf)
    # an exponential's argument of 600 is off by 600 2^-24, where the result still has a size: below 64 2^-24 of the whole
    near(y, ry, 64 * U)
    near(r["grad_x"], rg["grad_x"], 64 * U)
    near(r["grad_w"], rg["grad_w"], SUMS, terms["grad_w"])
