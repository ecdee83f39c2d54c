"""The weights' gradients of the causal convolution as sums: long batches, lengths on
both sides of a thread's run and of a workgroup's eight, and slopes of far negative
values.

Bounds, relative to the sizes of the terms.  A thread adds at most 256 tokens in
float32, a workgroup the eight runs; workgroups are joined by eight in float32 and these
in float64, and the result is rounded once: a product, min(T, 256) + 8 + 3 additions and
the rounding, whatever the batch and the length.  A term with SiLU is met with at most 48 roundings more (z's five
products, an exponential, a reciprocal, the slope's three)."""
import sys

import numpy as np
import pytest

from tests.ssm_helpers import conv_ref, near, store

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def sums(T, silu=True):
    return (min(T, 256) + 8 + 3 + 2 + (48 if silu else 0)) * U


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def test_terms_of_one_size_over_a_long_batch():
    """(1 + 2^-7)^2 = 1 + 2^-6 + 2^-14 a token: additions to more than 1024 such terms lose
    the last part in float32, always downwards."""
    import torch
    from test_regression_amd import mesa
    say("case conv long batch")
    B, T, D = 512, 32768, 4
    x = torch.full((B, T, D), 1 + 2.0 ** -7, dtype=torch.bfloat16, device="cuda")
    r = mesa.mesa_causal_conv_backward(x, torch.ones((1, D), device="cuda"), x, torch.zeros(D, device="cuda"), silu=False)
    torch.cuda.synchronize()
    for name, one in (("grad_w", (1 + 2.0 ** -7) ** 2), ("grad_bias", 1 + 2.0 ** -7)):
        got, want = r[name].double().cpu().numpy(), B * T * one
        assert np.abs(got - want).max() <= sums(T, False) * want, (name, (got - want) / want / U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,W", [(512, 2100, 3, 4), (515, 1030, 4, 2)])
def test_long_runs(B, T, D, W, dtype):
    """Batches whose workgroups fill the card, so that a thread's run is long, and the same
    gradients from run to run."""
    import torch
    from test_regression_amd import mesa
    say("case conv long runs", (B, T, D, W, dtype))
    rng = np.random.default_rng(T)
    x, xf = store(rng.standard_normal((B, T, D)) + 1.0, dtype)
    dy, dyf = store(rng.standard_normal((B, T, D)) + 1.0, dtype)
    w, wf = store(rng.standard_normal((W, D)) / W, "f32")
    bias, bf = store(rng.standard_normal(D), "f32")
    args = (x.cuda(), w.cuda(), dy.cuda(), bias.cuda())
    r, again = mesa.mesa_causal_conv_backward(*args), mesa.mesa_causal_conv_backward(*args)
    torch.cuda.synchronize()
    _, _, rg, terms = conv_ref(xf, wf, bf, dy=dyf)
    for n in ("grad_w", "grad_bias"):
        near(r[n], rg[n], sums(T), terms[n], what=n)
        assert torch.equal(r[n], again[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 3, 4])
@pytest.mark.parametrize("T", [15, 16, 17, 127, 128, 129])
def test_lengths_around_the_runs(T, W, dtype):
    import torch
    from test_regression_amd import mesa
    say("case conv runs", (T, W, dtype))
    rng = np.random.default_rng(T)
    for D in (5, 260):
        x, xf = store(rng.standard_normal((3, T, D)), dtype)
        dy, dyf = store(rng.standard_normal((3, T, D)), dtype)
        w, wf = store(rng.standard_normal((W, D)) / W, "f32")
        bias, bf = store(rng.standard_normal(D), "f32")
        lens = [T, T - 1, T // 2]
        r = mesa.mesa_causal_conv_backward(x.cuda(), w.cuda(), dy.cuda(), bias.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda())
        y = mesa.mesa_causal_conv(x.cuda(), w.cuda(), bias.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        ry, _, rg, terms = conv_ref(xf, wf, bf, None, lens, True, dyf)
        out = 2.0 ** -8 if dtype == "bf16" else 0.0
        near(y, ry, out + 96 * U, what="y")
        near(r["grad_x"], rg["grad_x"], out + 112 * U, what="grad_x")
        for n in ("grad_w", "grad_bias"):
            near(r[n], rg[n], sums(T), terms[n], what=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("z", [-81.875, -65.625, -12.0, 2.0])
def test_slopes_of_far_values(z, dtype):
    """Float32 gradients of the weights take the exponential to its own rounding, of
    bfloat16 rows too.  z = bias + x is exact here, so a term is met with the exponential
    (1 of its own, and what ln 2 in float32 leaves of its power: 2^-28 of z, 5 at most), a
    sum, a reciprocal (2), the slope's three operations (in which 1 - s is off by two
    roundings of 1 where s is near it, times z), the product, and 3 + 8 additions: 24
    roundings."""
    import torch
    from test_regression_amd import mesa
    say("case conv far values", z, dtype)
    x, xf = store(np.full((1, 4, 4), 0.5), dtype)
    dy, dyf = store(np.ones((1, 4, 4)), dtype)
    w, wf = store(np.ones((1, 4)), "f32")
    bias, bf = store(np.full(4, z - 0.5), "f32")
    r = mesa.mesa_causal_conv_backward(x.cuda(), w.cuda(), dy.cuda(), bias.cuda())
    torch.cuda.synchronize()
    _, _, rg, _ = conv_ref(xf, wf, bf, dy=dyf)
    for n in ("grad_w", "grad_bias"):
        got = r[n].double().cpu().numpy()
        assert np.abs(got - rg[n]).max() <= 24 * U * np.abs(rg[n]).max(), (n, (got - rg[n]).max() / np.abs(rg[n]).max() / U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slopes_at_the_ends_of_the_range(dtype):
    """Slopes of values up to float32's largest are exactly 0 and 1."""
    import torch
    from test_regression_amd import mesa
    say("case conv range", dtype)
    x, xf = store(np.array([3.3e38, -3.3e38, 2.0e38, -2.0e38, 1e30, -1e30, 500.0, -500.0]).reshape(1, 1, 8), dtype)
    one, _ = store(np.ones((1, 1, 8)), dtype)
    r = mesa.mesa_causal_conv_backward(x.cuda(), torch.ones((1, 8), device="cuda"), one.cuda())
    y = mesa.mesa_causal_conv(x.cuda(), torch.ones((1, 8), device="cuda"))
    torch.cuda.synchronize()
    on = xf > 0
    assert np.array_equal(y.double().cpu().numpy(), np.where(on, xf, 0.0))
    assert np.array_equal(r["grad_x"].double().cpu().numpy(), np.where(on, 1.0, 0.0))
    assert np.array_equal(r["grad_w"].double().cpu().numpy()[0], np.where(on, xf, 0.0)[0, 0])
