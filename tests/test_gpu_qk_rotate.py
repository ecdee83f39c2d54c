"""The norm and rotation of queries and keys on the GPU (mesa_qk_rotate and its
gradients) against float64 with angles in long double (tests/ssm_helpers.py).

Bounds, relative L2.  Cosine and sine come from an angle of at most pi / 4 rounded to
float32 (2^-24 of it) after a reduction in float64, and polynomials of six terms: below
8 roundings of 2^-24; a norm's sum of up to 256 squares over lanes, its root and two
products: below 16; the rotation: 3.  So 32 2^-24.  The norm's gradient adds a second
sum and three products and is a difference: 64 2^-24 of its terms.  The weights'
gradients are sums over up to 2^12 rows in fixed order: 96 2^-24 of the terms they sum.
bfloat16 results add 2^-8.  At positions near 2^40 float64 holds a turn to 2^-53 of
2^40 / 6: 2^-15 of a radian would be lost beyond 2^38 turns; the test's turns stay
below 2^38, where the product's rounding is 2^-15 2^-1: the bound there is 2^-14."""
import sys

import numpy as np
import pytest

from tests.ssm_helpers import near, rotate_ref, store

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
OUT = {"f32": 32 * U, "bf16": 2.0 ** -8 + 32 * U}
GRAD = {"f32": 64 * U, "bf16": 2.0 ** -8 + 64 * U}
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


SIZES = [(1, 1, 1, 1, 16, 16), (2, 3, 1, 5, 32, 16), (1, 16, 4, 1, 128, 128), (3, 5, 5, 17, 64, 48), (2, 2, 2, 100, 256, 256),
         (1, 7, 1, 300, 16, 16), (5, 1, 0, 8, 128, 64), (1, 4, 2, 1500, 128, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,T,d,rot", SIZES)
def test_rotate(B, Hq, Hk, T, d, rot, inter, dtype):
    import torch
    from test_regression_amd import mesa
    say("case rotate", (B, Hq, Hk, T, d, rot, inter, dtype))
    rng = np.random.default_rng(B + T + d + rot)
    q, qf = store(rng.standard_normal((B, Hq, T, d)), dtype)
    k, kf = store(rng.standard_normal((B, Hk, T, d)), dtype) if Hk else (None, None)
    gq, gqf = store(rng.standard_normal((B, Hq, T, d)), dtype)
    gk, gkf = store(rng.standard_normal((B, Hk, T, d)), dtype) if Hk else (None, None)
    freqs, amp = mesa.mesa_rotary_frequencies(rot, 10000.0)
    ff = freqs.cpu().numpy()
    for norm, weights, where in ((True, True, "rows"), (False, False, "shared"), (True, False, "counted")):
        wq, wqf = store(1 + 0.3 * rng.standard_normal(d), "f32") if weights else (None, None)
        wk, wkf = store(1 + 0.3 * rng.standard_normal(d), "f32") if weights and Hk else (None, None)
        first = rng.integers(0, 200000, (B, 1)) if where == "rows" else np.full((B, 1), 777)
        pos = first + np.arange(T)
        p = torch.from_numpy(pos[0] if where == "shared" else pos).cuda()
        kw = dict(norm=norm, eps=1e-5, interleaved=inter, amplitude=1.25)
        kw.update(positions=None, position0=777) if where == "counted" else kw.update(positions=p)
        yq, yk = mesa.mesa_qk_rotate(c(q), c(k), freqs, wq=c(wq), wk=c(wk), **kw)
        r = mesa.mesa_qk_rotate_backward(c(q), c(k), c(gq), c(gk), freqs, wq=c(wq), wk=c(wk), **kw)
        torch.cuda.synchronize()
        for y, x, w, dy, name in ((yq, qf, wqf, gqf, "q"), (yk, kf, wkf, gkf, "k")):
            if x is None:
                assert y is None and r["grad_k"] is None and r["grad_wk"] is None
                continue
            ry, rdx, rdw, tx, tw = rotate_ref(x, ff, pos, w, norm, 1e-5, inter, 1.25, dy)
            near(y, ry, OUT[dtype], what="y" + name)
            near(r["grad_" + name], rdx, GRAD[dtype], tx, what="grad_" + name)
            if weights:
                near(r["grad_w" + name], rdw, SUMS, tw, what="grad_w" + name)
            else:
                assert r["grad_w" + name] is None


def test_far_positions():
    import torch
    from test_regression_amd import mesa
    say("case far positions")
    x, xf = store(np.random.default_rng(0).standard_normal((1, 2, 6, 64)), "f32")
    freqs, _ = mesa.mesa_rotary_frequencies(64)
    for base, bound in ((0, 32 * U), (1 << 20, 32 * U), (1 << 27, 32 * U), (-(1 << 27), 32 * U), (1 << 40, 2.0 ** -14)):
        pos = base + np.array([[0, 1, 5, 1000, 4097, 99991]])
        y, _ = mesa.mesa_qk_rotate(x.cuda(), None, freqs, torch.from_numpy(pos).cuda(), norm=False)
        torch.cuda.synchronize()
        near(y, rotate_ref(xf, freqs.cpu().numpy(), pos, norm=False), bound, what=base)


@pytest.mark.parametrize("inter", [False, True])
def test_views_rows_of_zeros_and_the_way_back(inter):
    """Queries and keys as slices of projection rows with an odd offset, gradients into
    slices; without a norm the gradients of the rotation undo it."""
    import torch
    from test_regression_amd import mesa
    say("case rotate views", inter)
    torch.manual_seed(0)
    B, T, Hq, Hk, d = 2, 37, 6, 2, 64
    rows = torch.randn((B, T, (Hq + Hk) * d + 3), device="cuda").to(torch.bfloat16)
    rows[0, 3] = 0
    cut = lambda r: (r[..., 1:1 + Hq * d].unflatten(-1, (Hq, d)).transpose(1, 2),  # noqa: E731
                     r[..., 1 + Hq * d:1 + (Hq + Hk) * d].unflatten(-1, (Hk, d)).transpose(1, 2))
    q, k = cut(rows)
    freqs, _ = mesa.mesa_rotary_frequencies(32)
    w = torch.rand(d, device="cuda")
    kw = dict(wq=w, wk=w + 1, interleaved=inter)
    yq, yk = mesa.mesa_qk_rotate(q, k, freqs, **kw)
    cq, ck = mesa.mesa_qk_rotate(q.contiguous(), k.contiguous(), freqs, **kw)
    grows = torch.full_like(rows, 5.0)
    gq, gk = cut(grows)
    r = mesa.mesa_qk_rotate_backward(q, k, yq, yk, freqs, grad_q=gq, grad_k=gk, **kw)
    r2 = mesa.mesa_qk_rotate_backward(q.contiguous(), k.contiguous(), yq, yk, freqs, **kw)
    torch.cuda.synchronize()
    assert torch.equal(yq, cq) and torch.equal(yk, ck) and all(torch.equal(r[n], r2[n]) for n in r)
    assert bool((yq[0, :, 3] == 0).all()) and bool(torch.isfinite(gq).all())
    assert bool((grows[..., 0] == 5).all()) and bool((grows[..., -2:] == 5).all())
    x = torch.randn((B, Hq, T, d), device="cuda")
    y, _ = mesa.mesa_qk_rotate(x, None, freqs, norm=False, interleaved=inter, position0=12345)
    b = mesa.mesa_qk_rotate_backward(x, None, y, None, freqs, norm=False, interleaved=inter, position0=12345)["grad_q"]
    torch.cuda.synchronize()
    near(b, x.double().cpu().numpy(), 32 * U)


def test_no_tokens():
    import torch
    from test_regression_amd import mesa
    freqs, _ = mesa.mesa_rotary_frequencies(16)
    z = torch.zeros((2, 3, 0, 16), device="cuda")
    w = torch.ones(16, device="cuda")
    y, _ = mesa.mesa_qk_rotate(z, None, freqs, wq=w)
    r = mesa.mesa_qk_rotate_backward(z, None, z, None, freqs, wq=w)
    torch.cuda.synchronize()
    assert y.shape == z.shape and bool((r["grad_wq"] == 0).all())
