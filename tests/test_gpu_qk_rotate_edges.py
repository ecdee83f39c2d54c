"""The rotation of queries and keys at its edges: positions up to 2^50, and features
beyond the rotated ones, which stay what they are.

Bounds, relative L2, as in tests/test_gpu_qk_rotate.py: 32 roundings of 2^-24, at any
of them.  The turn count p f / 2 pi is a product of a whole number
and two rounded ones; carried as a pair of float64 values it is off by 2^-100 of
itself, and by 2^-53 of what is left of a turn.  The reference's angles are exact
rationals: the frequencies are float64 numbers, 2 pi is taken to 60 digits."""
import sys
from fractions import Fraction

import numpy as np
import pytest

from tests.ssm_helpers import near, store

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def exact_angles(freqs, pos):
    """p f less whole turns, [T, pairs]: reduced exactly, then rounded to float64."""
    return np.array([[float((Fraction(int(p)) * Fraction(float(f))) % TWO_PI) for f in freqs] for p in pos])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("base", [0, 1 << 27, 1 << 33, -(1 << 36), 1 << 40, -(1 << 40), 1 << 49, 100000 - (1 << 50)])
def test_far_positions(base, inter):
    import torch
    from test_regression_amd import mesa
    say("case far", base, inter)
    d = 64
    rng = np.random.default_rng(3)
    x, xf = store(rng.standard_normal((1, 2, 6, d)), "f32")
    pos = base + np.array([0, 1, 5, 1000, 4097, 99991])
    freqs, _ = mesa.mesa_rotary_frequencies(d)
    y, _ = mesa.mesa_qk_rotate(x.cuda(), None, freqs, torch.from_numpy(pos[None]).cuda(), norm=False, interleaved=inter)
    counted, _ = mesa.mesa_qk_rotate(x.cuda()[:, :, :2].contiguous(), None, freqs, norm=False, interleaved=inter, position0=base)
    back = mesa.mesa_qk_rotate_backward(x.cuda(), None, y, None, freqs, torch.from_numpy(pos[None]).cuda(), norm=False,
                                        interleaved=inter)["grad_q"]
    torch.cuda.synchronize()
    ang = exact_angles(freqs.cpu().numpy(), pos)
    cos, sin = np.cos(ang), np.sin(ang)
    a, b = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    ref = np.empty_like(xf)
    ref[..., a], ref[..., b] = xf[..., a] * cos - xf[..., b] * sin, xf[..., b] * cos + xf[..., a] * sin
    # token by token, so that one position's error does not vanish in the others'
    for t in range(6):
        near(y[:, :, t], ref[:, :, t], 32 * U, what=(base, t))
    assert torch.equal(counted, y[:, :, :2])
    near(back, xf, 64 * U)   # the rotation and its transpose


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(32, 16), (64, 48), (128, 32)])
def test_features_past_the_rotation_stay(d, rot, inter, dtype):
    """Without a norm, features rot and up are the input's to the bit, infinities, NaN and
    the largest values too, and leave their neighbours alone; so are their gradients."""
    import torch
    from test_regression_amd import mesa
    say("case past the rotation", (d, rot, inter, dtype))
    x, _ = store(np.random.default_rng(d).standard_normal((2, 3, 5, d)), dtype)
    x = x.cuda()
    special = torch.tensor([float("inf"), float("-inf"), float("nan"), torch.finfo(x.dtype).min], device="cuda").to(x.dtype)
    plain = x.clone()
    x[..., rot + 1::4] = special[torch.arange(x[..., rot + 1::4].numel(), device="cuda") % 4].view_as(x[..., rot + 1::4])
    freqs, _ = mesa.mesa_rotary_frequencies(rot)
    kw = dict(norm=False, interleaved=inter, position0=100, amplitude=1.5)
    y, _ = mesa.mesa_qk_rotate(x, None, freqs, **kw)
    g = mesa.mesa_qk_rotate_backward(x, None, x, None, freqs, **kw)["grad_q"]
    yp, _ = mesa.mesa_qk_rotate(plain, None, freqs, **kw)
    gp = mesa.mesa_qk_rotate_backward(plain, None, plain, None, freqs, **kw)["grad_q"]
    torch.cuda.synchronize()
    for got, clean in ((y, yp), (g, gp)):
        want = torch.cat([clean[..., :rot], x[..., rot:]], -1)
        nan = want.isnan()
        assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want[~nan])


def test_weight_gradients_of_many_tokens():
    """Equal terms of which a float32 sum of 256 loses just under half a last place with
    every addition from 128 on: 2^25 tokens of one head at position 0, where the rotation
    is the identity, with rows of ones, whose norm is exactly one.  A lane adds 16 terms in
    float32, workgroups and lanes are joined in float64 but for batches of eight: below 32
    roundings of 2^-24."""
    import torch
    from test_regression_amd import mesa
    say("case many tokens")
    T, d = 1 << 25, 16
    term = 1 + 0.49 * 2.0 ** -16 + 2.0 ** -23
    term = float(np.float32(term))
    x = torch.ones((1, 1, 1, d), device="cuda").expand(1, 1, T, d)
    dy = torch.full((1, 1, T, d), term, device="cuda")
    freqs, _ = mesa.mesa_rotary_frequencies(16)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    r = mesa.mesa_qk_rotate_backward(x, None, dy, None, freqs, pos, torch.ones(d, device="cuda"), eps=2.0 ** -40)
    torch.cuda.synchronize()
    got = r["grad_wq"].double().cpu().numpy()
    assert np.abs(got - T * term).max() <= 32 * U * T * term, (got - T * term) / (T * term) / U


@pytest.mark.parametrize("inter", [False, True])
def test_positions_without_an_angle(inter):
    """Positions that float64 does not hold, such as a padded batch may leave, turn by some
    angle: rows stay finite and keep their size to the polynomials' error at pi / 2."""
    import torch
    from test_regression_amd import mesa
    say("case no angle", inter)
    ends = torch.tensor([-(1 << 63), (1 << 63) - 1, 1 << 62, -(1 << 55) + 12345, (1 << 52) + 1, -(1 << 51) - 3], device="cuda")
    x = torch.randn((1, 2, 6, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    freqs, _ = mesa.mesa_rotary_frequencies(64)
    y, _ = mesa.mesa_qk_rotate(x, None, freqs, ends, norm=False, interleaved=inter)
    g = mesa.mesa_qk_rotate_backward(x, None, x, None, freqs, ends, norm=False, interleaved=inter)["grad_q"]
    torch.cuda.synchronize()
    for r in (y, g):
        # cos^2 + sin^2 of the polynomials at 1.6 is off by 1.6^11 / 11! and 1.6^12 / 12! of about one: below 2^-16
        assert bool(((r.norm(dim=-1) / x.norm(dim=-1) - 1).abs() <= 2.0 ** -16).all())
