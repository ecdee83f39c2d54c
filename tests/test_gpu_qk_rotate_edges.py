"""The rotation of queries and keys at its edges: features beyond the rotated ones, which
stay what they are."""
import sys

import numpy as np
import pytest

from tests.ssm_helpers import store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


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
