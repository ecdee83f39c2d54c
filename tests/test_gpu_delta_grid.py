"""A step of more sequences than 2^32 / 8192 heads of 128 x 128: its launch has
an eighth of 2^32 threads, its states 40 GiB."""
import pytest

from tests.test_gpu_delta import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def test_step_of_many_sequences():
    import torch
    from test_regression_amd import mesa
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free memory")
    N, H, d = 40000, 16, 128
    say("case delta step", (N, H, d))
    gen = torch.Generator(device="cuda").manual_seed(3)
    one = lambda *s: torch.randn(N, H, *s, device="cuda", generator=gen)  # noqa: E731
    q, k, v = (one(d).mul_(0.088).bfloat16() for _ in range(3))
    gamma, beta = (one().sigmoid() for _ in range(2))
    S = torch.full((N, H, d, d), 0.25, device="cuda")
    S[:2], S[-2:] = (torch.randn(2, H, d, d, device="cuda", generator=gen) for _ in range(2))
    ends = [torch.cat([x[:2], x[-2:]]).contiguous() for x in (q, k, v, gamma, beta, S)]
    out = mesa.mesa_delta_step(q, k, v, gamma, beta, S)
    o = mesa.mesa_delta_step(*ends)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([out[:2], out[-2:]]), o)
    assert torch.equal(torch.cat([S[:2], S[-2:]]), ends[-1])
