"""How many bits the delta rule's bfloat16 outputs keep before their rounding:
outputs in which large terms cancel.

In a chunk, o_t = G_t q_t.S + sum_j P_tj b_j e_j over the tokens j <= t, with S
the chunk's start state, P_tj = D_tj q_t.k_j and e_j = v_j - g_j S_{j-1} k_j.
The last token's value is chosen, per column, so that its own term takes away
all others up to the rounding of that value to bfloat16: what is left is some
2^-9 of the terms, and an error of the terms is seen in full.

Bound: the output's rounding, 2^-8 of it; 2^-14 of the terms P_tj e_j (P's
second part, a byte, is off by 2^-3 of at most 2^-11); and 1.5e-5
(tests/delta_helpers.py) of everything summed to 22 bits.  A dot product's
error is made of its products' errors, so it is held to the sum of their
magnitudes, |q_i| |S_i| and |k_i| |S_i|, and not to what is left of that sum:
a column's q.S may be small by chance where its products are not.  Terms of 11
bits would be off by up to 2^-12 for each of their two factors.
"""
import numpy as np
import pytest

from tests.delta_helpers import F32, delta_inputs, delta_ref, store
from tests.test_gpu_delta import forward, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (16, 32)])
@pytest.mark.parametrize("T,start", [(1, True), (2, False), (40, True), (130, True), (4100, False)])
def test_cancelling_terms(T, start, dk, dv, dtype):
    say("case delta cancelling terms", (T, start, dk, dv, dtype))
    t, f = delta_inputs(401 + T + dk, 1, 2, 2, T, dk, dv, "bf16", start=start, lo=0.97)
    # the last query lies along its key, so that its token's own term can be large
    q = f["q"].copy()
    q[:, :, -1] = f["k"][:, :, -1] + 0.5 * q[:, :, -1]
    t["q"], f["q"] = store(q, "bf16")
    t["beta"][:, :, -1] = 0.9
    f["beta"] = t["beta"].double().numpy()

    def rest(to):   # up to token `to`: the state, each e_j and what it is summed of, the last chunk's start state
        S, e, d, c0 = f["state"], [], [], (T - 1) // 64 * 64
        for j in range(to):
            if j == c0:
                S0 = S
            g, b = f["gamma"][:, :, j, None, None], f["beta"][:, :, j, None, None]
            k = f["k"][:, :, j, None, :]
            S = g * S
            err = f["v"][:, :, j, :, None] - (S * k).sum(-1, keepdims=True)
            e.append(err[..., 0])
            d.append(np.abs(S * k).sum(-1) + np.abs(f["v"][:, :, j]))
            S = S + b * err * k
        if to == c0:
            S0 = S
        return S, e, d, S0, c0

    S, e, d, S0, c0 = rest(T - 1)
    qt, kt = f["q"][:, :, -1, None, :], f["k"][:, :, -1, None, :]
    g, b = f["gamma"][:, :, -1, None], f["beta"][:, :, -1, None]
    P = b * (qt * kt).sum(-1)
    Sq, Sk = g * (S * qt).sum(-1), g * (S * kt).sum(-1)
    v = f["v"].copy()
    v[:, :, -1] = Sk - Sq / P          # o = g S q + P (v - g S k) = 0
    t["v"], f["v"] = store(v, "bf16")
    if dtype == "f32":
        t = {n: None if x is None else x.float() for n, x in t.items()}
    # the terms' magnitudes, and those of the products they are summed of
    L = np.cumsum(np.log(f["gamma"][:, :, c0:]), -1)
    G = np.exp(L[..., -1, None])
    terms, sums = np.zeros_like(Sq), G * np.abs(S0 * qt).sum(-1)
    own = np.abs(f["v"][:, :, -1] - Sk), g * np.abs(S * kt).sum(-1) + np.abs(f["v"][:, :, -1])
    for i, (ej, dj) in enumerate([*zip(np.abs(e[c0:]), d[c0:]), own]):
        Pj = f["beta"][:, :, c0 + i] * (np.abs(qt[:, :, 0]) * np.abs(f["k"][:, :, c0 + i])).sum(-1)
        Pj = (np.exp(L[..., -1] - L[..., i]) * Pj)[..., None]
        terms, sums = terms + Pj * ej, sums + Pj * dj
    large = G * np.abs((S0 * qt).sum(-1)) + np.abs(P) * own[0]
    o, _ = forward(t)
    ro, _ = delta_ref(f)
    off, ref = np.abs(o - ro)[:, :, -1], np.abs(ro[:, :, -1])
    say(f"  left {np.linalg.norm(ref) / np.linalg.norm(large):.1e} off {np.linalg.norm(off) / np.linalg.norm(large):.1e} of the large terms")
    assert np.linalg.norm(ref) < 2.0 ** -7 * np.linalg.norm(large)
    bound = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * ref + (2.0 ** -14 if dtype == "bf16" else 0.0) * terms + F32 * sums
    assert (off <= bound).all(), (off / bound).max()
