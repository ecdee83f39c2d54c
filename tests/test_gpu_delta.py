"""The gated delta rule on the GPU (mesa_delta_forward, mesa_delta_step)
against its token-by-token float64 form, at the sizes where a chunked kernel
can go wrong.  The bounds are derived in tests/delta_helpers.py."""
import sys

import numpy as np
import pytest

from tests.delta_helpers import F32, delta_inputs, delta_ref, rel, tol

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
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def forward(t, **kw):
    import torch
    from test_regression_amd import mesa
    d = dev(t)
    out, final = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], return_final=True, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), final.double().cpu().numpy()


def check(t, f, dtype):
    o, S = forward(t)
    ro, rS = delta_ref(f)
    eo, eS = rel(o, ro), rel(S, rS)
    say(f"  rel_l2 out={eo:.2e} final={eS:.2e}")
    assert eo <= tol(dtype) and eS <= F32
    return o, S


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 15, 64, 65, 130, 300])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 32), (128, 128), (64, 256), (128, 16)])
def test_delta_forward_shapes(dk, dv, T, dtype):
    seed = 100 + dk + dv + T
    say("case delta", dict(dk=dk, dv=dv, T=T, dtype=dtype, seed=seed))
    check(*delta_inputs(seed, 2, 2, 2, T, dk, dv, dtype, start=T % 2 == 0), dtype)


@pytest.mark.parametrize("B,Hk,H,T", [(1, 1, 1, 77), (1, 1, 3, 200), (3, 2, 6, 129), (2, 5, 5, 64), (1, 9, 9, 33)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_forward_heads(B, Hk, H, T, dtype):
    say("case delta heads", (B, Hk, H, T, dtype))
    check(*delta_inputs(7 + T, B, Hk, H, T, 64, 128, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_forward_long(dtype):
    say("case delta long", dtype)
    check(*delta_inputs(11, 1, 2, 2, 2000, 128, 64, dtype, lo=0.97), dtype)


# Long sequences of few heads are passed over in segments at once (from about
# 30 chunks on): ragged last segments, odd head counts, every width.
LONG = [(1, 1, 1, 2100, 16, 16), (1, 1, 3, 2500, 32, 64), (1, 2, 2, 4160, 64, 128), (1, 1, 1, 2300, 128, 256),
        (2, 1, 1, 8229, 16, 32), (1, 3, 3, 3000, 128, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv", LONG)
def test_delta_forward_segments(B, Hk, H, T, dk, dv, dtype):
    say("case delta segments", (B, Hk, H, T, dk, dv, dtype))
    check(*delta_inputs(13 + T, B, Hk, H, T, dk, dv, dtype, start=T % 2 == 0, lo=0.97), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["strong", "none", "full", "still", "same_keys", "orthogonal", "tiny", "huge", "zeros",
                                  "reset"])
def test_delta_forward_hard_inputs(what, dtype):
    import torch
    say("case delta hard", what, dtype)
    t, f = delta_inputs(23, 1, 2, 2, 200, 64, 64, dtype)

    def put(name, fn):
        x = t[name].clone()
        fn(x)
        t[name], f[name] = x, x.double().numpy()
    if what == "strong":      # decays that underflow over a chunk
        put("gamma", lambda x: x.copy_(torch.rand_like(x) * 0.1 + 1e-4))
    elif what == "none":      # no decay, full writes
        put("gamma", lambda x: x.fill_(1.0))
        put("beta", lambda x: x.fill_(1.0))
    elif what == "full":
        put("beta", lambda x: x.fill_(1.0))
    elif what == "still":     # nothing is written: the state only decays
        put("beta", lambda x: x.zero_())
    elif what == "same_keys":  # every token rewrites the same entry
        put("beta", lambda x: x.fill_(1.0))
        put("k", lambda x: x.copy_(x[:, :, :1].expand_as(x).clone()))
    elif what == "orthogonal":
        put("k", lambda x: x.copy_(torch.eye(64)[torch.arange(200) % 64].expand_as(x)))
    elif what == "tiny":
        for n in ("v", "state"):
            put(n, lambda x: x.mul_(2.0 ** -60))
    elif what == "huge":
        for n in ("v", "state"):
            put(n, lambda x: x.mul_(2.0 ** 60))
    elif what == "zeros":     # rows of zeros among the keys and queries
        put("k", lambda x: x[:, :, ::3].zero_())
        put("q", lambda x: x[:, :, 1::3].zero_())
    elif what == "reset":     # a gate of 0 forgets everything before it
        put("gamma", lambda x: x.index_fill_(2, torch.tensor([0, 70, 71, 128]), 0.0))
    o, S = check(t, f, dtype)
    if what == "reset":
        # what follows the reset at 128 is the rule from nothing
        t2 = {n: (x[:, :, 128:].contiguous() if x is not None and n != "state" else None) for n, x in t.items()}
        o2, S2 = forward(t2)
        assert rel(o[:, :, 128:], o2) <= tol(dtype) and rel(S, S2) <= F32


def test_delta_forward_bf16_rounds_the_float_result():
    """The bf16 call's outputs are the float32 call's on the same values within
    the documented 11-bit products and one rounding, element by element."""
    say("case delta bf16 against f32")
    t, _ = delta_inputs(31, 1, 2, 2, 256, 128, 128, "bf16")
    o, S = forward(t)
    o2, S2 = forward({n: None if x is None else x.float() for n, x in t.items()})
    assert rel(S, S2) <= F32
    # two products of 11-bit operands, each term off by at most 3 2^-12; a
    # row's terms sum to at most |q| |S| + ... < 8 times the largest output
    assert np.abs(o - o2).max() <= (2.0 ** -8 + 8 * 3 * 2.0 ** -12) * np.abs(o2).max()


def test_delta_pieces_equal_the_whole_and_padding_is_inert():
    import torch
    say("case delta pieces")
    t, f = delta_inputs(41, 2, 2, 4, 230, 64, 64, "f32")
    o, S = check(t, f, "f32")
    cut = lambda a, b: {n: x if n == "state" else x[:, :, a:b].contiguous() for n, x in t.items()}  # noqa: E731
    o1, S1 = forward(cut(0, 100))
    rest = cut(100, 230)
    rest["state"] = torch.from_numpy(S1).float()
    o2, S2 = forward(rest)
    assert rel(np.concatenate([o1, o2], 2), o) <= F32 and rel(S2, S) <= F32
    # padded behind the end with gate 1 and strength 0: the state stays
    pad = {n: x if n == "state" else torch.cat([x, x[:, :, :37]], 2) for n, x in t.items()}
    pad["gamma"][:, :, 230:] = 1.0
    pad["beta"][:, :, 230:] = 0.0
    op, Sp = forward(pad)
    assert rel(op[:, :, :230], o) <= F32 and rel(Sp, S) <= F32


def test_delta_forward_no_tokens_in_place_state_and_repeat():
    import torch
    from test_regression_amd import mesa
    say("case delta no tokens")
    t, f = delta_inputs(51, 1, 2, 2, 90, 32, 32, "bf16")
    d = dev(t)
    e = {n: x if n == "state" else x[:, :, :0].contiguous() for n, x in d.items()}
    out, S = mesa.mesa_delta_forward(e["q"], e["k"], e["v"], e["gamma"], e["beta"], d["state"], return_final=True)
    assert out.shape == (1, 2, 0, 32) and torch.equal(S, d["state"])
    _, S = mesa.mesa_delta_forward(e["q"], e["k"], e["v"], e["gamma"], e["beta"], return_final=True)
    assert bool((S == 0).all())
    # the final state over the initial one; the same call twice gives the same bits
    a = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], return_final=True)
    s = d["state"].clone()
    b = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], s, final_state=s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], s)


def test_delta_forward_writes_only_its_outputs():
    import torch
    from test_regression_amd import mesa
    say("case delta guards")
    t, _ = delta_inputs(61, 2, 1, 2, 70, 64, 32, "bf16")
    d = dev(t)
    big = torch.full((2 * 2 * 70 * 32 + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[128:128 + 2 * 2 * 70 * 32].view(2, 2, 70, 32)
    nbytes = mesa.mesa_delta_workspace_bytes(2, 2, 70, 64, 32, mesa.MESA_DTYPE_BF16)
    ws = torch.full((nbytes + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    r, _ = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], out=out,
                                   workspace=ws[256:256 + nbytes])
    torch.cuda.synchronize()
    ref, _ = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"])
    assert torch.equal(r, ref)
    assert bool((big[:128] == 7).all()) and bool((big[-128:] == 7).all())
    assert bool((ws[:256] == 0x5a).all()) and bool((ws[-256:] == 0x5a).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hk,H,dk,dv", [(1, 1, 1, 16, 16), (1, 4, 4, 64, 64), (3, 2, 6, 32, 128), (2, 3, 3, 128, 256),
                                          (5, 1, 2, 16, 32), (130, 16, 16, 128, 128), (7, 1, 1, 64, 16)])
def test_delta_step(N, Hk, H, dk, dv, dtype):
    import torch
    from test_regression_amd import mesa
    say("case delta step", (N, Hk, H, dk, dv, dtype))
    t, f = delta_inputs(71 + N, N, Hk, H, 1, dk, dv, dtype)
    d = dev(t)
    one = {n: x if n == "state" else x[:, :, 0].contiguous() for n, x in d.items()}
    out = mesa.mesa_delta_step(one["q"], one["k"], one["v"], one["gamma"], one["beta"], one["state"])
    torch.cuda.synchronize()
    ro, rS = delta_ref(f)
    # sums of at most 128 float terms: 2 log2(128) + 4 roundings of 2^-24 each, twice
    bound = 36 * 2.0 ** -24
    assert rel(one["state"].double().cpu(), rS) <= bound
    assert rel(out.double().cpu(), ro[:, :, 0]) <= bound + (2.0 ** -8 if dtype == "bf16" else 0.0)


def test_prompt_then_tokens():
    """A prompt through the sequence call, then tokens one at a time on its final state."""
    import torch
    from test_regression_amd import mesa
    say("case delta prompt then tokens")
    t, f = delta_inputs(81, 2, 2, 4, 140, 64, 128, "f32")
    d = dev(t)
    p = {n: x if n == "state" else x[:, :, :128].contiguous() for n, x in d.items()}
    out, S = mesa.mesa_delta_forward(p["q"], p["k"], p["v"], p["gamma"], p["beta"], p["state"], return_final=True)
    outs = [out]
    for i in range(128, 140):
        one = {n: d[n][:, :, i].contiguous() for n in ("q", "k", "v", "gamma", "beta")}
        outs.append(mesa.mesa_delta_step(one["q"], one["k"], one["v"], one["gamma"], one["beta"], S)[:, :, None])
    torch.cuda.synchronize()
    ro, rS = delta_ref(f)
    assert rel(torch.cat(outs, 2).double().cpu(), ro) <= F32 and rel(S.double().cpu(), rS) <= F32


def backward_errors(t, f, dtype, seed, with_final=True):
    import torch
    from test_regression_amd import mesa
    rng = np.random.default_rng(seed)
    d = dev(t)
    go = torch.from_numpy(rng.standard_normal(t["v"].shape)).to(t["v"].dtype)
    shape = f["state"].shape
    gf = torch.from_numpy(0.3 * rng.standard_normal(shape)).float() if with_final else None
    g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go.cuda(), d["state"],
                                 grad_final=None if gf is None else gf.cuda())
    torch.cuda.synchronize()
    _, _, ref = delta_ref(f, go.double().numpy(), None if gf is None else gf.double().numpy())
    assert (g["grad_state"] is None) == (t["state"] is None)
    got = {n: x.double().cpu().numpy() for n, x in g.items() if x is not None}
    return {n: rel(x, ref[n]) for n, x in got.items()}, got, ref


# Gradients: the backward's chain is the forward's and its own, twice the
# products and inverses of the bound in delta_helpers; the roundings of
# bfloat16 gradients come on top.
GRAD_F32 = 2 * F32


def grad_tol(name, dtype):
    return GRAD_F32 + (2.0 ** -8 if dtype == "bf16" and name in ("grad_q", "grad_k", "grad_v") else 0.0)


def check_grads(t, f, dtype, seed, with_final=True):
    errs, got, ref = backward_errors(t, f, dtype, seed, with_final)
    say("  " + " ".join(f"{n[5:]}={e:.1e}" for n, e in errs.items()))
    for n, e in errs.items():
        assert e <= grad_tol(n, dtype), n
    return got, ref


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 15, 64, 65, 130, 300])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 32), (128, 128), (64, 256), (128, 16)])
def test_delta_backward_shapes(dk, dv, T, dtype):
    seed = 300 + dk + dv + T
    say("case delta backward", dict(dk=dk, dv=dv, T=T, dtype=dtype, seed=seed))
    check_grads(*delta_inputs(seed, 2, 2, 2, T, dk, dv, dtype, start=T % 2 == 0), dtype, seed, T % 3 == 0)


@pytest.mark.parametrize("B,Hk,H,T", [(1, 1, 1, 77), (1, 1, 3, 200), (3, 2, 6, 129), (1, 9, 9, 33)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_backward_heads(B, Hk, H, T, dtype):
    say("case delta backward heads", (B, Hk, H, T, dtype))
    check_grads(*delta_inputs(17 + T, B, Hk, H, T, 64, 128, dtype), dtype, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,H,T,dk,dv", LONG)
def test_delta_backward_segments(B, Hk, H, T, dk, dv, dtype):
    say("case delta backward segments", (B, Hk, H, T, dk, dv, dtype))
    check_grads(*delta_inputs(19 + T, B, Hk, H, T, dk, dv, dtype, start=T % 2 == 0, lo=0.97), dtype, T, T % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["strong", "none", "still", "same_keys", "zeros", "reset", "silent"])
def test_delta_backward_hard_inputs(what, dtype):
    import torch
    say("case delta backward hard", what, dtype)
    t, f = delta_inputs(29, 1, 2, 2, 200, 64, 64, dtype)

    def put(name, fn):
        x = t[name].clone()
        fn(x)
        t[name], f[name] = x, x.double().numpy()
    if what == "strong":
        put("gamma", lambda x: x.copy_(torch.rand_like(x) * 0.1 + 1e-2))
    elif what == "none":
        put("gamma", lambda x: x.fill_(1.0))
        put("beta", lambda x: x.fill_(1.0))
    elif what == "still":     # strength 0: its own gradient does not vanish
        put("beta", lambda x: x[:, :, ::2].zero_())
    elif what == "same_keys":
        put("beta", lambda x: x.fill_(0.9))
        put("k", lambda x: x.copy_(x[:, :, :1].expand_as(x).clone()))
    elif what == "zeros":
        put("k", lambda x: x[:, :, ::3].zero_())
        put("q", lambda x: x[:, :, 1::3].zero_())
    elif what == "reset":
        put("gamma", lambda x: x.index_fill_(2, torch.tensor([70, 128]), 0.0))
    elif what == "silent":    # values and start of zeros: only the values' gradients remain
        put("v", lambda x: x.zero_())
        put("state", lambda x: x.zero_())
    if what in ("reset", "silent"):
        errs, got, ref = backward_errors(t, f, dtype, 5)
        if what == "reset":
            at = np.array([70, 128])
            assert (got["grad_gamma"][:, :, at] == 0).all()
            got["grad_gamma"][:, :, at] = ref["grad_gamma"][:, :, at] = 0
            assert rel(got["grad_gamma"], ref["grad_gamma"]) <= GRAD_F32
            assert all(e <= grad_tol(n, dtype) for n, e in errs.items() if n != "grad_gamma"), errs
        else:
            for n in ("grad_q", "grad_k", "grad_gamma", "grad_beta"):
                assert (got[n] == 0).all(), n
            assert errs["grad_v"] <= grad_tol("grad_v", dtype) and errs["grad_state"] <= GRAD_F32
    else:
        check_grads(t, f, dtype, 5)


def test_delta_backward_against_differences():
    """The gradients of the GPU's own float32 forward, by central differences of
    a projection of it in the float64 definition."""
    say("case delta backward differences")
    t, f = delta_inputs(91, 1, 1, 2, 70, 16, 16, "f32")
    got, ref = check_grads(t, f, "f32", 91)
    rng = np.random.default_rng(91)
    go = rng.standard_normal(t["v"].shape).astype(np.float32).astype(np.float64)
    gf = (0.3 * rng.standard_normal(f["state"].shape)).astype(np.float32).astype(np.float64)
    for n in ("q", "k", "v", "gamma", "beta", "state"):
        d = rng.standard_normal(f[n].shape)
        h = 1e-5
        vals = []
        for s in (h, -h):
            o, S = delta_ref({**f, n: f[n] + s * d})
            vals.append((o * go).sum() + (S * gf).sum())
        num, ana = (vals[0] - vals[1]) / (2 * h), float((got["grad_" + n] * d).sum())
        # truncation h^2 and cancellation 1e-16 / h of sums of some thousand terms
        assert abs(num - ana) <= 1e-4 * max(1.0, np.linalg.norm(ref["grad_" + n]) * np.linalg.norm(d) / np.sqrt(d.size))


def test_delta_backward_no_tokens_repeat_and_in_place():
    import torch
    from test_regression_amd import mesa
    say("case delta backward no tokens, repeat")
    t, _ = delta_inputs(95, 1, 2, 4, 150, 32, 32, "bf16")
    d = dev(t)
    go, gf = torch.randn_like(d["v"]), torch.randn_like(d["state"])
    args = (d["q"], d["k"], d["v"], d["gamma"], d["beta"], go, d["state"])
    a = mesa.mesa_delta_backward(*args, grad_final=gf)
    b = mesa.mesa_delta_backward(*args, grad_final=gf)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    e = [x[:, :, :0].contiguous() for x in args[:6]]
    g = mesa.mesa_delta_backward(*e, d["state"], grad_final=gf)
    assert torch.equal(g["grad_state"], gf) and g["grad_q"].shape == (1, 2, 0, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_keys_of_mixed_sizes(dtype):
    """Keys and queries of very different lengths in a chunk, and padded tokens
    whose keys are longer than any that write."""
    import torch
    say("case delta mixed sizes", dtype)
    t, f = delta_inputs(97, 1, 2, 2, 200, 64, 64, dtype)
    size = 2.0 ** -(torch.arange(200) % 9).float()[:, None]
    idle = torch.arange(200) % 7 == 3
    size[idle] = 2.0 ** 8
    for n in ("q", "k"):
        t[n] = (t[n].float() * size).to(t[n].dtype)      # powers of two: exact
    t["beta"][:, :, idle] = 0.0
    f.update({n: t[n].double().numpy() for n in ("q", "k", "beta")})
    # q of 2^8 would drown the others' outputs: those tokens are read apart
    o, S = forward(t)
    ro, rS = delta_ref(f)
    on = ~idle.numpy()
    assert rel(S, rS) <= F32 and rel(o[:, :, on], ro[:, :, on]) <= tol(dtype) and rel(o[:, :, ~on], ro[:, :, ~on]) <= tol(dtype)
    t["q"][:, :, idle] = 0.0
    f["q"] = t["q"].double().numpy()
    errs, got, ref = backward_errors(t, f, dtype, 97)
    # the gradients of the idle tokens' strengths come from keys 2^8 long, and
    # theirs and the others' are off in proportion to their own
    for n in ("grad_q", "grad_k", "grad_v", "grad_gamma", "grad_state"):
        assert errs[n] <= grad_tol(n, dtype), (n, errs)
    for m in (on, ~on):
        assert rel(got["grad_beta"][:, :, m], ref["grad_beta"][:, :, m]) <= GRAD_F32


@pytest.mark.parametrize("what", ["q", "k", "v", "gamma", "beta"])
def test_delta_nan_stays_in_its_head(what):
    import torch
    from test_regression_amd import mesa
    say("case delta nan", what)
    t, _ = delta_inputs(101, 2, 2, 2, 200, 64, 64, "f32")
    d = dev(t)
    go, gf = torch.randn_like(d["v"]), torch.randn_like(d["state"])
    run = lambda: (mesa.mesa_delta_forward(*d.values(), return_final=True),  # noqa: E731
                   mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go, d["state"], grad_final=gf))
    (o, S), g = run()
    d[what][1, 0, 100] = float("nan")
    (o2, S2), g2 = run()
    torch.cuda.synchronize()
    pick = lambda x: torch.cat([x[0], x[1, 1:]])  # noqa: E731
    assert torch.equal(pick(o), pick(o2)) and torch.equal(pick(S), pick(S2))
    for n in g:
        assert torch.equal(pick(g[n]), pick(g2[n])), n
    # chunks before the token's keep their outputs, and it does not go unseen
    assert torch.equal(o[1, 0, :64], o2[1, 0, :64])
    assert bool(o2[1, 0, 100].isnan().all())
    if what != "q":
        assert bool(o2[1, 0, 128:].isnan().all()) and bool(S2[1, 0].isnan().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_segments_state_in_place(dtype):
    """The final state over the initial one where segments run at once."""
    import torch
    from test_regression_amd import mesa
    say("case delta segments in place", dtype)
    t, _ = delta_inputs(103, 1, 1, 2, 4100, 64, 64, dtype, lo=0.97)
    d = dev(t)
    a = mesa.mesa_delta_forward(*d.values(), return_final=True)
    s = d["state"].clone()
    b = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], s, final_state=s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], s)


def test_delta_more_than_2_31_elements():
    """The last row of a batch whose tensors pass 2^31 elements and 2^32 bytes."""
    import torch
    from test_regression_amd import mesa
    B, H, T, d = 258, 16, 4096, 128
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free memory")
    say("case delta large", (B, H, T, d))
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda: torch.randn(B, H, T, d, dtype=torch.bfloat16, device="cuda", generator=gen)  # noqa: E731
    q, k, v = new().mul_(0.088), new().mul_(0.088), new()
    gamma = torch.rand(B, H, T, device="cuda", generator=gen).mul_(0.2).add_(0.8)
    beta = torch.rand(B, H, T, device="cuda", generator=gen)
    last = [x[-1:].contiguous() for x in (q, k, v, gamma, beta)]
    out, S = mesa.mesa_delta_forward(q, k, v, gamma, beta, return_final=True)
    o1, S1 = mesa.mesa_delta_forward(*last, return_final=True)
    say("  forward")
    assert torch.equal(out[-1:], o1) or rel(out[-1:].double().cpu(), o1.double().cpu()) <= 2 * tol("bf16")
    assert rel(S[-1:].double().cpu(), S1.double().cpu()) <= 2 * F32
    g = mesa.mesa_delta_backward(q, k, v, gamma, beta, out)
    g1 = mesa.mesa_delta_backward(*last, out[-1:].contiguous())
    torch.cuda.synchronize()
    say("  backward")
    for n in g:
        if g[n] is not None:
            assert torch.equal(g[n][-1:], g1[n]), n
    del g, g1, out, q, k, v
    torch.cuda.empty_cache()
    # the step over states of more than 2^32 bytes
    N = 4200
    S = torch.randn(N, H, d, d, device="cuda", generator=gen)
    one = lambda: torch.randn(N, H, d, dtype=torch.bfloat16, device="cuda", generator=gen).mul_(0.088)  # noqa: E731
    q, k, v, ga = one(), one(), one(), torch.rand(N, H, device="cuda", generator=gen)
    S1 = S[-2:].clone()
    o = mesa.mesa_delta_step(q, k, v, ga, ga, S)
    o1 = mesa.mesa_delta_step(*(x[-2:].contiguous() for x in (q, k, v, ga, ga)), S1)
    torch.cuda.synchronize()
    assert torch.equal(o[-2:], o1) and torch.equal(S[-2:], S1)
