"""The state space layer as it is used: rows of a projection through the causal
convolution, its slices as x, b and c, the norm and rotation of b and c, the scan, norm
and gate of the outputs, and all gradients back into the rows' gradient; a prompt and
its tokens; captured in a graph; on two streams at once.

Every operator is held to its float64 form on what the one before it gave, with its own
bound (tests/ssm_helpers.py and the operators' own tests)."""
import sys

import numpy as np
import pytest

from tests import test_gpu_causal_conv as conv_test, test_gpu_qk_rotate as rotate_test
from tests.ssm_helpers import F32, conv_ref, near, rotate_ref, ssm_inputs, ssm_ref, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    """The layer's parameters and sizes: rows of H dv values, Hk dk of b, Hk dk of c."""

    def __init__(self, mesa, seed, B, Hk, H, dk, dv, dtype, W=4):
        import torch
        self.mesa, self.Hk, self.H, self.dk, self.dv, self.W = mesa, Hk, H, dk, dv, W
        self.D = H * dv + 2 * Hk * dk
        self.type = torch.bfloat16 if dtype == "bf16" else torch.float32
        rng = np.random.default_rng(seed)
        p = dict(w=rng.standard_normal((W, self.D)) / 2, bias=0.1 * rng.standard_normal(self.D),
                 A=-np.exp(rng.uniform(-1.5, 2.5, H)), skip=rng.standard_normal(H), dt_bias=rng.uniform(-4, 0, H),
                 wc=1 + 0.2 * rng.standard_normal(dk), wb=1 + 0.2 * rng.standard_normal(dk),
                 norm=1 + 0.2 * rng.standard_normal((H, dv)))
        self.p, self.f = {}, {}
        for n, y in p.items():
            t, self.f[n] = store(y, "f32")
            self.p[n] = t.cuda()
        self.freqs, _ = mesa.mesa_rotary_frequencies(dk, 10000.0)

    def heads(self, rows):
        """x, b, c as views of rows [B, T, D]."""
        a, s = self.H * self.dv, self.Hk * self.dk
        cut = lambda i, n, d: rows[..., i:i + n].unflatten(-1, (-1, d)).transpose(1, 2)  # noqa: E731
        return cut(0, a, self.dv), cut(a, s, self.dk), cut(a + s, s, self.dk)

    def forward(self, rows, dt, gate, lens=None, hist=None, state=None, position0=0, ws=None):
        m, p = self.mesa, self.p
        r = {}
        r["y"], r["hist"] = m.mesa_causal_conv(rows, p["w"], p["bias"], hist, lens=lens, return_hist=True)
        r["x"], r["b"], r["c"] = self.heads(r["y"])
        r["rc"], r["rb"] = m.mesa_qk_rotate(r["c"], r["b"], self.freqs, wq=p["wc"], wk=p["wb"], position0=position0)
        r["o"], r["state"] = m.mesa_ssm_forward(r["x"], r["rb"], r["rc"], dt.transpose(1, 2), p["A"], p["skip"], p["dt_bias"], state,
                                                lens=lens, return_final=True, workspace=ws)
        r["n"] = m.mesa_gate_norm(r["o"], gate, p["norm"])
        return r

    def backward(self, r, rows, dt, gate, grad, lens=None, hist=None, state=None, position0=0, ws=None):
        import torch
        m, p = self.mesa, self.p
        g = dict(gate=m.mesa_gate_norm_backward(r["o"], gate, p["norm"], grad))
        gy, gdt = torch.empty_like(r["y"]), torch.empty_like(dt)
        gx, gb, gc = self.heads(gy)
        g["ssm"] = m.mesa_ssm_backward(r["x"], r["rb"], r["rc"], dt.transpose(1, 2), p["A"], g["gate"]["grad_x"], p["skip"],
                                       p["dt_bias"], state, lens=lens, grad_x=gx, grad_dt=gdt.transpose(1, 2), workspace=ws)
        g["rot"] = m.mesa_qk_rotate_backward(r["c"], r["b"], g["ssm"]["grad_c"], g["ssm"]["grad_b"], self.freqs, wq=p["wc"],
                                             wk=p["wb"], position0=position0, grad_q=gc, grad_k=gb)
        g["conv"] = m.mesa_causal_conv_backward(rows, p["w"], gy, p["bias"], hist, lens=lens)
        g["gy"] = gy
        return g


def inputs(seed, L, B, T):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(L.type)  # noqa: E731
    return r(B, T, L.D), r(B, T, L.H), r(B, T, L.H, L.dv), r(B, T, L.H, L.dv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,lens", [(2, 150, 1, 3, 32, 64, (150, 41)), (1, 1, 2, 2, 16, 32, None),
                                                 (1, 1290, 1, 2, 64, 32, None)])
def test_layer_and_its_gradients(B, T, Hk, H, dk, dv, lens, dtype):
    import torch
    from test_regression_amd import mesa
    say("case layer", (B, T, Hk, H, dk, dv, lens, dtype))
    L = Layer(mesa, 3, B, Hk, H, dk, dv, dtype)
    rows, dt, gate, grad = inputs(5, L, B, T)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    r = L.forward(rows, dt, gate, lens=n)
    g = L.backward(r, rows, dt, gate, grad, lens=n)
    torch.cuda.synchronize()
    f, pos = L.f, np.broadcast_to(np.arange(T), (B, T))
    y, carried, rc, terms = conv_ref(f64(rows), f["w"], f["bias"], None, lens, True, f64(g["gy"]))
    near(r["y"], y, conv_test.OUT[dtype], what="conv")
    assert np.array_equal(f64(r["hist"]), carried)
    near(g["conv"]["grad_x"], rc["grad_x"], conv_test.GRAD[dtype], what="grad rows")
    near(g["conv"]["grad_w"], rc["grad_w"], conv_test.SUMS, terms["grad_w"], what="grad_w")
    near(g["conv"]["grad_bias"], rc["grad_bias"], conv_test.SUMS, terms["grad_bias"], what="grad_bias")
    views = dict(zip("xbc", L.heads(g["gy"])))
    for name, w, got, dw in (("c", "wc", "grad_c", "grad_wq"), ("b", "wb", "grad_b", "grad_wk")):
        ry, rdx, rdw, tx, tw = rotate_ref(f64(r[name]), L.freqs.cpu().numpy(), pos, f[w], dy=f64(g["ssm"][got]))
        near(r["r" + name], ry, rotate_test.OUT[dtype], what="rotated " + name)
        near(views[name], rdx, rotate_test.GRAD[dtype], tx, what="gradient of " + name)
        near(g["rot"][dw], rdw, rotate_test.SUMS, tw, what=dw)
    s = dict(x=f64(r["x"]), b=f64(r["rb"]), c=f64(r["rc"]), dt=f64(dt.transpose(1, 2)), A=f["A"], D=f["skip"],
             dt_bias=f["dt_bias"], state=np.zeros((B, H, dv, dk)), lens=[T] * B if lens is None else lens)
    out, S, rs, terms = ssm_ref(s, f64(g["gate"]["grad_x"]))
    near(r["o"], out, what="scan")
    near(r["state"], S, what="state")
    # The gate norm's gradient g is orthogonal to the scan's outputs (scaling a row does not
    # change its norm).  One token without a start has o = (D b.c + skip) x, so that x.g = 0
    # in exact arithmetic, and grad_b = D c' x.g, grad_c = D b x.g are sums of terms that
    # cancel: what is left of them is roundings.  A sum's error is at most the bound's part
    # of its terms' sizes, which are the gradients of the absolute values.
    size = dict(s, **{n_: np.abs(s[n_]) for n_ in ("x", "b", "c", "D")})
    whole = ssm_ref(size, np.abs(f64(g["gate"]["grad_x"])))[2]
    terms.update({n_: np.linalg.norm(whole[n_]) for n_ in ("grad_b", "grad_c")})
    got = dict(g["ssm"], grad_x=views["x"])
    for n_, ref in rs.items():
        if n_ != "grad_state":
            near(got[n_], ref, terms=terms.get(n_, 0.0), what=n_)
    ot = f64(r["o"]).transpose(0, 2, 1, 3)
    gt = f64(gate)
    near(r["n"], ot / np.sqrt((ot * ot).mean(-1, keepdims=True) + 1e-6) * f["norm"] * gt / (1 + np.exp(-gt)), what="gate norm")


def test_prompt_then_tokens():
    """A prompt with its history and state kept, then tokens one by one in place, are the
    rows of the whole sequence.  float32; each token's history and state differ from the
    whole's by the bounds' roundings, which the norms keep relative: 4 operators' bounds."""
    import torch
    from test_regression_amd import mesa
    say("case prompt and tokens")
    L = Layer(mesa, 9, 2, 1, 4, 32, 64, "f32")
    rows, dt, gate, _ = inputs(6, L, 2, 133)
    whole = L.forward(rows, dt, gate)
    r = L.forward(rows[:, :129], dt[:, :129], gate[:, :129].contiguous())
    hist, state = r["hist"], r["state"]
    for t in range(129, 133):
        y, h = mesa.mesa_causal_conv(rows[:, t:t + 1], L.p["w"], L.p["bias"], hist, hist_out=hist, return_hist=True)
        assert h is hist
        x, b, c = L.heads(y)
        c, b = mesa.mesa_qk_rotate(c, b, L.freqs, wq=L.p["wc"], wk=L.p["wb"], position0=t)
        o = mesa.mesa_ssm_step(x[:, :, 0], b[:, :, 0], c[:, :, 0], dt[:, t], L.p["A"], state, L.p["skip"], L.p["dt_bias"])
        n = mesa.mesa_gate_norm(o[:, :, None], gate[:, t:t + 1].contiguous(), L.p["norm"])
        torch.cuda.synchronize()
        near(n, f64(whole["n"][:, t:t + 1]), 4 * F32, what=t)
    near(state, f64(whole["state"]), 4 * F32)


@pytest.mark.parametrize("dtype,T,dk,dv", [("bf16", 130, 64, 64), ("f32", 1100, 32, 32)])
def test_captured_layer_replays(dtype, T, dk, dv):
    """Forward and gradients in one graph with one workspace, replayed with other rows
    between eager calls and synchronisations: every replay is the eager result, to the bit."""
    import torch
    from test_regression_amd import mesa
    say("case graph", (dtype, T, dk, dv))
    L = Layer(mesa, 11, 2, 1, 2, dk, dv, dtype)
    rows, dt, gate, grad = inputs(8, L, 2, T)
    state = torch.randn(2, 2, dv, dk, device="cuda")
    code = 1 if dtype == "bf16" else 0
    ws = torch.empty(max(mesa.mesa_ssm_workspace_bytes(2, 2, T, dk, dv, code), 16,
                         mesa.mesa_ssm_backward_workspace_bytes(2, 1, 2, T, dk, dv, code)), dtype=torch.uint8, device="cuda")

    def calls():
        r = L.forward(rows, dt, gate, state=state, ws=ws)
        g = L.backward(r, rows, dt, gate, grad, state=state, ws=ws)
        s = state.clone()
        o = mesa.mesa_ssm_step(r["x"][:, :, 0], r["rb"][:, :, 0], r["rc"][:, :, 0], dt[:, 0], L.p["A"], s, L.p["skip"], L.p["dt_bias"])
        return [*r.values(), g["gy"], s, o, *[x for q in ("gate", "ssm", "rot", "conv") for x in g[q].values() if x is not None]]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for i in range(4):
        rows.copy_(torch.randn_like(rows))
        dt.copy_(torch.randn_like(dt))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for j, (x, y) in enumerate(zip(got, calls())):
            assert torch.equal(x, y), (i, j)
        torch.cuda.synchronize()


def test_layers_on_two_streams_at_once():
    import torch
    from test_regression_amd import mesa
    say("case two streams")
    layers = [Layer(mesa, s, 1, 1, 2, 64, 64, "bf16") for s in (1, 2)]
    ins = [inputs(s, L, 1, 1200) for s, L in zip((3, 4), layers)]

    def both(L, rows, dt, gate, grad):
        r = L.forward(rows, dt, gate)
        g = L.backward(r, rows, dt, gate, grad)
        return [*r.values(), *[x for q in ("gate", "ssm", "rot", "conv") for x in g[q].values() if x is not None]]
    ref = [both(L, *i) for L, i in zip(layers, ins)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(layers[i], *ins[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(run, ref[i]))


def test_a_given_stream_owns_what_is_allocated():
    import torch
    from test_regression_amd import mesa
    say("case given stream")
    t, _ = ssm_inputs(5, 1, 1, 2, 1100, 64, 64, "f32")
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    go = torch.randn_like(d["x"])
    rows, w = torch.randn(1, 1100, 64, device="cuda"), torch.randn(4, 64, device="cuda")
    freqs, _ = mesa.mesa_rotary_frequencies(64)
    head = (d["x"], d["b"], d["c"], d["dt"], d["A"])
    one = [y[:, :, 0].contiguous() for y in (d["x"], d["b"], d["c"], d["dt"])]

    def calls(s):
        o, S = mesa.mesa_ssm_forward(*head, d["D"], d["dt_bias"], d["state"], return_final=True, stream=s)
        g = mesa.mesa_ssm_backward(*head, go, d["D"], d["dt_bias"], d["state"], stream=s)
        y = mesa.mesa_causal_conv(rows, w, stream=s)
        gy = mesa.mesa_causal_conv_backward(rows, w, rows, stream=s)
        q, k = mesa.mesa_qk_rotate(d["x"], d["b"], freqs, stream=s)
        gq = mesa.mesa_qk_rotate_backward(d["x"], d["b"], d["x"], d["b"], freqs, stream=s)
        return [o, S, y, q, k, *[x for e in (g, gy, gq) for x in e.values() if x is not None]]
    ref = calls(None)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = [calls(stream) for _ in range(3)]
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(16)]   # must not take the workspaces
    state = d["state"].clone()
    step = mesa.mesa_ssm_step(*one, d["A"], state, d["D"], d["dt_bias"], stream=stream)
    torch.cuda.synchronize()
    for run in got:
        assert all(torch.equal(x, y) for x, y in zip(run, ref))
    assert torch.isfinite(step).all() and len(junk) == 16


@pytest.mark.parametrize("T", [100, 1100])
def test_states_in_place(T):
    """The final state over the initial one, the start's gradient over the end's: with and
    without segments."""
    import torch
    from test_regression_amd import mesa
    say("case in place", T)
    t, f = ssm_inputs(13, 2, 1, 2, T, 32, 64, "f32", lens=(T, T // 2))
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    head = (d["x"], d["b"], d["c"], d["dt"], d["A"])
    o, S = mesa.mesa_ssm_forward(*head, d["D"], d["dt_bias"], d["state"], lens=d["lens"], return_final=True)
    state = d["state"].clone()
    o2, _ = mesa.mesa_ssm_forward(*head, d["D"], d["dt_bias"], state, lens=d["lens"], final_state=state)
    assert torch.equal(o, o2) and torch.equal(S, state)
    go, gof = store(np.random.default_rng(1).standard_normal(f["x"].shape), "f32")
    gf, gff = store(np.random.default_rng(2).standard_normal(f["state"].shape), "f32")
    g = mesa.mesa_ssm_backward(*head, go.cuda(), d["D"], d["dt_bias"], d["state"], lens=d["lens"], grad_final=gf.cuda())
    torch.cuda.synchronize()
    _, _, ref, terms = ssm_ref(f, gof, gff)
    for n, y in ref.items():
        near(g[n], y, terms=terms.get(n, 0.0), what=n)
    # the C call with the start's gradient over the end's
    L, code = mesa.lib(), 0
    r, buf = {n: torch.full_like(y, float("nan")) for n, y in g.items() if y is not None}, gf.cuda()
    ws = torch.empty(mesa.mesa_ssm_backward_workspace_bytes(2, 1, 2, T, 32, 64, code), dtype=torch.uint8, device="cuda")
    p, gc = (lambda y: y.data_ptr()), go.cuda()
    st = L.mesa_ssm_backward(p(d["x"]), None, p(d["b"]), None, p(d["c"]), None, code, p(d["dt"]), None, code, p(d["A"]), p(d["D"]),
                             p(d["dt_bias"]), 1, p(d["state"]), p(d["lens"]), p(gc), p(buf), 2, 1, 2, T, 32, 64, p(r["grad_x"]), None,
                             p(r["grad_b"]), None, p(r["grad_c"]), None, p(r["grad_dt"]), None, p(r["grad_A"]), p(r["grad_D"]),
                             p(r["grad_dt_bias"]), p(buf), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for n, y in r.items():
        assert torch.equal(buf if n == "grad_state" else y, g[n]), n


@pytest.mark.parametrize("B,H,T,dk,dv", [(2, 130, 130, 32, 32), (1, 110, 1100, 32, 128), (1, 220, 70, 64, 16)])
def test_many_heads(B, H, T, dk, dv):
    """More workgroups than CUs, and just as many: no segments either way."""
    import torch
    from test_regression_amd import mesa
    say("case many heads", (B, H, T, dk, dv))
    t, f = ssm_inputs(17, B, 1, H, T, dk, dv, "bf16")
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    o, S = mesa.mesa_ssm_forward(d["x"], d["b"], d["c"], d["dt"], d["A"], d["D"], d["dt_bias"], d["state"], return_final=True)
    torch.cuda.synchronize()
    ro, rS = ssm_ref(f)
    near(o, ro)
    near(S, rS)


def test_kernels_are_counted():
    import torch
    from test_regression_amd import mesa
    say("case profile")
    L = Layer(mesa, 3, 1, 1, 2, 32, 32, "f32")
    rows, dt, gate, grad = inputs(5, L, 1, 70)
    torch.cuda.synchronize()
    mesa.profile_reset()
    mesa.profile_enable(True)
    try:
        r = L.forward(rows, dt, gate)
        L.backward(r, rows, dt, gate, grad)
        torch.cuda.synchronize()
        for kernel in (mesa.KERNEL_CAUSAL_CONV, mesa.KERNEL_CAUSAL_CONV_BWD, mesa.KERNEL_SSM_SCAN, mesa.KERNEL_SSM_STATES,
                       mesa.KERNEL_SSM_GRADS, mesa.KERNEL_QK_ROTATE, mesa.KERNEL_QK_ROTATE_BWD):
            ms, calls = mesa.profile_read(kernel)
            assert calls >= 1 and ms > 0.0, kernel
    finally:
        mesa.profile_enable(False)
        mesa.profile_reset()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens", [(1100, (1100, 70, 0)), (130, (1, 64, 130))])
def test_nothing_behind_a_length_is_read(T, lens, dtype):
    """NaN behind the rows' lengths and in the workspaces: the results of clean rows, bit for bit."""
    import torch
    from test_regression_amd import mesa
    say("case behind lengths", (T, lens, dtype))
    B, Hk, H, dk, dv, W, code = 3, 1, 2, 64, 32, 3, 1 if dtype == "bf16" else 0
    t, _ = ssm_inputs(23, B, Hk, H, T, dk, dv, dtype, lens=lens)
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    gen = torch.Generator(device="cuda").manual_seed(1)
    d["go"] = torch.randn(B, H, T, dv, device="cuda", generator=gen).to(d["x"].dtype)
    d["rows"], d["dy"] = (torch.randn(B, T, 40, device="cuda", generator=gen).to(d["x"].dtype) for _ in range(2))
    hist = torch.randn(B, W - 1, 40, device="cuda", generator=gen).to(d["x"].dtype)
    w, gf = torch.randn(W, 40, device="cuda", generator=gen), torch.randn(B, H, dv, dk, device="cuda", generator=gen)

    def calls(fill):
        ws = lambda n: torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        head = [d[n] for n in ("x", "b", "c", "dt", "A")]
        o, S = mesa.mesa_ssm_forward(*head, d["D"], d["dt_bias"], d["state"], lens=d["lens"], return_final=True,
                                     workspace=ws(mesa.mesa_ssm_workspace_bytes(B, H, T, dk, dv, code)))
        g = mesa.mesa_ssm_backward(*head, d["go"], d["D"], d["dt_bias"], d["state"], lens=d["lens"], grad_final=gf,
                                   workspace=ws(mesa.mesa_ssm_backward_workspace_bytes(B, Hk, H, T, dk, dv, code)))
        y, h = mesa.mesa_causal_conv(d["rows"], w, None, hist, lens=d["lens"], return_hist=True)
        gy = mesa.mesa_causal_conv_backward(d["rows"], w, d["dy"], None, hist, lens=d["lens"],
                                            workspace=ws(mesa.mesa_causal_conv_backward_workspace_bytes(B, T, 40, W)))
        torch.cuda.synchronize()
        return [o, S, y, h, *[x for q in (g, gy) for x in q.values() if x is not None]]
    ref = calls(0)
    for b, n in enumerate(lens):
        for name in ("x", "b", "c", "go"):
            d[name][b, :, n:] = float("nan")
        for name in ("rows", "dy"):
            d[name][b, n:] = float("nan")
        d["dt"][b, :, n:] = float("nan")
    for i, (x, y) in enumerate(zip(calls(255), ref)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("B,Hk,H,T,dk,dv", [(1, 1, 3, 520, 32, 32), (1, 1, 2, 1290, 128, 64), (2, 1, 12, 700, 16, 16)])
def test_segments_of_few_chunks(B, Hk, H, T, dk, dv):
    """Short segments, the last of them with few chunks or none, both directions."""
    import torch
    from test_regression_amd import mesa
    say("case short segments", (B, Hk, H, T, dk, dv))
    t, f = ssm_inputs(31, B, Hk, H, T, dk, dv, "f32")
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    rng = np.random.default_rng(2)
    go, gof = store(rng.standard_normal((B, H, T, dv)), "f32")
    gf, gff = store(rng.standard_normal((B, H, dv, dk)), "f32")
    head = [d[n] for n in ("x", "b", "c", "dt", "A")]
    o, S = mesa.mesa_ssm_forward(*head, d["D"], d["dt_bias"], d["state"], return_final=True)
    g = mesa.mesa_ssm_backward(*head, go.cuda(), d["D"], d["dt_bias"], d["state"], grad_final=gf.cuda())
    torch.cuda.synchronize()
    ro, rS, rg, terms = ssm_ref(f, gof, gff)
    near(o, ro)
    near(S, rS)
    for n, y in rg.items():
        near(g[n], y, terms=terms.get(n, 0.0), what=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pairs_before_a_token_leave_nothing(dtype):
    """Outputs whose gradients end at token 20: later step sizes change nothing.  Their
    gradients are differences of the same float64 products E_ij summed two ways, at most
    64 64 additions of 2^-53 of the terms each: below 2^-40 of A times the sum of |E|."""
    import torch
    from test_regression_amd import mesa
    say("case pairs before", dtype)
    B, H, T, dk, dv, last = 2, 3, 64, 32, 64, 20
    t, f = ssm_inputs(41, B, 1, H, T, dk, dv, dtype, start=False)
    d = {n: None if x is None else x.cuda() for n, x in t.items()}
    d["dt"] = d["dt"].float()
    go, gof = store(np.random.default_rng(3).standard_normal((B, H, T, dv)), dtype)
    go[:, :, last:] = 0
    gof[:, :, last:] = 0
    g = mesa.mesa_ssm_backward(d["x"], d["b"], d["c"], d["dt"], d["A"], go.cuda(), d["D"], d["dt_bias"])
    torch.cuda.synchronize()
    step = np.log1p(np.exp(f["dt"] + f["dt_bias"][:, None]))
    pairs = np.abs(gof @ f["x"].transpose(0, 1, 3, 2)) * np.abs(f["c"] @ f["b"].transpose(0, 1, 3, 2)) * step[:, :, None]
    most = np.tril(pairs).sum((2, 3)) * np.abs(f["A"])
    late = np.abs(f64(g["grad_dt"])[:, :, last:]).max(-1)
    assert (late <= 2.0 ** -40 * most).all(), (late / most).max()
