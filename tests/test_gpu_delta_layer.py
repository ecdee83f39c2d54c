"""The new operators as a layer uses them together: pre-normalised residual,
q/k pre-processing, the delta rule, norm and gate of its outputs; its gradients;
captured in a graph; on other streams."""
import sys

import numpy as np
import pytest

from tests.delta_helpers import F32, delta_inputs, delta_ref, rel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def block(mesa, p, h, y, state, T):
    """residual_norm -> projections -> delta rule -> gate norm -> projection, for [1, T] tokens of 2 heads."""
    h, n = mesa.mesa_residual_norm(h, y, p["w1"], p["scale"], 1e-6)
    heads = lambda m, d: (n @ m).view(1, T, 2, d).transpose(1, 2).contiguous()  # noqa: E731
    q, k = (mesa.mesa_qk_preprocess(heads(p[m], 32), p["conv"]) for m in ("wq", "wk"))
    v = heads(p["wv"], 64)
    gamma, beta = ((n @ p[m]).sigmoid().t().reshape(1, 2, T).contiguous() for m in ("wg", "wb"))
    o, state = mesa.mesa_delta_forward(q, k, v, gamma, beta, state, return_final=True)
    gate = (n @ p["wgate"]).view(1, T, 2, 64)
    return h, mesa.mesa_gate_norm(o, gate, p["w2"], 1e-6).view(T, 128) @ p["wo"], state


def params():
    import torch
    torch.manual_seed(7)
    D = 96
    r = lambda *s: 0.1 * torch.randn(*s, device="cuda")  # noqa: E731
    return dict(w1=1 + r(D), scale=0.5 + r(D), conv=r(2, 3, 32) + 0.3, wq=r(D, 64), wk=r(D, 64), wv=r(D, 128), wg=r(D, 2) + 0.02,
                wb=r(D, 2), wgate=r(D, 128), w2=1 + r(2, 64), wo=r(128, D)), D


def test_a_block_whole_and_in_pieces():
    import torch
    from test_regression_amd import mesa
    say("case block")
    p, D = params()
    T = 150
    h, y = torch.randn(T, D, device="cuda"), torch.randn(T, D, device="cuda")
    S0 = torch.zeros(1, 2, 64, 32, device="cuda")
    h1, o1, S1 = block(mesa, p, h, y, S0, T)
    torch.cuda.synchronize()
    # the same block in float64 on the CPU
    c = {n: x.double().cpu().numpy() for n, x in p.items()}
    z = h.double().cpu().numpy() + c["scale"] * y.double().cpu().numpy()
    n = z / np.sqrt((z * z).mean(-1, keepdims=True) + 1e-6) * c["w1"]
    heads = lambda m, d: (n @ c[m]).reshape(1, T, 2, d).transpose(0, 2, 1, 3)  # noqa: E731

    def conv(x):
        x = np.concatenate([np.zeros((1, 2, 2, 32)), x], 2)
        s = sum(c["conv"][None, :, j, None, :] * x[:, :, 2 - j:2 - j + T] for j in range(3))
        return s / np.linalg.norm(s, axis=-1, keepdims=True)
    sg = lambda x: 1 / (1 + np.exp(-x))  # noqa: E731
    f = dict(q=conv(heads("wq", 32)), k=conv(heads("wk", 32)), v=heads("wv", 64), state=np.zeros((1, 2, 64, 32)),
             gamma=sg(n @ c["wg"]).T.reshape(1, 2, T), beta=sg(n @ c["wb"]).T.reshape(1, 2, T))
    o, S = delta_ref(f)
    ot = o.transpose(0, 2, 1, 3)
    gate = (n @ c["wgate"]).reshape(1, T, 2, 64)
    u = ot / np.sqrt((ot * ot).mean(-1, keepdims=True) + 1e-6) * c["w2"] * gate * sg(gate)
    ref = u.reshape(T, 128) @ c["wo"]
    # the projections' float32 products of up to 128 terms and the norms add to the rule's bound
    assert rel(h1.cpu(), z) <= F32 and rel(S1.cpu(), S) <= 2 * F32 and rel(o1.cpu(), ref) <= 3 * F32


def test_captured_calls_share_a_workspace_and_replay():
    """A step, a sequence call, its gradients and the norms captured in one
    graph, replayed between eager calls and synchronisations."""
    import torch
    from test_regression_amd import mesa
    say("case graph")
    t, _ = delta_inputs(3, 2, 2, 4, 130, 64, 64, "bf16")
    d = {n: x.cuda() for n, x in t.items()}
    go = torch.randn_like(d["v"])
    w, w2 = torch.ones(4, 64, device="cuda"), torch.ones(256, device="cuda")
    need = max(mesa.mesa_delta_workspace_bytes(2, 4, 130, 64, 64, 1),
               mesa.mesa_delta_backward_workspace_bytes(2, 2, 4, 130, 64, 64, 1))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    gate = torch.randn(2, 130, 4, 64, device="cuda").bfloat16()
    res = torch.randn(260, 256, device="cuda")

    def calls():
        o, S = mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], return_final=True,
                                       workspace=ws)
        g = mesa.mesa_delta_backward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], go, d["state"], workspace=ws)
        y = mesa.mesa_gate_norm(o, gate, w)
        gy = mesa.mesa_gate_norm_backward(o, gate, w, y)
        z, n = mesa.mesa_residual_norm(res, y.view(260, 256), w2)
        gr = mesa.mesa_residual_norm_backward(res, y.view(260, 256), w2, n)
        s = d["state"].clone()
        one = {k: d[k][:, :, 5].contiguous() for k in ("q", "k", "v", "gamma", "beta")}
        os = mesa.mesa_delta_step(one["q"], one["k"], one["v"], one["gamma"], one["beta"], s)
        return [o, S, y, z, n, s, os, *[x for q in (g, gy, gr) for x in q.values() if x is not None]]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for i in range(4):
        d["v"].copy_(torch.randn_like(d["v"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for j, (x, y) in enumerate(zip(got, calls())):
            assert torch.equal(x, y), (i, j)
        torch.cuda.synchronize()


def test_calls_on_a_given_stream():
    """Two streams at once, each with its own workspace and outputs."""
    import torch
    from test_regression_amd import mesa
    say("case streams")
    ins = [{n: x.cuda() for n, x in delta_inputs(s, 1, 4, 4, 700, 64, 64, "f32")[0].items()} for s in (1, 2)]
    ref = [mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], return_final=True) for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [mesa.mesa_delta_forward(d["q"], d["k"], d["v"], d["gamma"], d["beta"], d["state"], return_final=True, stream=s)
           for _ in range(3) for d, s in zip(ins, streams)]
    # allocations of the current stream meanwhile must not take the workspaces
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    for i, (o, S) in enumerate(got):
        assert torch.equal(o, ref[i % 2][0]) and torch.equal(S, ref[i % 2][1])
    assert len(junk) == 16


def test_captured_long_prompt_carries_its_state():
    """A sequence long enough for segments, captured with its final state over
    its initial one: each replay takes the state on, as eager calls do."""
    import torch
    from test_regression_amd import mesa
    say("case graph, segments")
    t, _ = delta_inputs(7, 1, 1, 2, 4100, 64, 64, "bf16", lo=0.97)
    d = {n: x.cuda() for n, x in t.items()}
    args = [d[n] for n in ("q", "k", "v", "gamma", "beta")]
    ws = torch.empty(mesa.mesa_delta_workspace_bytes(1, 2, 4100, 64, 64, 1), dtype=torch.uint8, device="cuda")
    out, state = torch.empty_like(d["v"]), d["state"].clone()
    call = lambda: mesa.mesa_delta_forward(*args, state, out=out, final_state=state, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    state.copy_(d["state"])
    eager = d["state"].clone()
    for i in range(3):
        graph.replay()
        o, eager = mesa.mesa_delta_forward(*args, eager, return_final=True)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(state, eager), i


def test_calls_on_two_streams_at_once():
    import torch
    from test_regression_amd import mesa
    say("case two streams")
    d = [{n: x.cuda() for n, x in delta_inputs(s, 1, 2, 2, 1000, 64, 64, "bf16")[0].items()} for s in (8, 9)]
    go = [torch.randn_like(x["v"]) for x in d]
    fwd = lambda x, s: mesa.mesa_delta_forward(*x.values(), return_final=True, stream=s)  # noqa: E731
    bwd = lambda x, g, s: mesa.mesa_delta_backward(x["q"], x["k"], x["v"], x["gamma"], x["beta"], g, x["state"], stream=s)  # noqa: E731
    ref = [(fwd(x, None), bwd(x, g, None)) for x, g in zip(d, go)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append((fwd(d[i], s), bwd(d[i], go[i], s)))
    torch.cuda.synchronize()
    for i in range(2):
        for f, b in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(f, ref[i][0]))
            assert all(torch.equal(b[n], ref[i][1][n]) for n in b)
