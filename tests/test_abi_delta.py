"""The entry points of the gated delta rule and of the norms around a layer, on
the CPU: their workspace sizes, and what they refuse before touching the device.

The C calls get fake pointers (never dereferenced): every one fails validation.
"""
import ctypes

import pytest

from test_regression_amd import mesa

OK, INVALID, UNSUPPORTED, WS_SMALL, HIPERR = range(5)
FAKE, OTHER = 0x10000, 0x20000   # 16-byte aligned, never dereferenced
F32, BF16 = mesa.MESA_DTYPE_F32, mesa.MESA_DTYPE_BF16

DELTA = dict(q=FAKE, k=FAKE, v=FAKE, dtype=F32, gamma=FAKE, beta=FAKE)
HEADS = dict(Hk=2, H=4)
ENTRIES = {
    "mesa_delta_forward": dict(DELTA, state0=FAKE, B=1, **HEADS, T=100, dk=64, dv=64, out=OTHER, final_state=FAKE,
                               workspace=FAKE, workspace_bytes=1 << 40, stream=None),
    "mesa_delta_backward": dict(DELTA, state0=FAKE, grad_out=FAKE, grad_final=FAKE, B=1, **HEADS, T=100, dk=64, dv=64,
                                grad_q=OTHER, grad_k=OTHER, grad_v=OTHER, grad_gamma=OTHER, grad_beta=OTHER,
                                grad_state=OTHER, workspace=FAKE, workspace_bytes=1 << 40, stream=None),
    "mesa_delta_step": dict(DELTA, state=FAKE, N=3, **HEADS, dk=64, dv=64, out=OTHER, stream=None),
    "mesa_gate_norm": dict(x=FAKE, x_dtype=F32, gate=FAKE, dtype=BF16, w=FAKE, eps=1e-6, B=1, H=2, T=5, d=64, y=OTHER,
                           stream=None),
    "mesa_gate_norm_backward": dict(x=FAKE, x_dtype=F32, gate=FAKE, dtype=BF16, w=FAKE, eps=1e-6, grad_y=FAKE, B=1, H=2,
                                    T=5, d=64, grad_x=OTHER, grad_gate=OTHER, grad_w=OTHER, workspace=FAKE,
                                    workspace_bytes=1 << 40, stream=None),
    "mesa_residual_norm": dict(h=FAKE, h_dtype=F32, y=FAKE, dtype=BF16, scale=FAKE, w=FAKE, eps=1e-6, R=5, D=100,
                               h_out=FAKE + 4096, n=OTHER, stream=None),
    "mesa_residual_norm_backward": dict(h=FAKE, h_dtype=F32, y=FAKE, dtype=BF16, scale=FAKE, w=FAKE, eps=1e-6,
                                        grad_n=FAKE, grad_h_out=FAKE, R=5, D=100, grad_h=OTHER, grad_y=OTHER,
                                        grad_w=OTHER, grad_scale=OTHER, workspace=FAKE, workspace_bytes=1 << 40,
                                        stream=None),
}


def call(name, **kw):
    a = dict(ENTRIES[name])
    assert set(kw) <= set(a), kw
    a.update(kw)
    L = mesa.lib()
    st = getattr(L, name)(*(ctypes.c_float(v) if n == "eps" else v for n, v in a.items()))
    return st, L.mesa_last_error_message().decode()


def refused(name, status, needle, **kw):
    st, msg = call(name, **kw)
    assert st == status, (name, kw, st, msg)
    assert needle in msg, (name, kw, msg)


NULLS = {
    "mesa_delta_forward": "q k v gamma beta out workspace",
    "mesa_delta_backward": "q k v gamma beta grad_out grad_q grad_k grad_v grad_gamma grad_beta workspace",
    "mesa_delta_step": "q k v gamma beta state out",
    "mesa_gate_norm": "x w y",
    "mesa_gate_norm_backward": "x w grad_y grad_x grad_w workspace",
    "mesa_residual_norm": "h w n",
    "mesa_residual_norm_backward": "h w grad_n grad_h grad_w workspace",
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in NULLS.items() for a in args.split()])
def test_null_pointers(name, arg):
    refused(name, INVALID, "non-null", **{arg: None})


POINTERS = [(n, a) for n, args in ENTRIES.items() for a, v in args.items() if v in (FAKE, OTHER, FAKE + 4096)]
WORDS = ("gamma", "beta", "grad_gamma", "grad_beta", "grad_w", "grad_scale")   # need the alignment of a float only


@pytest.mark.parametrize("name,arg", POINTERS)
def test_misaligned_pointers(name, arg):
    base = ENTRIES[name][arg]
    refused(name, INVALID, "misaligned", **{arg: base + (2 if arg in WORDS else 8)})


@pytest.mark.parametrize("name", [n for n in ENTRIES if "delta" in n])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INVALID, "dtype 2"), (dict(dtype=-1), INVALID, "dtype -1"),
    (dict(B=0), INVALID, "positive"), (dict(Hk=0), INVALID, "positive"), (dict(H=0), INVALID, "positive"),
    (dict(H=-4), INVALID, "positive"), (dict(T=-1), INVALID, "positive"),
    (dict(dk=0), INVALID, "positive"), (dict(dv=-16), INVALID, "positive"),
    (dict(H=3), INVALID, "multiple"), (dict(Hk=4, H=2), INVALID, "multiple"),
    (dict(dk=48), UNSUPPORTED, "dk=48"), (dict(dk=256), UNSUPPORTED, "dk=256"), (dict(dk=8), UNSUPPORTED, "dk=8"),
    (dict(dv=48), UNSUPPORTED, "dv=48"), (dict(dv=512), UNSUPPORTED, "dv=512"),
    (dict(B=1 << 20, H=1 << 10), INVALID, "grid too large"),
    (dict(B=1 << 30, H=1 << 30), INVALID, "grid too large"),
    (dict(B=1 << 12, T=(1 << 31) - 1), INVALID, "grid too large"),
])
def test_delta_sizes(name, kw, status, needle):
    if "step" in name:   # one token
        kw = {"N" if n == "B" else n: v for n, v in kw.items()}
        if kw.pop("T", None) is not None:
            kw, status, needle = dict(N=0), INVALID, "positive"
    refused(name, status, needle, **kw)


@pytest.mark.parametrize("name,outs,ins", [
    ("mesa_delta_forward", ("out",), ("q", "k", "v")),
    ("mesa_delta_step", ("out",), ("q", "k", "v")),
    ("mesa_delta_backward", ("grad_q", "grad_k", "grad_v"), ("q", "k", "v", "grad_out")),
    ("mesa_gate_norm", ("y",), ("x", "gate")),
    ("mesa_gate_norm_backward", ("grad_x", "grad_gate"), ("x", "gate", "grad_y")),
    ("mesa_residual_norm", ("n",), ("h", "y", "h_out")),
    ("mesa_residual_norm", ("h_out",), ("y",)),
    ("mesa_residual_norm_backward", ("grad_h", "grad_y"), ("h", "y", "grad_n", "grad_h_out")),
])
def test_outputs_over_inputs(name, outs, ins):
    for o in outs:
        for i in ins:
            refused(name, INVALID, "alias", **{o: 0x30000, i: 0x30000})


@pytest.mark.parametrize("name", ["mesa_gate_norm", "mesa_gate_norm_backward"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(x_dtype=2), INVALID, "x_dtype 2"), (dict(dtype=7), INVALID, "dtype 7"),
    (dict(B=0), INVALID, "positive"), (dict(H=0), INVALID, "positive"), (dict(T=-1), INVALID, "positive"),
    (dict(d=0), INVALID, "positive"), (dict(d=48), UNSUPPORTED, "d=48"), (dict(d=512), UNSUPPORTED, "d=512"),
    (dict(eps=0.0), INVALID, "eps"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=float("inf")), INVALID, "eps"),
    (dict(B=1 << 20, T=1 << 20), INVALID, "grid too large"),
])
def test_gate_norm_sizes(name, kw, status, needle):
    refused(name, status, needle, **kw)


@pytest.mark.parametrize("name", ["mesa_residual_norm", "mesa_residual_norm_backward"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(h_dtype=2), INVALID, "h_dtype 2"), (dict(dtype=-1), INVALID, "dtype -1"),
    (dict(R=-1), INVALID, "positive"), (dict(D=0), INVALID, "positive"), (dict(D=16385), UNSUPPORTED, "D=16385"),
    (dict(eps=0.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(R=(1 << 31) - 1), INVALID, "grid too large"), (dict(R=1 << 25, D=2048), INVALID, "grid too large"),
])
def test_residual_norm_sizes(name, kw, status, needle):
    refused(name, status, needle, **kw)


def test_optional_tensors_come_together():
    refused("mesa_gate_norm_backward", INVALID, "grad_gate", grad_gate=None)
    refused("mesa_gate_norm_backward", INVALID, "grad_gate", gate=None)
    refused("mesa_residual_norm", INVALID, "h_out", h_out=None)
    refused("mesa_residual_norm", INVALID, "scale needs y", y=None)
    refused("mesa_residual_norm", INVALID, "h_out", y=None, scale=None)
    refused("mesa_residual_norm_backward", INVALID, "scale needs y", y=None)
    refused("mesa_residual_norm_backward", INVALID, "grad_y", grad_y=None)
    refused("mesa_residual_norm_backward", INVALID, "grad_y", grad_scale=None)
    refused("mesa_residual_norm_backward", INVALID, "grad_y", scale=None)


@pytest.mark.parametrize("name,need", [
    ("mesa_delta_forward", lambda: mesa.mesa_delta_workspace_bytes(1, 4, 100, 64, 64, F32)),
    ("mesa_delta_backward", lambda: mesa.mesa_delta_backward_workspace_bytes(1, 2, 4, 100, 64, 64, F32)),
    ("mesa_gate_norm_backward", lambda: mesa.lib().mesa_gate_norm_backward_workspace_bytes(1, 2, 5, 64)),
    ("mesa_residual_norm_backward", lambda: mesa.lib().mesa_residual_norm_backward_workspace_bytes(5, 100)),
])
def test_small_workspaces(name, need):
    n = need()
    assert n > 0
    refused(name, WS_SMALL, f"{n} needed", workspace_bytes=n - 1)
    refused(name, WS_SMALL, f"{n} needed", workspace_bytes=0)


def test_workspace_sizes():
    f, b = mesa.mesa_delta_workspace_bytes, mesa.mesa_delta_backward_workspace_bytes
    assert f(1, 4, 0, 64, 64, F32) == f(0, 4, 10, 64, 64, F32) == f(1, 4, 10, 64, 64, 9) == 0
    assert b(1, 0, 4, 10, 64, 64, F32) == b(1, 2, 4, 0, 64, 64, F32) == b(1, 2, 4, 10, 64, 64, 9) == 0
    # per head and chunk, not per token; float planes twice bf16's
    assert f(1, 1, 1, 64, 64, F32) == f(1, 1, 64, 64, 64, F32) < f(1, 1, 65, 64, 64, F32)
    assert f(2, 3, 64, 64, 64, BF16) == 6 * f(1, 1, 64, 64, 64, BF16) < 6 * f(1, 1, 64, 64, 64, F32)
    # few heads of a long sequence: the segments' states come on top; many heads have none
    n, many = 256, 512
    per_chunk = f(1, 1, 64, 128, 128, BF16)
    assert f(1, many, 64 * n, 128, 128, BF16) == many * n * per_chunk
    assert f(1, 1, 64 * n, 128, 128, BF16) > n * per_chunk
    # shared heads keep their own heads' gradients until they are summed
    assert b(1, 2, 4, 100, 64, 64, F32) - b(1, 4, 4, 100, 64, 64, F32) == 2 * 4 * 100 * 64 * 4
    g, r = mesa.lib().mesa_gate_norm_backward_workspace_bytes, mesa.lib().mesa_residual_norm_backward_workspace_bytes
    assert g(1, 2, 0, 64) == g(1, 2, 5, 0) == r(0, 64) == r(5, 0) == 0
    assert g(1, 2, 5, 64) == 2 * 64 * 4 and r(5, 100) == 2 * 2 * 100 * 4
    assert r(1 << 20, 100) == 512 * 2 * 100 * 4


def test_kernel_names():
    names = [mesa.kernel_name(i) for i in (
        mesa.KERNEL_DELTA_PREP, mesa.KERNEL_DELTA_SCAN, mesa.KERNEL_DELTA_STEP, mesa.KERNEL_DELTA_BWD_SCAN,
        mesa.KERNEL_DELTA_GRADS, mesa.KERNEL_GATE_NORM, mesa.KERNEL_GATE_NORM_BWD, mesa.KERNEL_RESIDUAL_NORM,
        mesa.KERNEL_RESIDUAL_NORM_BWD)]
    assert len(set(names)) == 9 and all(n.split("_")[0] in ("delta", "gate", "residual") for n in names)
    for i in (*range(9, 16), 25, -1):
        with pytest.raises(ValueError, match="kernel id"):
            mesa.profile_read(i)


# ---- the Python calls ----
torch = pytest.importorskip("torch")


def delta_tensors():
    z = torch.zeros
    return dict(q=z(1, 2, 5, 16), k=z(1, 2, 5, 16), v=z(1, 4, 5, 32), gamma=z(1, 4, 5), beta=z(1, 4, 5),
                state=z(1, 4, 32, 16))


def step_tensors():
    t = delta_tensors()
    return {n: x if n == "state" else x[:, :, 0].contiguous() for n, x in t.items()}


def delta_call(kind, **kw):
    t = step_tensors() if kind == "step" else delta_tensors()
    t.update({n: x for n, x in kw.items() if n in t})
    rest = {n: x for n, x in kw.items() if n not in t}
    if kind == "step":
        return mesa.mesa_delta_step(*t.values(), **rest)
    if kind == "forward":
        return mesa.mesa_delta_forward(*t.values(), **rest)
    go = rest.pop("grad_out", torch.zeros(1, 4, 5, 32))
    return mesa.mesa_delta_backward(t["q"], t["k"], t["v"], t["gamma"], t["beta"], go, t["state"], **rest)


@pytest.mark.parametrize("kind", ["forward", "backward", "step"])
def test_delta_calls_refuse_wrong_shapes(kind):
    good = step_tensors() if kind == "step" else delta_tensors()
    for n, x in good.items():
        with pytest.raises((ValueError, TypeError), match="must have shape|dimension|multiple|dims"):
            delta_call(kind, **{n: torch.zeros(*x.shape[:-1], x.shape[-1] + 16)})
        with pytest.raises((ValueError, TypeError)):
            delta_call(kind, **{n: x[0]})
    with pytest.raises(ValueError, match="multiple"):
        v = torch.zeros(*good["v"].shape)[:, :3]
        delta_call(kind, v=v)
    if kind != "backward":
        with pytest.raises(ValueError, match="out must have shape"):
            delta_call(kind, out=torch.zeros(3))
    else:
        with pytest.raises(ValueError, match="grad_out must have shape"):
            delta_call(kind, grad_out=torch.zeros(1, 4, 32, 5))
        with pytest.raises(ValueError, match="grad_final must have shape"):
            delta_call(kind, grad_final=torch.zeros(1, 4, 16, 32))


@pytest.mark.parametrize("kind", ["forward", "backward", "step"])
def test_delta_calls_refuse_cpu_tensors_and_types(kind):
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        delta_call(kind)                                       # CPU tensors
    for n in ("q", "gamma", "state"):
        x = (step_tensors() if kind == "step" else delta_tensors())[n]
        with pytest.raises((ValueError, TypeError)):
            delta_call(kind, **{n: x.half()})


def test_norm_calls_refuse_wrong_arguments():
    x, gate, w = torch.zeros(1, 2, 5, 16), torch.zeros(1, 5, 2, 16), torch.zeros(2, 16)
    bad = (ValueError, TypeError)
    for args in [(x[0], gate, w), (x, torch.zeros(1, 2, 5, 16), w), (x, gate, torch.zeros(16))]:
        with pytest.raises(bad):
            mesa.mesa_gate_norm(*args)
        with pytest.raises(bad):
            mesa.mesa_gate_norm_backward(*args, torch.zeros(1, 5, 2, 16))
    with pytest.raises(ValueError, match="out must have shape"):
        mesa.mesa_gate_norm(x, gate, w, out=torch.zeros(1, 2, 5, 16))
    with pytest.raises(ValueError, match="out_dtype"):
        mesa.mesa_gate_norm(x, gate, w, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="grad_y must have shape"):
        mesa.mesa_gate_norm_backward(x, gate, w, torch.zeros(1, 2, 5, 16))
    h, y, w = torch.zeros(3, 10), torch.zeros(3, 10), torch.zeros(10)
    for args in [(h[0], y, w), (h, torch.zeros(3, 11), w), (h, y, torch.zeros(11)), (h, y, w[None])]:
        with pytest.raises(bad):
            mesa.mesa_residual_norm(*args)
        with pytest.raises(bad):
            mesa.mesa_residual_norm_backward(*args, torch.zeros(3, 10))
    with pytest.raises(ValueError, match="need y"):
        mesa.mesa_residual_norm(h, None, w, scale=w)
    with pytest.raises(ValueError, match="need y"):
        mesa.mesa_residual_norm(h, None, w, h_out=torch.zeros(3, 10))
    with pytest.raises(ValueError, match="out_dtype"):
        mesa.mesa_residual_norm(h, y, w, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="grad_n must have shape"):
        mesa.mesa_residual_norm_backward(h, y, w, torch.zeros(3, 11))
    for call in (lambda: mesa.mesa_gate_norm(x, gate, torch.zeros(2, 16)), lambda: mesa.mesa_residual_norm(h, y, w)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()                                             # CPU tensors
