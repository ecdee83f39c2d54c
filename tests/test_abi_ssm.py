"""The entry points of the state space layer and of the rotation, on the CPU: their
workspace sizes, the rotation's frequencies, and what the calls refuse before they
touch the device.

The C calls get fake pointers (never dereferenced): every one fails validation.
"""
import ctypes
import math

import pytest

from test_regression_amd import mesa

OK, INVALID, UNSUPPORTED, WS_SMALL, HIPERR = range(5)
F32, BF16 = mesa.MESA_DTYPE_F32, mesa.MESA_DTYPE_BF16
BIG = 1 << 40


def S(*v):
    return (ctypes.c_int64 * len(v))(*v)


class P(int):
    """A tensor's fake address."""


def addresses(**kw):
    """The arguments with every tensor (None below) in 64 MiB of its own."""
    n, out = 0, {}
    for k, v in kw.items():
        if v is P:
            n += 1
            v = P((n + 16) << 26)
        out[k] = v
    return out


CONV = dict(x=P, xs=None, dtype=F32, w=P, width=4, bias=P, silu=1, hist=P)
SSM = dict(x=P, xs=None, b=P, bs=None, c=P, cs=None, dtype=F32, dt=P, dts=None, dt_dtype=F32, A=P, D=P, dt_bias=P, softplus=1)
ROT = dict(q=P, qs=None, k=P, ks=None, dtype=F32, freqs=P, rot=32, interleaved=0, amplitude=1.0, positions=P, pos_stride=5,
           position0=0, wq=P, wk=P, norm=1, eps=1e-6)
SIZES = dict(B=8, Hk=2, H=16, T=100, dk=64, dv=64)   # every tensor has 32 bytes or more
ENTRIES = {n: addresses(**a) for n, a in {
    "mesa_causal_conv": dict(CONV, hist_out=P, lens=P, B=8, T=5, D=40, y=P, stream=None),
    "mesa_causal_conv_backward": dict(CONV, lens=P, grad_y=P, B=8, T=5, D=40, grad_x=P, gxs=None, grad_w=P, grad_bias=P,
                                      grad_hist=P, workspace=P, workspace_bytes=BIG, stream=None),
    "mesa_ssm_forward": dict(SSM, state0=P, lens=P, **SIZES, out=P, final_state=P, workspace=P, workspace_bytes=BIG, stream=None),
    "mesa_ssm_backward": dict(SSM, state0=P, lens=P, grad_out=P, grad_final=P, **SIZES, grad_x=P, gxs=None, grad_b=P, gbs=None,
                              grad_c=P, gcs=None, grad_dt=P, gds=None, grad_A=P, grad_D=P, grad_dt_bias=P, grad_state=P,
                              workspace=P, workspace_bytes=BIG, stream=None),
    "mesa_ssm_step": dict(SSM, state=P, N=3, Hk=2, H=16, dk=64, dv=64, out=P, stream=None),
    "mesa_qk_rotate": dict(ROT, B=1, Hq=4, Hk=2, T=5, d=64, yq=P, yk=P, stream=None),
    "mesa_qk_rotate_backward": dict(ROT, grad_yq=P, grad_yk=P, B=1, Hq=4, Hk=2, T=5, d=64, grad_q=P, gqs=None, grad_k=P,
                                    gks=None, grad_wq=P, grad_wk=P, workspace=P, workspace_bytes=BIG, stream=None),
}.items()}


def call(name, **kw):
    a = dict(ENTRIES[name])
    assert set(kw) <= set(a), kw
    a.update(kw)
    L = mesa.lib()
    st = getattr(L, name)(*a.values())
    return st, L.mesa_last_error_message().decode()


def refused(name, status, needle, **kw):
    st, msg = call(name, **kw)
    assert st == status, (name, kw, st, msg)
    assert needle in msg, (name, kw, msg)


NULLS = {
    "mesa_causal_conv": "x w y",
    "mesa_causal_conv_backward": "x w grad_y grad_x grad_w workspace",
    "mesa_ssm_forward": "x b c dt A out",
    "mesa_ssm_backward": "x b c dt A grad_out grad_x grad_b grad_c grad_dt grad_A workspace",
    "mesa_ssm_step": "x b c dt A state out",
    "mesa_qk_rotate": "q k freqs yq yk",
    "mesa_qk_rotate_backward": "q k freqs grad_yq grad_yk grad_q grad_k",
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in NULLS.items() for a in args.split()])
def test_null_pointers(name, arg):
    refused(name, INVALID, "non-null", **{arg: None})


POINTERS = [(n, a) for n, args in ENTRIES.items() for a, v in args.items() if isinstance(v, P)]
# what may lie at any element (or word) of its type
STRIDED = ("x", "b", "c", "dt", "q", "k", "grad_x", "grad_b", "grad_c", "grad_dt", "grad_q", "grad_k")
WORDS = ("lens", "A", "D", "dt_bias", "grad_w", "grad_bias", "grad_A", "grad_D", "grad_dt_bias", "grad_wq", "grad_wk")


@pytest.mark.parametrize("name,arg", POINTERS)
def test_misaligned_pointers(name, arg):
    by = 2 if arg in STRIDED + WORDS else 4 if arg in ("freqs", "positions") else 8
    refused(name, INVALID, "misaligned", **{arg: ENTRIES[name][arg] + by})


@pytest.mark.parametrize("name", ["mesa_ssm_forward", "mesa_ssm_backward", "mesa_ssm_step"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INVALID, "dtype 2"), (dict(dt_dtype=-1), INVALID, "dt_dtype -1"),
    (dict(B=0), INVALID, "positive"), (dict(Hk=0), INVALID, "positive"), (dict(H=-4), INVALID, "positive"),
    (dict(T=-1), INVALID, "positive"), (dict(dk=0), INVALID, "positive"), (dict(dv=-16), INVALID, "positive"),
    (dict(H=3), INVALID, "multiple"), (dict(Hk=4, H=2), INVALID, "multiple"),
    (dict(dk=48), UNSUPPORTED, "dk=48"), (dict(dk=256), UNSUPPORTED, "dk=256"), (dict(dv=8), UNSUPPORTED, "dv=8"),
    (dict(dv=256), UNSUPPORTED, "dv=256"), (dict(B=1 << 20, H=1 << 10), INVALID, "grid too large"),
    (dict(B=1 << 30, H=1 << 30), INVALID, "grid too large"), (dict(B=1 << 14, T=(1 << 31) - 1), INVALID, "grid too large"),
    (dict(xs=S(-1, 64, 256)), INVALID, "strides of x must not be negative"),
    (dict(cs=S(1, -2, 64)), INVALID, "strides of c must not be negative"),
    (dict(bs=S(1 << 61, 1 << 61, 64)), INVALID, "strides of b are too large"),
])
def test_ssm_sizes(name, kw, status, needle):
    kw = dict(kw)
    if "step" in name:   # one token
        if "T" in kw:
            pytest.skip("the step has one token")
        if "B" in kw:
            kw["N"] = kw.pop("B")
        if needle.startswith("strides of x"):
            kw["xs"] = S(-1, 64)
    elif needle.startswith("strides of x"):
        kw["B"] = 2
    refused(name, status, needle, **kw)


def test_token_strides_past_what_the_kernels_address():
    for name in ("mesa_ssm_forward", "mesa_ssm_backward"):
        refused(name, UNSUPPORTED, "token stride of x", x=1 << 44, xs=S(0, 64, 1 << 23))
        refused(name, UNSUPPORTED, "token stride of b", b=1 << 44, bs=S(0, 64, 1 << 23))


@pytest.mark.parametrize("name", ["mesa_causal_conv", "mesa_causal_conv_backward"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), INVALID, "dtype 3"), (dict(B=0), INVALID, "positive"), (dict(T=-1), INVALID, "positive"),
    (dict(D=0), INVALID, "positive"), (dict(width=0), INVALID, "positive"), (dict(width=5), UNSUPPORTED, "width 5"),
    (dict(B=1 << 20, T=1 << 16), INVALID, "grid too large"), (dict(xs=S(40, -1)), INVALID, "negative"),
])
def test_conv_sizes(name, kw, status, needle):
    refused(name, status, needle, **kw)


@pytest.mark.parametrize("name", ["mesa_qk_rotate", "mesa_qk_rotate_backward"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=3), INVALID, "dtype 3"), (dict(B=0), INVALID, "positive"), (dict(Hq=0), INVALID, "positive"),
    (dict(Hk=-1), INVALID, "positive"), (dict(T=-1), INVALID, "positive"), (dict(d=48), UNSUPPORTED, "d=48"),
    (dict(rot=8), UNSUPPORTED, "rot=8"), (dict(rot=24), UNSUPPORTED, "rot=24"), (dict(rot=80), UNSUPPORTED, "rot=80"),
    (dict(rot=0), UNSUPPORTED, "rot=0"), (dict(eps=0.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=float("inf")), INVALID, "eps"), (dict(norm=0), INVALID, "need the norm"), (dict(Hk=0), INVALID, "Hk = 0"),
    (dict(Hk=0, k=None), INVALID, "Hk = 0"), (dict(amplitude=0.0), INVALID, "amplitude"),
    (dict(amplitude=float("nan")), INVALID, "amplitude"), (dict(pos_stride=-1), INVALID, "positions_stride"),
    (dict(B=1 << 20, T=1 << 12), INVALID, "grid too large"), (dict(qs=S(0, 64, -64)), INVALID, "negative"),
])
def test_rotate_sizes(name, kw, status, needle):
    refused(name, status, needle, **kw)


def test_optional_tensors_come_together():
    refused("mesa_causal_conv_backward", INVALID, "grad_bias", grad_bias=None)
    refused("mesa_causal_conv_backward", INVALID, "grad_bias", bias=None)
    for n in ("D", "dt_bias", "grad_D", "grad_dt_bias"):
        refused("mesa_ssm_backward", INVALID, "grad_D and grad_dt_bias", **{n: None})
    for n in ("wq", "wk", "grad_wq", "grad_wk"):
        refused("mesa_qk_rotate_backward", INVALID, "grad_wq and grad_wk", **{n: None})


OUTS = {
    "mesa_causal_conv": "y hist_out",
    "mesa_causal_conv_backward": "grad_x grad_w grad_bias grad_hist workspace",
    "mesa_ssm_forward": "out final_state",
    "mesa_ssm_backward": "grad_x grad_b grad_c grad_dt grad_A grad_D grad_dt_bias grad_state workspace",
    "mesa_ssm_step": "out state",
    "mesa_qk_rotate": "yq yk",
    "mesa_qk_rotate_backward": "grad_q grad_k grad_wq grad_wk workspace",
}
ALLOWED = {("mesa_causal_conv", "hist_out", "hist"), ("mesa_ssm_forward", "final_state", "state0"),
           ("mesa_ssm_backward", "grad_state", "grad_final")}
PAIRS = [(n, o, t) for n, outs in OUTS.items() for o in outs.split() for t, v in ENTRIES[n].items()
         if isinstance(v, P) and t != o and not (t == "workspace" and n == "mesa_ssm_forward")]


@pytest.mark.parametrize("name,out,other", PAIRS)
@pytest.mark.parametrize("by", [0, 16, -16])
def test_shared_memory_is_refused(name, out, other, by):
    if by == 0 and ((name, out, other) in ALLOWED or (name, other, out) in ALLOWED):
        pytest.skip("allowed")
    st, msg = call(name, **{out: ENTRIES[name][other] + by})
    assert st == INVALID and "alias" in msg and out in msg and other in msg, msg


def test_workspace_of_segments_is_not_shared():
    big = dict(B=1, T=64 * 100, H=2, workspace_bytes=BIG)
    a = ENTRIES["mesa_ssm_forward"]
    refused("mesa_ssm_forward", INVALID, "alias", **big, workspace=a["x"])
    refused("mesa_ssm_forward", INVALID, "alias", **big, workspace=a["out"])


def rows_of(name, width, T, **kw):
    """The gradients of x, b and c as slices of rows of one buffer."""
    base, e = 1 << 36, 4
    H, Hk, dk, dv = 4, 2, 64, 64
    a = dict(H=H, Hk=Hk, grad_x=base, gxs=S(T * width, dv, width), grad_b=base + e * H * dv, gbs=S(T * width, dk, width),
             grad_c=base + e * (H * dv + Hk * dk), gcs=S(T * width, dk, width), B=2, T=T, dk=dk, dv=dv)
    a.update(kw)
    return call(name, **a)


def test_slices_of_one_row_are_told_apart():
    width, T = 4 * 64 + 4 * 64, 100
    # in order: the call gets as far as the first output that does share memory
    probe = dict(grad_A=ENTRIES["mesa_ssm_backward"]["A"])
    st, msg = rows_of("mesa_ssm_backward", width, T, **probe)
    assert st == INVALID and "grad_A must not alias A" in msg, msg
    # one element too far to the left, and rows that are too short
    st, msg = rows_of("mesa_ssm_backward", width, T, grad_b=(1 << 36) + 4 * (4 * 64 - 1), **probe)
    assert st == INVALID and "grad_b must not alias grad_x" in msg, msg
    st, msg = rows_of("mesa_ssm_backward", width - 1, T, **probe)
    assert st == INVALID and ("alias" in msg or "share memory" in msg) and "grad_A" not in msg, msg
    # heads of one buffer [B, 4 + 2 + 2, T, 64]
    n = T * 64
    st, msg = rows_of("mesa_ssm_backward", width, T, gxs=S(8 * n, n, 64), grad_b=(1 << 36) + 16 * n, gbs=S(8 * n, n, 64),
                      grad_c=(1 << 36) + 24 * n, gcs=S(8 * n, n, 64), **probe)
    assert st == INVALID and "grad_A must not alias A" in msg, msg


def test_rows_of_an_output_that_share_memory():
    refused("mesa_ssm_backward", INVALID, "rows of grad_x must not share memory", gxs=S(0, 64, 64))
    refused("mesa_ssm_backward", INVALID, "rows of grad_dt must not share memory", gds=S(100, 1, 3))
    refused("mesa_qk_rotate_backward", INVALID, "rows of grad_q must not share memory", gqs=S(1 << 20, 0, 64))
    refused("mesa_causal_conv_backward", INVALID, "rows of grad_x must not share memory", gxs=S(200, 39))
    refused("mesa_ssm_backward", INVALID, "rows of grad_c must not share memory", gcs=S(0, 6400, 64))


@pytest.mark.parametrize("name,need", [
    ("mesa_causal_conv_backward", lambda: mesa.lib().mesa_causal_conv_backward_workspace_bytes(8, 5, 40, 4)),
    ("mesa_qk_rotate_backward", lambda: mesa.lib().mesa_qk_rotate_backward_workspace_bytes(64)),
])
def test_small_workspaces(name, need):
    n = need()
    assert n > 0
    refused(name, WS_SMALL, f"{n} needed", workspace_bytes=n - 1)
    refused(name, WS_SMALL, f"{n} needed", workspace_bytes=0)


def test_workspaces_grow_and_hold_what_the_calls_take():
    """A workspace for the largest of a run of sizes serves all of them: the calls go on to the aliases."""
    f, b, c = (mesa.mesa_ssm_workspace_bytes, mesa.mesa_ssm_backward_workspace_bytes,
               mesa.lib().mesa_causal_conv_backward_workspace_bytes)
    A = ENTRIES["mesa_ssm_backward"]["A"]
    for dv in (16, 128):
        for H in (1, 2, 5, 16, 40, 600):
            sizes = [f(1, H, 64 * n - 3, 64, dv, BF16) for n in range(1, 120)]
            assert sizes == sorted(sizes)
            for n in range(1, 120, 7):
                _, msg = call("mesa_ssm_forward", B=1, Hk=1, H=H, T=64 * n - 3, dv=dv, out=A, workspace_bytes=sizes[-1], dtype=BF16)
                assert "alias" in msg, msg
            sizes = [b(1, 1, H, 64 * n - 3, 64, dv, BF16) for n in range(1, 120)]
            assert sizes == sorted(sizes)
            for n in range(1, 120, 7):
                _, msg = call("mesa_ssm_backward", B=1, Hk=1, H=H, T=64 * n - 3, dv=dv, grad_A=A, workspace_bytes=sizes[-1], dtype=BF16)
                assert "alias" in msg, msg
        for n in (1, 16, 33, 64, 500):
            sizes = [f(B, 3, 64 * n, 64, dv, F32) for B in range(1, 200)]
            assert sizes == sorted(sizes)
            sizes = [b(B, 1, 3, 64 * n, 64, dv, F32) for B in range(1, 200)]
            assert sizes == sorted(sizes)
            for B in range(1, 200, 9):
                for name, size in (("mesa_ssm_forward", f(199, 3, 64 * n, 64, dv, F32)), ("mesa_ssm_backward", sizes[-1])):
                    kw = dict(out=A) if name.endswith("forward") else dict(grad_A=A)
                    _, msg = call(name, B=B, Hk=1, H=3, T=64 * n, dv=dv, workspace_bytes=size, **kw)
                    assert "alias" in msg, msg
    sizes = [c(2, T, 40, 4) for T in range(1, 3000, 5)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert f(0, 1, 1, 64, 64, F32) == b(1, 2, 3, 64, 64, 64, F32) == c(1, 0, 8, 4) == f(1, 1, 64, 64, 64, 5) == 0


def test_kernel_names():
    ids = range(mesa.KERNEL_CAUSAL_CONV, mesa.KERNEL_QK_ROTATE_BWD + 1)
    names = [mesa.kernel_name(i) for i in ids]
    assert len(set(names)) == 8 and all(n.startswith(("causal_conv", "ssm_", "qk_rotate")) for n in names)
    for i in ids:
        assert mesa.profile_read(i) == (0.0, 0)
    for i in (*range(25, 32), ids[-1] + 1):
        with pytest.raises(ValueError, match="kernel id"):
            mesa.profile_read(i)


# ---- the rotation's frequencies ----
def test_frequencies():
    f, amp = mesa.mesa_rotary_frequencies(64, 500.0, device="cpu")
    assert amp == 1.0 and f.dtype is torch.float64
    assert f.tolist() == pytest.approx([500.0 ** (-2 * i / 64) for i in range(32)], rel=1e-15)
    lin, amp = mesa.mesa_rotary_frequencies(64, 500.0, mesa.MESA_ROTARY_LINEAR, 4.0, device="cpu")
    assert amp == 1.0 and lin.tolist() == pytest.approx((f / 4).tolist(), rel=1e-15)
    ntk, amp = mesa.mesa_rotary_frequencies(64, 500.0, mesa.MESA_ROTARY_BASE, 4.0, device="cpu")
    assert amp == 1.0 and ntk[0] == f[0] and ntk[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-13)
    assert bool((ntk[1:] < f[1:]).all())
    mix, amp = mesa.mesa_rotary_frequencies(64, 10000.0, mesa.MESA_ROTARY_PARTS, 8.0, 4096.0, 32.0, 1.0, device="cpu")
    f, _ = mesa.mesa_rotary_frequencies(64, device="cpu")
    assert amp == pytest.approx(1 + 0.1 * math.log(8.0), rel=1e-6)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(mix[turns > 32], f[turns > 32]) and torch.allclose(mix[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    between = (turns >= 1) & (turns <= 32)
    keep = (turns - 1) / 31
    assert bool(between.any()) and torch.allclose(mix[between], (f * keep + f / 8 * (1 - keep))[between], rtol=1e-14)


@pytest.mark.parametrize("args,needle", [
    ((0,), "rot=0"), ((15,), "rot=15"), ((16, 1.0), "base"), ((16, float("inf")), "base"), ((16, float("nan")), "base"),
    ((16, 1e4, 4), "scaling 4"), ((16, 1e4, -1), "scaling -1"), ((16, 1e4, 0, 2.0), "without scaling"),
    ((16, 1e4, 1, 0.5), "factor"), ((16, 1e4, 1, float("nan")), "factor"), ((2, 1e4, 2, 2.0), "slowest"),
    ((16, 1e4, 3, 2.0, 0.0), "context"), ((16, 1e4, 3, 2.0, 100.0, 1.0, 1.0), "fast"), ((16, 1e4, 3, 2.0, 100.0, 1.0, -1.0), "slow"),
])
def test_frequencies_refused(args, needle):
    with pytest.raises(ValueError, match=needle):
        mesa.mesa_rotary_frequencies(*args, device="cpu")


# ---- the Python calls ----
torch = pytest.importorskip("torch")


def ssm_tensors(step=False):
    z = torch.zeros
    t = dict(x=z(2, 4, 5, 32), b=z(2, 2, 5, 16), c=z(2, 2, 5, 16), dt=z(2, 4, 5), A=z(4), D=z(4), dt_bias=z(4), state=z(2, 4, 32, 16))
    return {n: v[:, :, 0].contiguous() if step and n in ("x", "b", "c", "dt") else v for n, v in t.items()}


def ssm_call(kind, **kw):
    t = ssm_tensors(kind == "step")
    t.update({n: v for n, v in kw.items() if n in t})
    rest = {n: v for n, v in kw.items() if n not in t}
    a = [t[n] for n in ("x", "b", "c", "dt", "A")]
    if kind == "step":
        return mesa.mesa_ssm_step(*a, t["state"], t["D"], t["dt_bias"], **rest)
    if kind == "backward":
        a.append(rest.pop("grad_out", torch.zeros(2, 4, 5, 32)))
    return getattr(mesa, "mesa_ssm_" + kind)(*a, t["D"], t["dt_bias"], t["state"], **rest)


@pytest.mark.parametrize("kind", ["forward", "backward", "step"])
def test_ssm_calls_refuse_wrong_arguments(kind):
    bad = (ValueError, TypeError)
    good = ssm_tensors(kind == "step")
    for n, v in good.items():
        with pytest.raises(bad, match="must have shape|dimension|multiple"):
            ssm_call(kind, **{n: torch.zeros(*v.shape[:-1], v.shape[-1] + 16)})
        with pytest.raises(bad):
            ssm_call(kind, **{n: v[0]})
        with pytest.raises(bad):
            ssm_call(kind, **{n: v.half()})
    with pytest.raises(ValueError, match="multiple"):
        ssm_call(kind, x=good["x"][:, :3])
    with pytest.raises(ValueError, match="device tensor"):
        ssm_call(kind)
    if kind != "step":
        with pytest.raises(ValueError, match="lens must have shape|device tensor"):
            ssm_call(kind, lens=torch.zeros(3, dtype=torch.int32))
    if kind == "backward":
        for n in ("grad_out", "grad_final", "grad_x", "grad_b", "grad_c", "grad_dt"):
            with pytest.raises(bad):
                ssm_call(kind, **{n: torch.zeros(1, 4, 3)})


def test_conv_and_rotate_calls_refuse_wrong_arguments():
    bad = (ValueError, TypeError)
    x, w, b = torch.zeros(2, 5, 12), torch.zeros(4, 12), torch.zeros(12)
    for args in [(x[0], w, b), (x, torch.zeros(4, 11), b), (x, w, torch.zeros(11)), (x, w, b, torch.zeros(2, 4, 12)), (x.half(), w, b),
                 (x.transpose(1, 2), torch.zeros(4, 5), torch.zeros(5)), (x, w, b)]:
        with pytest.raises(bad):
            mesa.mesa_causal_conv(*args)
    with pytest.raises(bad):
        mesa.mesa_causal_conv_backward(x, w, torch.zeros(2, 5, 11), b)
    q, k, f = torch.zeros(2, 4, 5, 32), torch.zeros(2, 2, 5, 32), torch.zeros(8, dtype=torch.float64)
    for a in [(q[0], k, f), (q, k[..., :16], f), (q, k, f.float()), (q, k.half(), f), (q, k, f, torch.zeros(2, 5)), (q, k, f),
              (q, k, f, torch.zeros(2, 4, dtype=torch.int64))]:
        with pytest.raises(bad):
            mesa.mesa_qk_rotate(*a)
    with pytest.raises(bad):
        mesa.mesa_qk_rotate_backward(q, k, q, None, f)
