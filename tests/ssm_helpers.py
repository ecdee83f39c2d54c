"""Plain float64 forms of the state space layer's operators and of the rotation,
and the error bounds their tests share.

The scan runs token by token on the CPU with the state S [dv, dk]:
  D_t = softplus(dt_t + bias),  S_t = e^{A D_t} S_{t-1} + D_t x_t b_t^T,  o_t = S_t c_t + skip x_t.

Bounds, relative L2.  A float32 result of the scan or of its gradients is met with at
most 256 roundings of 2^-24 on its way: a chunk sums 64 pairs and up to 128 features,
a decay is off by its exponent's rounding (x 2^-24 of a power 2^x, at most 2^-24) and
the exponential's, and what a state carries from chunk to chunk only shrinks.  Sums
over heads, chunks and rows are in float64 or add a few.  F32 = 256 2^-24.
Where the rows are bfloat16, what feeds the state enters in three parts (2^-27 of a
term, below float32's rounding), what feeds outputs in two (2^-18, for two operands of
a chain 2^-17).  BF16 = 2^-8 (the output's rounding) + 2^-17 + F32.
Differences of sums (the step sizes' gradients, parameters' gradients) are held to
the same part of the terms they are made of.
"""
import numpy as np

from tests.delta_helpers import rel, store  # noqa: F401

F32 = 256 * 2.0 ** -24
BF16 = 2.0 ** -8 + 2.0 ** -17 + F32


def tol(t):
    return BF16 if str(t) in ("bf16", "torch.bfloat16") else F32


def near(got, ref, bound=None, terms=0.0, what=""):
    """got, a tensor, against ref: relative to ref's norm, or to that of the terms it is a sum of."""
    g, ref = got.double().cpu().numpy(), np.asarray(ref, np.float64)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all() or not np.isfinite(ref).all(), what
    size = max(float(np.linalg.norm(ref)), float(terms))
    e = float(np.linalg.norm(g - ref))
    bound = tol(got.dtype) if bound is None else bound
    assert e <= bound * size + 1e-30, (what, e / max(size, 1e-300), bound)


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-np.clip(x, -700, 700)))


def ssm_inputs(seed, B, Hk, H, T, dk, dv, dtype, start=True, lens=None, dt_dtype=None, fast=False):
    """Tensors in their storage types and their float64 values.  `fast`: decays of many
    powers of two a token among slow ones."""
    rng = np.random.default_rng(seed)
    t, f = {}, {}
    for n, shape in (("x", (B, H, T, dv)), ("b", (B, Hk, T, dk)), ("c", (B, Hk, T, dk))):
        t[n], f[n] = store(rng.standard_normal(shape), dtype)
    t["dt"], f["dt"] = store(rng.standard_normal((B, H, T)), dt_dtype or dtype)
    A = -np.exp(rng.uniform(np.log(0.2), np.log(16.0), H))
    if fast:
        A *= np.where(rng.random(H) < 0.5, 40.0, 0.02)
    for n, y in (("A", A), ("D", 1 + 0.3 * rng.standard_normal(H)), ("dt_bias", rng.uniform(-5.0, 0.0, H)),
                 ("state", 0.5 * rng.standard_normal((B, H, dv, dk)))):
        t[n], f[n] = store(y, "f32")
    if not start:
        t["state"], f["state"] = None, np.zeros((B, H, dv, dk))
    f["lens"] = [T] * B if lens is None else list(lens)
    if lens is not None:
        import torch
        t["lens"] = torch.tensor(f["lens"], dtype=torch.int32)
    else:
        t["lens"] = None
    return t, f


def ssm_ref(f, grad_out=None, grad_final=None, plus=True):
    """out and final state, and with grad_out the gradients of <out, grad_out> + <final,
    grad_final>, from the definition, a token at a time.  `terms` holds the sizes of what
    the step sizes' and parameters' gradients are sums of."""
    x, b, c, dt, A, skip, bias = (f[n] for n in ("x", "b", "c", "dt", "A", "D", "dt_bias"))
    B, H, T, dv = x.shape
    Hk, dk = b.shape[1], b.shape[3]
    r = H // Hk
    b, c = np.repeat(b, r, 1), np.repeat(c, r, 1)
    raw = dt + bias[:, None]
    step = softplus(raw) if plus else raw
    live = np.arange(T)[None, :] < np.asarray(f["lens"])[:, None]          # [B, T]
    step = np.where(live[:, None], step, 0.0)
    with np.errstate(under="ignore"):
        decay = np.exp(step * A[:, None])
    x, b, c = (np.where(live[:, None, :, None], y, 0.0) for y in (x, b, c))
    S = f["state"].copy()
    out, before = np.zeros((B, H, T, dv)), []
    for t in range(T):
        before.append(S)
        S = decay[:, :, t, None, None] * S + (step[:, :, t, None] * x[:, :, t])[..., None] * b[:, :, t, None, :]
        out[:, :, t] = (S * c[:, :, t, None, :]).sum(-1) + skip[:, None] * x[:, :, t]
    out = np.where(live[:, None, :, None], out, 0.0)
    if grad_out is None:
        return out, S
    g = {n: np.zeros(y.shape) for n, y in (("x", x), ("b", b), ("c", c), ("dt", dt))}
    terms_dt, dstep, dlog = np.zeros(dt.shape), np.zeros(dt.shape), np.zeros(dt.shape)
    R = np.zeros_like(S) if grad_final is None else grad_final.copy()
    after = S
    go = np.where(live[:, None, :, None], grad_out, 0.0)
    for t in reversed(range(T)):
        do, bt, ct, xt, st = go[:, :, t], b[:, :, t], c[:, :, t], x[:, :, t], step[:, :, t, None]
        g["c"][:, :, t] = (after * do[..., None]).sum(2)
        R = R + do[..., None] * ct[:, :, None, :]
        Rb, Rx = (R * bt[:, :, None, :]).sum(-1), (R * xt[..., None]).sum(2)
        g["x"][:, :, t] = st * Rb + skip[:, None] * do
        g["b"][:, :, t] = st * Rx
        dstep[:, :, t] = (Rb * xt).sum(-1)
        dlog[:, :, t] = (R * before[t]).sum((2, 3)) * decay[:, :, t]
        mix = np.abs(R * before[t]).sum((2, 3)) * decay[:, :, t]
        terms_dt[:, :, t] = (np.abs(Rb * xt)).sum(-1) + np.abs(A) * mix
        R = R * decay[:, :, t, None, None]
        after = before[t]
    slope = sigmoid(raw) if plus else np.ones_like(raw)
    on = live[:, None]
    graw = np.where(on, (dstep + A[:, None] * dlog) * slope, 0.0)
    tdt = np.where(on, terms_dt * slope, 0.0)
    fold = lambda y: y.reshape(B, Hk, r, T, dk).sum(2)  # noqa: E731
    grads = dict(grad_x=np.where(live[:, None, :, None], g["x"], 0.0), grad_b=fold(g["b"]), grad_c=fold(g["c"]), grad_dt=graw,
                 grad_A=(step * dlog).sum((0, 2)), grad_D=(go * x).sum((0, 2, 3)), grad_dt_bias=graw.sum((0, 2)),
                 grad_state=R)
    terms = dict(grad_dt=np.linalg.norm(tdt), grad_dt_bias=np.linalg.norm(tdt.sum((0, 2))),
                 grad_A=np.linalg.norm((tdt / np.maximum(slope, 1e-300) * step / np.maximum(np.abs(A[:, None]), 1e-300)).sum((0, 2))),
                 grad_D=np.linalg.norm(np.abs(go * x).sum((0, 2, 3))))
    return out, S, grads, terms


def conv_ref(x, w, bias=None, hist=None, lens=None, silu=True, dy=None):
    """y, the carried rows, and with dy the gradients."""
    B, T, D = x.shape
    W = w.shape[0]
    lens = [T] * B if lens is None else list(lens)
    past = np.zeros((B, W - 1, D)) if hist is None else hist
    full = np.concatenate([past, x], 1)
    live = (np.arange(T)[None, :] < np.asarray(lens)[:, None])[..., None]
    z = np.zeros((B, T, D)) + (0.0 if bias is None else bias)
    for j in range(W):
        z = z + w[j] * full[:, W - 1 - j:W - 1 - j + T]
    s = sigmoid(z) if silu else np.ones_like(z)
    y = np.where(live, z * s, 0.0)
    carried = np.stack([full[b, n:n + W - 1] for b, n in enumerate(lens)])
    if dy is None:
        return y, carried
    dz = np.where(live, dy * (s * (1.0 + z * (1.0 - s)) if silu else 1.0), 0.0)
    df = np.zeros_like(full)
    dw, terms = np.zeros_like(w), np.zeros_like(w)
    for j in range(W):
        df[:, W - 1 - j:W - 1 - j + T] += w[j] * dz
        part = dz * full[:, W - 1 - j:W - 1 - j + T]
        dw[j] = part.sum((0, 1))
        terms[j] = np.abs(part).sum((0, 1))
    return y, carried, dict(grad_x=df[:, W - 1:], grad_hist=df[:, :W - 1], grad_w=dw, grad_bias=dz.sum((0, 1))), dict(
        grad_w=np.linalg.norm(terms), grad_bias=np.linalg.norm(np.abs(dz).sum((0, 1))))


def rotate_ref(x, freqs, pos, w=None, norm=True, eps=1e-6, interleaved=False, amplitude=1.0, dy=None):
    """x [B, H, T, d], pos [B, T]: y, and with dy (dx, dw, the terms' norms).  Angles in long double."""
    rot, d = 2 * len(freqs), x.shape[-1]
    ang = (pos[:, None, :, None].astype(np.longdouble) * freqs.astype(np.longdouble))
    cos, sin = (amplitude * np.cos(ang)).astype(np.float64), (amplitude * np.sin(ang)).astype(np.float64)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))

    def turn(v, sign):
        y = v.copy()
        y[..., a] = v[..., a] * cos - sign * v[..., b] * sin
        y[..., b] = v[..., b] * cos + sign * v[..., a] * sin
        return y

    rs = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else 1.0
    u = x * rs
    y = turn(u if w is None else u * w, 1.0)
    if dy is None:
        return y
    g = turn(dy, -1.0)
    if not norm:
        return y, g, None, np.linalg.norm(g), 0.0
    du = g if w is None else g * w
    dx = rs * (du - u * (du * u).mean(-1, keepdims=True))
    return y, dx, (g * u).sum((0, 1, 2)), np.linalg.norm(rs * du), np.linalg.norm(np.abs(g * u).sum((0, 1, 2)))
