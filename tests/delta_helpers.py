"""Plain float64 forms of the gated delta rule and of the norms around a layer,
and the error bounds their tests share.

The delta rule runs token by token on the CPU with the state S [dv, dk]:
  S_t = g_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   o_t = S_t q_t.

Bounds.  A rounding to bfloat16 is off by at most 2^-8 of the value, one to
float32 by 2^-24.  The library's products carry at most 3 2^-22 a term (two-part
splits) and sum in float32; a chunk passes a value through four such products
and the float32 inverse of a 64 x 64 unit triangle, and a state contracts from
chunk to chunk.  Counting 3 2^-22 for each of the four, as much again for the
inverse (64 steps of 2^-24 each) and the decays' 2^-23, and the same for the
state that came before, gives 2 (4 * 3 2^-22 + 64 2^-24 + 2^-23) = 1.4e-5 of the
largest magnitudes met; F32 = 1.5e-5 bounds relative L2 errors of float32 results.
bfloat16 results add their rounding and, for the outputs, two products of 11-bit
operands (3 2^-12 a term): BF16 = 2^-8 + 3 2^-12 + F32 bounds their relative L2
error (typical: 1.7e-3, roundings being spread evenly below half a step).
"""
import numpy as np

F32 = 1.5e-5
BF16 = 2.0 ** -8 + 3 * 2.0 ** -12 + F32


def tol(dtype):
    return BF16 if dtype == "bf16" else F32


def rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.linalg.norm(a))


def unit_rows(rng, *shape):
    """Unit rows whose neighbours are related (a short convolution's outputs)."""
    x = rng.standard_normal((*shape[:-2], shape[-2] + 2, shape[-1]))
    x = x[..., 2:, :] + 0.5 * x[..., 1:-1, :] + 0.2 * x[..., :-2, :]
    return x / np.linalg.norm(x, axis=-1, keepdims=True)


def store(x, dtype):
    """A CPU tensor in the storage type, and the float64 values it holds."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.double().numpy()


def delta_inputs(seed, B, Hk, H, T, dk, dv, dtype, start=True, lo=0.8):
    rng = np.random.default_rng(seed)
    x = dict(q=unit_rows(rng, B, Hk, T, dk), k=unit_rows(rng, B, Hk, T, dk), v=rng.standard_normal((B, H, T, dv)))
    t, f = {}, {}
    for n in x:
        t[n], f[n] = store(x[n], dtype)
    for n, y in (("gamma", rng.uniform(lo, 1.0, (B, H, T))), ("beta", rng.uniform(0.0, 1.0, (B, H, T))),
                 ("state", rng.standard_normal((B, H, dv, dk)) * 0.3)):
        t[n], f[n] = store(y, "f32")
    if not start:
        t["state"], f["state"] = None, np.zeros((B, H, dv, dk))
    return t, f


def delta_ref(f, grad_out=None, grad_final=None):
    """out, final state (and with grad_out the gradients of sum(out grad_out) +
    sum(final grad_final)) in float64, from the definition."""
    q, k, v, gamma, beta, S = (f[n] for n in ("q", "k", "v", "gamma", "beta", "state"))
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    r = H // Hk
    qh, kh = np.repeat(q, r, 1), np.repeat(k, r, 1)
    out = np.zeros((B, H, T, dv))
    S = S.copy()
    before = []
    for t in range(T):
        before.append(S)
        g, b, kt = gamma[:, :, t, None, None], beta[:, :, t, None, None], kh[:, :, t, None, :]
        S = g * S
        S = S - b * (S * kt).sum(-1, keepdims=True) * kt + b * v[:, :, t, :, None] * kt
        out[:, :, t] = (S * qh[:, :, t, None, :]).sum(-1)
    if grad_out is None:
        return out, S
    dS = np.zeros_like(S) if grad_final is None else grad_final.copy()
    dq, dk_, dv_ = np.zeros((B, H, T, dk)), np.zeros((B, H, T, dk)), np.zeros((B, H, T, dv))
    dg, db = np.zeros((B, H, T)), np.zeros((B, H, T))
    for t in reversed(range(T)):
        g, b = gamma[:, :, t, None, None], beta[:, :, t, None, None]
        kt, qt, do = kh[:, :, t, None, :], qh[:, :, t, None, :], grad_out[:, :, t, :, None]
        Sd = g * before[t]
        e = v[:, :, t, :, None] - (Sd * kt).sum(-1, keepdims=True)
        dq[:, :, t] = (do * (Sd + b * e * kt)).sum(2)
        dS = dS + do * qt
        de = b * (dS * kt).sum(-1, keepdims=True)
        dv_[:, :, t] = de[..., 0]
        db[:, :, t] = (dS * e * kt).sum((2, 3))
        dk_[:, :, t] = (dS * b * e).sum(2) - (de * Sd).sum(2)
        dS = dS - de * kt
        dg[:, :, t] = (dS * before[t]).sum((2, 3))
        dS = g * dS
    shared = lambda x: x.reshape(B, Hk, r, T, dk).sum(2)  # noqa: E731
    return out, S, dict(grad_q=shared(dq), grad_k=shared(dk_), grad_v=dv_, grad_gamma=dg, grad_beta=db, grad_state=dS)
