"""Cases of the library's selective state space layer and of its query and key rotation, for timing and for
comparing outputs.

The layer's short causal convolution runs over the rows of an input projection, per channel:

    y_t = silu(sum_{j<W} w_j x_{t-j} + bias),

and its state space scan keeps, per batch row and head, a state S (dv x dk) that decays by what the token says:

    D_t = softplus(dt_t + dt_bias),   S_t = exp(A D_t) S_{t-1} + D_t x_t b_t^T,   o_t = S_t c_t + D x_t,

over whole prompts of different lengths, as its gradients, and one token at a time.  b and c play the key's and
the query's part, and several heads may share them.  The rotation takes the RMS norm of each head's queries and
keys (or of b and c) and turns their pairs of features by an angle that grows with the token's position.

With `own` false, run() computes these from elementary torch operations in float32 (the angles in float64); with
`own` true it calls the library.  exact() computes them in float64, the scan token by token.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64          # tokens per chunk of the plain form
DIMS = (16, 32, 64, 128)
EPS = 1e-6


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def listed():
    return [
        # the convolution of one layer in a training step: forward and gradients, over x, b and c together
        dict(name="conv_train", op="conv", dtype="bf16", B=8, T=4096, D=2304, W=4, hist=False, lens=False, grad=True),
        # one decoded token for each of the benchmark's 256 sequences, the carried rows updated in place
        dict(name="conv_decode", op="conv", dtype="bf16", B=256, T=1, D=2304, W=4, hist=True, lens=False, grad=False),
        # the scan of one layer over the benchmark's headline batch
        dict(name="ssm_layer", op="ssm", dtype="bf16", B=8, Hk=1, H=32, T=4096, dk=128, dv=64, start=False, lens=False),
        # one long prompt taken on from a carried state
        dict(name="ssm_prompt", op="ssm", dtype="bf16", B=1, Hk=2, H=16, T=16384, dk=128, dv=128, start=True,
             lens=False),
        # three short prompts of different lengths in float32, padded to one batch: a call whose latency counts
        dict(name="ssm_short", op="ssm", dtype="f32", B=3, Hk=1, H=4, T=100, dk=64, dv=64, start=False, lens=True),
        # the gradients of a layer in a training step
        dict(name="ssm_grad_layer", op="ssm_grad", dtype="bf16", B=2, Hk=1, H=32, T=4096, dk=128, dv=64, start=False,
             lens=False),
        # the gradients in float32 of an odd length, through the carried and the final state of a padded batch
        dict(name="ssm_grad_ragged", op="ssm_grad", dtype="f32", B=2, Hk=2, H=8, T=1023, dk=64, dv=128, start=True,
             lens=True),
        # one decoded token for each of the benchmark's 256 sequences
        dict(name="ssm_step_batch", op="ssm_step", dtype="bf16", N=256, Hk=1, H=32, dk=128, dv=64),
        # one decoded token of one sequence
        dict(name="ssm_step_one", op="ssm_step", dtype="f32", N=1, Hk=1, H=4, dk=64, dv=64),
        # queries and keys of a layer in a training step, normed and rotated: forward and gradients
        dict(name="rotate_train", op="rotate", dtype="bf16", B=8, Hq=16, Hk=4, T=4096, d=128, rot=128,
             interleaved=False, norm=True, far=False, grad=True),
        # one decoded token of 256 sequences at far positions of a stretched context
        dict(name="rotate_decode", op="rotate", dtype="bf16", B=256, Hq=16, Hk=4, T=1, d=128, rot=128,
             interleaved=False, norm=True, far=True, grad=False),
        # a part of each head in neighbouring pairs, float32, an odd length, without a norm
        dict(name="rotate_part", op="rotate", dtype="f32", B=3, Hq=8, Hk=8, T=1023, d=64, rot=32, interleaved=True,
             norm=False, far=False, grad=True),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["conv", "ssm", "ssm", "ssm_grad", "ssm_grad", "ssm_step", "rotate"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "conv":
        B, D = _log(rng, 1, 64), _log(rng, 4, 640) * 8
        D -= rng.choice([0, 0, 0, 1, 3])
        return dict(op=op, dtype=dtype, B=B, T=max(1, min(_log(rng, 1, 8192), 8 * 4096 * 2304 // (2 * B * D))), D=D,
                    W=rng.choice([2, 3, 4]), hist=rng.random() < 0.5, lens=rng.random() < 0.3, grad=rng.random() < 0.6)
    if op in ("ssm", "ssm_grad"):
        Hk = _log(rng, 1, 4)
        H = Hk * rng.choice([1, 2, 4, 7, 8])
        dk, dv, T, B = rng.choice(DIMS), rng.choice(DIMS), _log(rng, 1, 8192), _log(rng, 1, 8)
        # at most the work of the listed layer
        most = (16 if op == "ssm" else 4) * 16 * 4096 * 128 * 64 // 2
        while B * H * T * dk * dv > most:
            if B > 1:
                B //= 2
            else:
                T //= 2
        return dict(op=op, dtype=dtype, B=B, Hk=Hk, H=H, T=T, dk=dk, dv=dv, start=rng.random() < 0.5,
                    lens=rng.random() < 0.3)
    if op == "ssm_step":
        Hk = _log(rng, 1, 4)
        return dict(op=op, dtype=dtype, N=_log(rng, 1, 128), Hk=Hk, H=Hk * rng.choice([1, 4, 5, 8]),
                    dk=rng.choice(DIMS), dv=rng.choice(DIMS))
    d = rng.choice([32, 64, 128, 256])
    B, Hq = _log(rng, 1, 64), _log(rng, 1, 32)
    Hk = rng.choice([x for x in range(1, Hq + 1) if Hq % x == 0])
    return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, T=max(1, min(_log(rng, 1, 8192), 8 * 20 * 4096 * 128 // (2 * B * (Hq + Hk) * d))),
                d=d, rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.6,
                far=rng.random() < 0.5, grad=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """Angles per token of the rotated pairs, float64, and the factor on the rotation.  Far positions come with a
    context stretched 8 times: slow pairs are slowed down by that, fast ones are left, those between are mixed."""
    n = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if not case["far"]:
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)                       # of the original context
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (scale * torch.randn(shape, generator=g, device=DEV)).to(dtype)

    def lengths(B, T):
        n = torch.randint(T // 2, T + 1, (B,), generator=g, device=DEV)
        return n.to(torch.int32)

    def step_sizes(H):
        """A and dt_bias as such layers start: step sizes over (0.001, 0.1), decays of 1 to 16 a unit step."""
        A = -(1.0 + 15.0 * torch.rand((H,), generator=g, device=DEV))
        d = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((H,), generator=g, device=DEV))
        return A, d + torch.log(-torch.expm1(-d))

    c, dt, s = case, _dt(case["dtype"]), dict(case=case)
    if c["op"] == "conv":
        B, T, D, W = (c[n] for n in ("B", "T", "D", "W"))
        s["x"] = normal(B, T, D, dtype=dt)
        s["w"], s["bias"] = normal(W, D, scale=W ** -0.5), normal(D, scale=0.1)
        s["hist"] = normal(B, W - 1, D, dtype=dt) if c["hist"] else None
        s["lens"] = lengths(B, T) if c["lens"] else None
        s["grad_y"] = normal(B, T, D, dtype=dt) if c["grad"] else None
    elif c["op"] in ("ssm", "ssm_grad"):
        B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        # the rows of the convolution's output: x, b and c of a token side by side
        rows = normal(B, T, H * dv + 2 * Hk * dk)
        s["rows"] = (rows / (1.0 + torch.exp(-rows))).to(dt)
        s["dt"] = normal(B, T, H, dtype=dt)
        s["A"], s["dt_bias"] = step_sizes(H)
        s["D"] = 1.0 + normal(H, scale=0.1)
        s["state"] = normal(B, H, dv, dk, scale=0.3) if c["start"] else None
        s["lens"] = lengths(B, T) if c["lens"] else None
        if c["op"] == "ssm_grad":
            s["grad_out"] = normal(B, H, T, dv, dtype=dt)
            s["grad_final"] = normal(B, H, dv, dk, scale=0.3) if c["start"] else None
    elif c["op"] == "ssm_step":
        N, Hk, H, dk, dv = (c[n] for n in ("N", "Hk", "H", "dk", "dv"))
        rows = normal(N, H * dv + 2 * Hk * dk)
        s["rows"] = (rows / (1.0 + torch.exp(-rows))).to(dt)
        s["dt"] = normal(N, H, dtype=dt)
        s["A"], s["dt_bias"] = step_sizes(H)
        s["D"] = 1.0 + normal(H, scale=0.1)
        s["state"] = normal(N, H, dv, dk, scale=0.3)
    else:
        B, Hq, Hk, T, d = (c[n] for n in ("B", "Hq", "Hk", "T", "d"))
        # the rows of a projection: the queries and keys of a token side by side
        s["rows"] = normal(B, T, (Hq + Hk) * d, dtype=dt)
        far = 60000 if c["far"] else 0
        first = torch.randint(0, far + 1, (B, 1), generator=g, device=DEV)
        s["positions"] = first + torch.arange(T, device=DEV)
        f, s["amplitude"] = _frequencies(c)
        s["freqs"] = f.to(DEV)
        s["wq"], s["wk"] = (1.0 + normal(d, scale=0.1), 1.0 + normal(d, scale=0.1)) if c["norm"] else (None, None)
        s["grad_q"] = normal(B, Hq, T, d, dtype=dt) if c["grad"] else None
        s["grad_k"] = normal(B, Hk, T, d, dtype=dt) if c["grad"] else None
    return s


def _split(rows, H, dv, Hk, dk):
    """x, b and c of the rows, by head, as views."""
    lead, a, n = rows.shape[:-1], H * dv, Hk * dk
    x = rows[..., :a].unflatten(-1, (H, dv))
    b = rows[..., a:a + n].unflatten(-1, (Hk, dk))
    c = rows[..., a + n:].unflatten(-1, (Hk, dk))
    return [t.transpose(1, 2) if len(lead) == 2 else t for t in (x, b, c)]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _valid(lens, B, T):
    """[B, T] truth values: the tokens that a row has."""
    at = torch.arange(T, device=DEV)
    return at < (torch.full((B, 1), T, device=DEV) if lens is None else lens[:, None])


# ---------------------------------------------------------------- the plain forms

def _conv(s):
    x, w, bias, hist, lens, dy = (s[n] for n in ("x", "w", "bias", "hist", "lens", "grad_y"))
    B, T, D = x.shape
    W = w.shape[0]
    if own:
        from test_regression_amd import mesa
        if hist is None:
            r = dict(y=mesa.mesa_causal_conv(x, w, bias, lens=lens))
        else:
            y, h = mesa.mesa_causal_conv(x, w, bias, hist, lens=lens, hist_out=hist if dy is None else None, return_hist=True)
            r = dict(y=y, hist=h)
        if dy is not None:
            g = mesa.mesa_causal_conv_backward(x, w, dy, bias, hist, lens=lens)
            r.update({k: v for k, v in g.items() if v is not None})
        return r
    past = torch.zeros((B, W - 1, D), device=DEV) if hist is None else hist.float()
    full = torch.cat([past, x.float()], 1)
    live = _valid(lens, B, T)[..., None]
    z = bias + sum(w[j] * full[:, W - 1 - j:W - 1 - j + T] for j in range(W))
    sig = 1.0 / (1.0 + torch.exp(-z))
    r = dict(y=torch.where(live, z * sig, 0.0).to(x.dtype))
    if hist is not None:
        end = torch.full((B,), T, device=DEV) if lens is None else lens
        at = end[:, None].long() + torch.arange(W - 1, device=DEV)
        last = full.gather(1, at[..., None].expand(B, W - 1, D)).to(x.dtype)
        r["hist"] = last if dy is not None else hist.copy_(last)
    if dy is not None:
        dz = torch.where(live, dy.float() * sig * (1.0 + z * (1.0 - sig)), 0.0)
        pad = torch.nn.functional.pad(dz, [0, 0, W - 1, W - 1])
        df = sum(w[j] * pad[:, j:j + T + W - 1] for j in range(W))       # of the carried rows and x
        r["grad_x"] = df[:, W - 1:].to(x.dtype)
        r["grad_w"] = torch.stack([(dz * full[:, W - 1 - j:W - 1 - j + T]).sum((0, 1)) for j in range(W)])
        r["grad_bias"] = dz.sum((0, 1))
        if hist is not None:
            r["grad_hist"] = df[:, :W - 1].to(x.dtype)
    return r


class _Chunked:
    """The scan in chunks, float32.  Per chunk with start state S (dk x dv here), the prefix sums L of the log
    decays and L_ij = exp(L_i - L_j) (j <= i), P_ij = L_ij (c_i . b_j) and X = diag(D) x:
        O = P X + diag(exp L) C S,   S' = exp(L_C) S + (diag(exp(L_C - L)) B)^T X."""

    def __init__(self, s):
        c = s["case"]
        B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        self.case, self.rep, self.n = c, H // Hk, -(-T // CHUNK)
        self.live = _valid(s["lens"], B, T)
        n = self.n

        def chunks(x):
            x = torch.nn.functional.pad(x, [0, 0] * (x.dim() - 3) + [0, n * CHUNK - T])
            return x.reshape(B * H, n, CHUNK, *x.shape[3:])

        live = self.live[:, None, :, None]
        x, b, cc = (torch.where(live, t.float(), 0.0) for t in _split(s["rows"], H, dv, Hk, dk))
        self.x, self.b, self.c = chunks(x), chunks(b.repeat_interleave(self.rep, 1)), chunks(cc.repeat_interleave(self.rep, 1))
        raw = s["dt"].float().transpose(1, 2) + s["dt_bias"][:, None]
        self.raw = chunks(raw)
        step = raw.clamp(min=0.0) + torch.log1p(torch.exp(-raw.abs()))
        self.step = chunks(torch.where(self.live[:, None], step, 0.0))
        self.A = s["A"].repeat(B)[:, None, None]
        self.L = (self.step * self.A).double().cumsum(-1)
        low = torch.ones((CHUNK, CHUNK), device=DEV).tril()
        self.D = torch.exp((self.L[..., :, None] - self.L[..., None, :]).clamp(max=0.0)).float() * low
        self.G, self.end = self.L.exp().float(), torch.exp(self.L[..., -1:] - self.L).float()
        self.CB = self.c @ self.b.transpose(-1, -2)
        self.skip = s["D"].repeat(B)[:, None, None, None]
        self.S0 = (torch.zeros((B * H, dk, dv), device=DEV) if s["state"] is None
                   else s["state"].reshape(B * H, dv, dk).transpose(1, 2))

    def whole(self, x, heads=None):
        c = self.case
        x = x.reshape(c["B"], heads or c["H"], self.n * CHUNK, *x.shape[3:])[:, :, :c["T"]]
        return x

    def states(self):
        S, kept = self.S0, []
        add = (self.b * (self.end * self.step)[..., None]).transpose(-1, -2) @ self.x
        for i in range(self.n):
            kept.append(S)
            S = self.G[:, i, -1, None, None] * S + add[:, i]
        return torch.stack(kept, 1), S

    def forward(self):
        c = self.case
        S, final = self.states()
        o = (self.D * self.CB) @ (self.step[..., None] * self.x) + self.G[..., None] * (self.c @ S) + self.skip * self.x
        return self.whole(o), final.transpose(1, 2).reshape(c["B"], c["H"], c["dv"], c["dk"])

    def backward(self, grad_out, grad_final):
        c = self.case
        B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        S, _ = self.states()
        do = torch.where(self.live[:, None, :, None], grad_out.float(), 0.0)
        do = torch.nn.functional.pad(do, [0, 0, 0, self.n * CHUNK - T]).reshape(B * H, self.n, CHUNK, dv)
        R = torch.zeros_like(self.S0) if grad_final is None else grad_final.reshape(B * H, dv, dk).transpose(1, 2)
        add, kept = (self.G[..., None] * self.c).transpose(-1, -2) @ do, [None] * self.n
        for i in reversed(range(self.n)):
            kept[i] = R
            R = self.G[:, i, -1, None, None] * R + add[:, i]
        dS = R
        R = torch.stack(kept, 1)
        dM = do @ self.x.transpose(-1, -2)
        Z = self.D * dM * self.step[..., None, :]
        read, write = self.G[..., None] * (do @ S.transpose(-1, -2)), self.end[..., None] * (self.x @ R.transpose(-1, -2))
        dc, db = Z @ self.b + read, Z.transpose(-1, -2) @ self.c + self.step[..., None] * write
        v = (self.D * self.CB).transpose(-1, -2) @ do + self.end[..., None] * (self.b @ R)
        dx = self.step[..., None] * v + self.skip * do
        # a token's decay scales every pair around it, what is read after it, what was written before it, the carry
        E = (Z * self.CB).double().tril(-1)
        cross = E.sum(-2) - E.sum(-1)
        cross = cross.cumsum(-1) - cross
        rd = (read.double() * self.c).sum(-1).flip(-1).cumsum(-1).flip(-1)
        wr = self.step * (write.double() * self.b).sum(-1)
        wr = wr.cumsum(-1) - wr
        carry = self.G[..., -1:] * (S.double() * R).sum((-1, -2))[..., None]
        da = cross + rd + wr + carry                                  # of the log decay
        live = self.live.repeat_interleave(H, 0).float()
        live = torch.nn.functional.pad(live, [0, self.n * CHUNK - T]).reshape(B * H, self.n, CHUNK)
        draw = ((v.double() * self.x).sum(-1) + self.A * da) / (1.0 + torch.exp(-self.raw)) * live
        heads = lambda x: x.sum((1, 2)).reshape(B, H).sum(0).float()
        shared = lambda x: self.whole(x).reshape(B, Hk, self.rep, T, dk).sum(2)
        return dict(grad_x=self.whole(dx), grad_b=shared(db), grad_c=shared(dc), grad_dt=self.whole(draw),
                    grad_A=heads(self.step * da), grad_D=heads((do * self.x).sum(-1).double()), grad_dt_bias=heads(draw),
                    grad_state=dS.transpose(1, 2).reshape(B, H, dv, dk).contiguous())


def _ssm(s):
    c = s["case"]
    if own:
        from test_regression_amd import mesa
        x, b, cc = _split(s["rows"], c["H"], c["dv"], c["Hk"], c["dk"])
        out, final = mesa.mesa_ssm_forward(x, b, cc, s["dt"].transpose(1, 2), s["A"], s["D"], s["dt_bias"], s["state"],
                                           lens=s["lens"], return_final=True)
        return dict(out=out, final=final)
    out, final = _Chunked(s).forward()
    live = _valid(s["lens"], c["B"], c["T"])[:, None, :, None]
    return dict(out=torch.where(live, out, 0.0).to(s["rows"].dtype), final=final.contiguous())


def _ssm_grad(s):
    """The gradients of x, b and c go side by side into the rows of the convolution's gradient."""
    c, dt = s["case"], s["rows"].dtype
    rows = torch.empty_like(s["rows"])
    gx, gb, gc = _split(rows, c["H"], c["dv"], c["Hk"], c["dk"])
    if own:
        from test_regression_amd import mesa
        x, b, cc = _split(s["rows"], c["H"], c["dv"], c["Hk"], c["dk"])
        gdt = torch.empty_like(s["dt"])
        g = mesa.mesa_ssm_backward(x, b, cc, s["dt"].transpose(1, 2), s["A"], s["grad_out"], s["D"], s["dt_bias"],
                                   s["state"], lens=s["lens"], grad_final=s["grad_final"], grad_x=gx, grad_b=gb,
                                   grad_c=gc, grad_dt=gdt.transpose(1, 2))
    else:
        g = _Chunked(s).backward(s["grad_out"], s["grad_final"])
        gx.copy_(g["grad_x"])
        gb.copy_(g["grad_b"])
        gc.copy_(g["grad_c"])
        gdt = g["grad_dt"].transpose(1, 2).to(dt).contiguous()
    r = dict(grad_rows=rows, grad_dt=gdt, grad_A=g["grad_A"], grad_D=g["grad_D"], grad_dt_bias=g["grad_dt_bias"])
    if c["start"]:
        r["grad_state"] = g["grad_state"]
    return r


def _ssm_step(s):
    c, S = s["case"], s["state"]
    x, b, cc = _split(s["rows"], c["H"], c["dv"], c["Hk"], c["dk"])
    if own:
        from test_regression_amd import mesa
        return dict(out=mesa.mesa_ssm_step(x, b, cc, s["dt"], s["A"], S, s["D"], s["dt_bias"]), state=S)
    rep = c["H"] // c["Hk"]
    b, cc = (t.float().repeat_interleave(rep, 1)[:, :, None, :] for t in (b, cc))
    raw = s["dt"].float() + s["dt_bias"]
    step = raw.clamp(min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    S.mul_(torch.exp(step * s["A"])[..., None, None])
    S.add_((step[..., None] * x.float())[..., None] * b)
    return dict(out=((S * cc).sum(-1) + s["D"][:, None] * x.float()).to(s["rows"].dtype), state=S)


def _pairs(x, rot, interleaved):
    """The two features of every rotated pair."""
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _turn(x, cos, sin, rot, interleaved):
    a, b = _pairs(x, rot, interleaved)
    y = x.clone()
    ya, yb = _pairs(y, rot, interleaved)
    ya.copy_(a * cos - b * sin)
    yb.copy_(b * cos + a * sin)
    return y


def _rotate(s):
    c = s["case"]
    Hq, Hk, d, rot, inter = (c[n] for n in ("Hq", "Hk", "d", "rot", "interleaved"))
    q, k = (t.unflatten(-1, (-1, d)).transpose(1, 2) for t in (s["rows"][..., :Hq * d], s["rows"][..., Hq * d:]))
    if own:
        from test_regression_amd import mesa
        how = dict(norm=c["norm"], eps=EPS, interleaved=inter, amplitude=s["amplitude"])
        yq, yk = mesa.mesa_qk_rotate(q, k, s["freqs"], s["positions"], s["wq"], s["wk"], **how)
        r = dict(q=yq, k=yk)
        if c["grad"]:
            rows = torch.empty_like(s["rows"])
            gq, gk = (t.unflatten(-1, (-1, d)).transpose(1, 2) for t in (rows[..., :Hq * d], rows[..., Hq * d:]))
            g = mesa.mesa_qk_rotate_backward(q, k, s["grad_q"], s["grad_k"], s["freqs"], s["positions"], s["wq"], s["wk"],
                                             grad_q=gq, grad_k=gk, **how)
            r["grad_rows"] = rows
            if c["norm"]:
                r.update(grad_wq=g["grad_wq"], grad_wk=g["grad_wk"])
        return r
    angle = s["positions"].double()[:, None, :, None] * s["freqs"]
    cos, sin = (s["amplitude"] * angle.cos()).float(), (s["amplitude"] * angle.sin()).float()
    r, grads = {}, []
    for name, x, w, dy in (("q", q, s["wq"], s["grad_q"]), ("k", k, s["wk"], s["grad_k"])):
        n = x.float()
        if c["norm"]:
            rs = torch.rsqrt(n.square().mean(-1, keepdim=True) + EPS)
            n = n * rs
        r[name] = _turn(n if w is None else n * w, cos, sin, rot, inter).to(x.dtype)
        if c["grad"]:
            g = _turn(dy.float(), cos, -sin, rot, inter)
            if c["norm"]:
                r["grad_w" + name] = (g * n).sum((0, 1, 2))
                g = g * w
                g = rs * (g - n * (g * n).mean(-1, keepdim=True))
            grads.append(g.transpose(1, 2).flatten(2))
    if c["grad"]:
        r["grad_rows"] = torch.cat(grads, -1).to(s["rows"].dtype)
    return r


def run(state):
    return {"conv": _conv, "ssm": _ssm, "ssm_grad": _ssm_grad, "ssm_step": _ssm_step,
            "rotate": _rotate}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "conv":
        B, T, D, W = (c[n] for n in ("B", "T", "D", "W"))
        n, h, par = B * T * D, B * (W - 1) * D if c["hist"] else 0, 4 * (W + 1) * D
        if not c["grad"]:
            return dict(bytes=e * (2 * n + 2 * h) + par, flops=n * (2 * W + 4))
        return dict(bytes=e * (4 * n + 3 * h) + 2 * par, flops=n * (6 * W + 12))
    if c["op"] in ("ssm", "ssm_grad"):
        B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        n, state = B * H * T, 4 * B * H * dk * dv
        bc, x = 2 * e * B * Hk * T * dk, e * n * dv
        if c["op"] == "ssm":
            # the state decayed and written once a token, and read for c: two products of dk x dv
            return dict(bytes=bc + 2 * x + e * n + state * (2 if c["start"] else 1), flops=5 * n * dk * dv)
        return dict(bytes=2 * bc + 3 * x + 2 * e * n + (3 * state if c["start"] else 0), flops=14 * n * dk * dv)
    if c["op"] == "ssm_step":
        N, Hk, H, dk, dv = (c[n] for n in ("N", "Hk", "H", "dk", "dv"))
        return dict(bytes=8 * N * H * dk * dv + e * N * (2 * Hk * dk + 2 * H * dv + H), flops=5 * N * H * dk * dv)
    rows = c["B"] * c["T"]
    n = rows * (c["Hq"] + c["Hk"]) * c["d"]
    par = 8 * rows + 4 * c["rot"] + (8 * c["d"] if c["norm"] else 0)
    if not c["grad"]:
        return dict(bytes=2 * e * n + par, flops=10 * n)
    return dict(bytes=4 * e * n + 2 * par, flops=25 * n)


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_scan(c, f, lens):
    B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
    rep, a = H // Hk, H * dv
    rows = f["rows"]
    x = rows[..., :a].reshape(B, T, H, dv)
    b = rows[..., a:a + Hk * dk].reshape(B, T, Hk, dk).repeat_interleave(rep, 2)
    cc = rows[..., a + Hk * dk:].reshape(B, T, Hk, dk).repeat_interleave(rep, 2)
    step = torch.nn.functional.softplus(f["dt"] + f["dt_bias"], threshold=1e9)
    n = [T] * B if lens is None else lens.tolist()
    return x, b, cc, step, n


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = {n: x.double() if torch.is_tensor(x) and x.is_floating_point() else x for n, x in s.items()}
    if c["op"] == "conv":
        return _exact_conv(c, f)
    if c["op"] in ("ssm", "ssm_grad"):
        B, Hk, H, T, dk, dv = (c[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        x, b, cc, step, n = _exact_scan(c, f, s["lens"])
        live = torch.tensor([[t < m for m in n] for t in range(T)], device=DEV)          # [T, B]
        every = live.all(1).tolist()
        S = f["state"] if c["start"] else x.new_zeros((B, H, dv, dk))
        decay = torch.exp(step * f["A"])
        if c["op"] == "ssm":
            out = x.new_zeros((B, H, T, dv))
            for t in range(T):
                new = decay[:, t, :, None, None] * S + (step[:, t, :, None] * x[:, t])[..., None] * b[:, t, :, None, :]
                o = (new * cc[:, t, :, None, :]).sum(-1) + f["D"][:, None] * x[:, t]
                if every[t]:
                    S = new
                    out[:, :, t] = o
                else:
                    S = torch.where(live[t][:, None, None, None], new, S)
                    out[:, :, t] = torch.where(live[t][:, None, None], o, 0.0)
            return dict(out=out, final=S)
        group = max(1, int(48e9 / (8 * B * T * dk * dv)))       # heads whose states are kept at once
        gx, gb, gc, gs = (torch.zeros_like(t) for t in (x, b, cc, step))
        gdecay, dS = torch.zeros_like(step), torch.empty_like(S)
        for i in range(0, H, group):
            h = slice(i, min(H, i + group))
            kept = x.new_empty((T + 1, B, h.stop - i, dv, dk))
            kept[0] = S[:, h]
            for t in range(T):
                on = live[t][:, None, None, None]
                new = decay[:, t, h, None, None] * kept[t] + (step[:, t, h, None] * x[:, t, h])[..., None] * b[:, t, h, None, :]
                kept[t + 1] = new if every[t] else torch.where(on, new, kept[t])
            R = f["grad_final"][:, h] if c["start"] else torch.zeros_like(kept[0])
            for t in reversed(range(T)):
                on = live[t][:, None, None, None]
                do = f["grad_out"][:, h, t, :, None]
                gc[:, t, h] = (kept[t + 1] * do).sum(2)
                r = R + do * cc[:, t, h, None, :]
                rb, rx = (r * b[:, t, h, None, :]).sum(-1), (r * x[:, t, h, :, None]).sum(2)
                gx[:, t, h] = step[:, t, h, None] * rb + f["D"][h, None] * do[..., 0]
                gb[:, t, h] = step[:, t, h, None] * rx
                gs[:, t, h] = (rb * x[:, t, h]).sum(-1)
                gdecay[:, t, h] = (r * kept[t]).sum((2, 3)) * decay[:, t, h]
                r = r * decay[:, t, h, None, None]
                R = r if every[t] else torch.where(on, r, R)
            dS[:, h] = R
            del kept
        on = live.t()[..., None]
        gx, gb, gc = (torch.where(on[..., None], t, 0.0) for t in (gx, gb, gc))
        gdecay = torch.where(on, gdecay, 0.0)
        graw = torch.where(on, (gs + f["A"] * gdecay) * torch.sigmoid(f["dt"] + f["dt_bias"]), 0.0)
        rep = H // Hk
        gb, gc = (t.reshape(B, T, Hk, rep, dk).sum(3).flatten(2) for t in (gb, gc))
        do = torch.where(on[..., None], f["grad_out"].transpose(1, 2), 0.0)
        res = dict(grad_rows=torch.cat([gx.flatten(2), gb, gc], -1), grad_dt=graw, grad_A=(step * gdecay).sum((0, 1)),
                   grad_D=(do * x).sum((0, 1, 3)), grad_dt_bias=graw.sum((0, 1)))
        if c["start"]:
            res["grad_state"] = dS
        return res
    if c["op"] == "ssm_step":
        x, b, cc, step, _ = _exact_scan(dict(c, B=c["N"], T=1), dict(f, rows=f["rows"][:, None], dt=f["dt"][:, None]), None)
        S = torch.exp(step[:, 0] * f["A"])[..., None, None] * f["state"]
        S = S + (step[:, 0, :, None] * x[:, 0])[..., None] * b[:, 0, :, None, :]
        return dict(out=(S * cc[:, 0, :, None, :]).sum(-1) + f["D"][:, None] * x[:, 0], state=S)
    Hq, d, rot = c["Hq"], c["d"], c["rot"]
    rows = f["rows"].requires_grad_(c["grad"])
    z = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=DEV),
                    s["positions"].double()[:, None, :, None] * f["freqs"])
    ws = [w.requires_grad_(c["grad"]) for w in (f["wq"], f["wk"]) if w is not None]
    outs = []
    for i, x in enumerate((rows[..., :Hq * d], rows[..., Hq * d:])):
        x = x.reshape(*x.shape[:2], -1, d).transpose(1, 2)
        if c["norm"]:
            x = x / (x * x).mean(-1, keepdim=True).add(EPS).sqrt() * ws[i]
        p = x[..., :rot]
        p = p.reshape(*p.shape[:-1], -1, 2) if c["interleaved"] else p.reshape(*p.shape[:-1], 2, -1).transpose(-1, -2)
        p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * z)
        p = p.flatten(-2) if c["interleaved"] else p.transpose(-1, -2).flatten(-2)
        outs.append(torch.cat([p, x[..., rot:]], -1))
    r = dict(q=outs[0].detach(), k=outs[1].detach())
    if c["grad"]:
        g = torch.autograd.grad(outs, [rows, *ws], (f["grad_q"], f["grad_k"]))
        r["grad_rows"] = g[0]
        if c["norm"]:
            r.update(grad_wq=g[1], grad_wk=g[2])
    return r


def _exact_conv(c, f):
    """The convolution as a sum of shifted rows, its gradients by torch's differentiation, in pieces of channels."""
    B, T, D, W = (c[n] for n in ("B", "T", "D", "W"))
    n = torch.full((B,), T, device=DEV) if f["lens"] is None else f["lens"].long()
    live = torch.arange(T, device=DEV)[None, :, None] < n[:, None, None]
    parts = []
    for i in range(0, D, 512):
        ch = slice(i, min(D, i + 512))
        x, w, bias = (t[..., ch].contiguous().requires_grad_(c["grad"]) for t in (f["x"], f["w"], f["bias"]))
        hist = (f["hist"][..., ch].contiguous() if c["hist"] else x.new_zeros((B, W - 1, x.shape[-1]))).detach()
        hist.requires_grad_(c["grad"])
        rows = torch.cat([hist, x], 1)
        acc = bias.expand(B, T, -1)
        for j in range(W):
            acc = acc + w[j] * rows[:, W - 1 - j:W - 1 - j + T]
        y = torch.where(live, torch.nn.functional.silu(acc), 0.0)
        r = dict(y=y.detach())
        if c["hist"]:
            r["hist"] = torch.stack([rows[b, m:m + W - 1].detach() for b, m in enumerate(n.tolist())])
        if c["grad"]:
            g = torch.autograd.grad(y, (x, w, bias, hist), f["grad_y"][..., ch])
            r.update(grad_x=g[0], grad_w=g[1], grad_bias=g[2])
            if c["hist"]:
                r["grad_hist"] = g[3]
        parts.append(r)
    return {k: torch.cat([p[k] for p in parts], -1) for k in parts[0]}
