"""Measured cases of the state space layer's operators: the short causal convolution (conv), the selective
state space scan (ssm) and the root-mean-square norm (norm), each in its prompt, training and single-token forms.

`run` computes an operator from elementary torch operations (own = False) or calls the library (own = True).
`exact` steps the definitions in float64, token by token.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
BLOCK = 128          # values of a row that share one scale of the 8-bit output
E4M3_MAX = 448.0
CHUNK = 64           # tokens per block of the plain form's products


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _conv(name, op, B, T, D, K, dtype, lens=False):
    return dict(name=name, op=op, B=B, T=T, D=D, K=K, dtype=dtype, lens=lens)


def _ssm(name, op, B, H, G, T, N, P, dtype, lens=False, layout="tokens"):
    return dict(name=name, op=op, B=B, H=H, G=G, T=T, N=N, P=P, dtype=dtype, lens=lens, layout=layout)


def _norm(name, op, rows, D, dtype, residual=False, gate=False, bits8=False):
    return dict(name=name, op=op, rows=rows, D=D, dtype=dtype, residual=residual, gate=gate, bits8=bits8)


def listed():
    return [
        # a padded batch of prompts through the convolution of a layer of 24 heads of 64, one group of 128 states
        _conv("conv_prompt", "conv_fwd", 8, 2048, 24 * 64 + 2 * 128, 4, "bf16", lens=True),
        # the same layer's training step
        _conv("conv_train", "conv_bwd", 8, 2048, 24 * 64 + 2 * 128, 4, "bf16"),
        # one token of a small serving batch: the smallest call, launch latency
        _conv("conv_token", "conv_step", 4, 1, 12 * 64 + 2 * 64, 4, "bf16"),
        # the 16K-token behaviour sequence of the recurrence's headline workload: few pairs, a long axis
        _ssm("ssm_rec16k", "ssm_fwd", 2, 4, 1, 16384, 64, 64, "bf16", layout="heads"),
        # a padded batch of prompts of a language-model layer, 24 heads sharing one group of 128 states
        _ssm("ssm_prompt", "ssm_fwd", 8, 24, 1, 2048, 128, 64, "bf16", lens=True),
        # float32, odd length, narrow heads and two groups
        _ssm("ssm_odd_f32", "ssm_fwd", 3, 6, 2, 509, 32, 32, "f32", layout="heads"),
        # the training step's backward at the 130M-scale layer's batch and length (hidden 768: 12 heads of 64)
        _ssm("ssm_train", "ssm_bwd", 8, 12, 1, 2048, 128, 64, "bf16"),
        # float32 backward, odd length
        _ssm("ssm_train_f32", "ssm_bwd", 2, 6, 2, 333, 32, 32, "f32", layout="heads"),
        # one token of a full serving batch: the state's bytes
        _ssm("ssm_token", "ssm_step", 256, 24, 1, 1, 128, 64, "bf16"),
        # between two layers: residual added, 8-bit output for the next projection
        _norm("norm_residual_8bit", "norm_fwd", 16384, 1536, "bf16", residual=True, bits8=True),
        # after a scan: rows of one head (2 x 4 x 16384 of 64), gated
        _norm("norm_head_gate", "norm_fwd", 2 * 4 * 16384, 64, "bf16", gate=True),
        # the norm's backward in training, hidden 768, with the residual stream's gradient
        _norm("norm_train", "norm_bwd", 16384, 768, "bf16", residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_bwd", "ssm_step",
                     "norm_fwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("conv"):
        D, K = _log_int(rng, 16, 6144), rng.choice([2, 3, 4, 4])
        if op == "conv_step":
            c = _conv("", op, _log_int(rng, 1, 512), 1, D, K, dtype)
        else:
            T = _log_int(rng, 1, 16384)
            B = _log_int(rng, 1, max(1, min(64, (1 << 24) // (T * D) + 1)))
            c = _conv("", op, B, T, D, K, dtype, lens=op == "conv_fwd" and rng.random() < 0.5)
    elif op.startswith("ssm"):
        G = rng.choice([1, 1, 2, 4])
        H, N, P = G * rng.choice([1, 2, 3, 6, 8]), rng.choice([16, 32, 64, 128]), rng.choice([32, 64, 128])
        layout = rng.choice(["tokens", "heads"])
        if op == "ssm_step":
            c = _ssm("", op, _log_int(rng, 1, 256), H, G, 1, N, P, dtype, layout=layout)
        else:
            most = 200_000 if op == "ssm_fwd" else 100_000          # tokens x heads
            T = min(_log_int(rng, 1, 16384), most // H)
            B = _log_int(rng, 1, max(1, min(32, most // (T * H))))
            c = _ssm("", op, B, H, G, T, N, P, dtype, lens=op == "ssm_fwd" and rng.random() < 0.5, layout=layout)
    else:
        D = _log_int(rng, 32, 8192)
        rows = _log_int(rng, 1, max(1, min(131072, (1 << 23) // D)))
        fwd = op == "norm_fwd"
        c = _norm("", op, rows, D, dtype, residual=rng.random() < 0.5, gate=rng.random() < 0.5,
                  bits8=fwd and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ty = _type(case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = {"case": case}
    if case["op"].startswith("conv"):
        B, T, D, K = (case[k] for k in "BTDK")
        s["x"] = randn(B, 1, T, D).to(ty)                    # token-major rows: one "head" of all channels
        s["w"], s["bias"] = (randn(1, K, D) / math.sqrt(K)), 0.1 * randn(1, D)
        if case["op"] == "conv_bwd":
            s["dy"] = randn(B, 1, T, D).to(ty)
        if case["op"] == "conv_step":
            s["x"], s["state"] = s["x"][:, :, 0].contiguous(), randn(B, 1, K - 1, D).to(ty)
        if case["lens"]:
            s["lens"] = torch.randint(0, T + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
            s["y"] = torch.zeros(B, 1, T, D, dtype=ty, device=DEV)
    elif case["op"].startswith("ssm"):
        B, H, G, T, N, P = (case[k] for k in ("B", "H", "G", "T", "N", "P"))
        if case["layout"] == "tokens":                       # views of the convolution's output rows
            rows = randn(B, T, H * P + 2 * G * N).to(ty)
            s["x"] = rows[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
            s["Bm"] = rows[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
            s["Cm"] = rows[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2)
        else:
            s["x"], s["Bm"], s["Cm"] = randn(B, H, T, P).to(ty), randn(B, G, T, N).to(ty), randn(B, G, T, N).to(ty)
        s["dt"] = 0.5 * randn(B, H, T)
        step = torch.exp(math.log(1e-3) + rand(H) * math.log(100.0))      # step sizes of 1e-3 .. 1e-1
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"], s["D"] = -(1 + 15 * rand(H)), randn(H)
        if case["op"] == "ssm_bwd":
            s["dy"] = randn(B, T, H, P).to(ty).transpose(1, 2) if case["layout"] == "tokens" else randn(B, H, T, P).to(ty)
            s["dS"] = randn(B, H, N, P)
        else:
            s["S"] = randn(B, H, N, P)
        if case["op"] == "ssm_step":
            s["x"], s["Bm"], s["Cm"], s["dt"] = s["x"][:, :, 0], s["Bm"][:, :, 0], s["Cm"][:, :, 0], s["dt"][:, :, 0].contiguous()
        if case["lens"]:
            s["lens"] = torch.randint(0, T + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
            s["y"] = torch.zeros(B, H, T, P, dtype=ty, device=DEV)
    else:
        rows, D = case["rows"], case["D"]
        s["x"], s["w"] = randn(rows, D).to(ty), 1 + 0.1 * randn(D)
        if case["gate"]:
            s["gate"] = randn(rows, D).to(ty)
        if case["residual"]:
            s["residual"] = 2 * randn(rows, D).to(ty)        # backward: the residual stream's own gradient
        if case["op"] == "norm_bwd":
            s["dy"] = randn(rows, D).to(ty)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms, float32
# ---------------------------------------------------------------------------------------------------------------------
def _silu_parts(z):
    """silu(z) and its derivative."""
    sig = torch.sigmoid(z)
    return z * sig, sig * (1 + z * (1 - sig))


def _keep(lens, T):
    return torch.arange(T, device=DEV)[None, :] < lens[:, None]


def _plain_conv_fwd(s):
    x, w = s["x"], s["w"]
    B, H, T, D = x.shape
    K = w.shape[1]
    xp = torch.nn.functional.pad(x.float(), (0, 0, K - 1, 0))
    pre = sum(xp[:, :, j:j + T] * w[None, :, j, None] for j in range(K)) + s["bias"][None, :, None]
    y = _silu_parts(pre)[0].to(x.dtype)
    if "lens" not in s:
        return y, xp[:, :, T:].to(x.dtype)
    s["y"].copy_(torch.where(_keep(s["lens"], T)[:, None, :, None], y, s["y"]))
    last = s["lens"].long()[:, None, None, None] + torch.arange(K - 1, device=DEV)[None, None, :, None]
    return s["y"], xp.gather(2, last.expand(B, H, K - 1, D)).to(x.dtype)


def _plain_conv_bwd(s):
    x, w, dy = s["x"], s["w"], s["dy"].float()
    T, K = x.shape[2], w.shape[1]
    xp = torch.nn.functional.pad(x.float(), (0, 0, K - 1, 0))
    pre = sum(xp[:, :, j:j + T] * w[None, :, j, None] for j in range(K)) + s["bias"][None, :, None]
    g = dy * _silu_parts(pre)[1]
    gp = torch.nn.functional.pad(g, (0, 0, 0, K - 1))
    dx = sum(gp[:, :, K - 1 - j:K - 1 - j + T] * w[None, :, j, None] for j in range(K))
    dw = torch.stack([(xp[:, :, j:j + T] * g).sum((0, 2)) for j in range(K)], 1)
    return dx.to(x.dtype), dw, g.sum((0, 2))


def _plain_conv_step(s):
    x, w, state = s["x"], s["w"], s["state"]
    rows = torch.cat([state, x[:, :, None]], 2)
    y = _silu_parts((rows.float() * w[None]).sum(2) + s["bias"][None])[0].to(x.dtype)
    state.copy_(rows[:, :, 1:])
    return y, state


def _softplus(z):
    return torch.where(z > 20, z, torch.log1p(torch.exp(z)))


def _chunks(t, nc):
    """[B, H, T, ...] as float32 [B, H, nc, CHUNK, ...], padded with zeros."""
    pad = nc * CHUNK - t.shape[2]
    t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 3) + (0, pad))
    return t.unflatten(2, (nc, CHUNK))


class _Parts:
    """What the forward and the backward of the scan share: steps, decays and products of one pass."""

    def __init__(self, s):
        x, dt = s["x"], s["dt"]
        self.B, self.H, self.T, self.P = x.shape
        self.G, self.N = s["Bm"].shape[1], s["Bm"].shape[3]
        self.nc = nc = -(-self.T // CHUNK)
        self.z = dt + s["dt_bias"][None, :, None]
        d, x = _softplus(self.z), x.float()
        if "lens" in s:
            keep = _keep(s["lens"], self.T)[:, None]
            d, x = torch.where(keep, d, 0.0), torch.where(keep[..., None], x, 0.0)
        self.d = _chunks(d, nc)
        self.x, self.b, self.c = _chunks(x, nc), _chunks(s["Bm"].float(), nc), _chunks(s["Cm"].float(), nc)
        cum = (self.d.double() * s["A"].double()[None, :, None, None]).cumsum(-1)      # log decay, long sums: 64 bits
        low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
        self.low = low
        self.L = (cum[..., :, None] - cum[..., None, :]).masked_fill_(~low, -math.inf).float().exp_()
        self.gm = self.c @ self.b.transpose(-1, -2).contiguous()                       # C B^T per group
        tot = cum[..., -1]
        run = tot.cumsum(-1)
        before = torch.nn.functional.pad(run, (1, 0))                                  # log decay in front of chunk i
        # decay from the end of chunk j to the start of chunk i, i > j
        e = before[..., :, None] - run[..., None, :]
        i, j = torch.arange(nc + 1, device=DEV)[:, None], torch.arange(nc, device=DEV)[None, :]
        self.E = e.masked_fill_(i <= j, -math.inf).float().exp_()
        self.before = before.float().exp()
        self.out = cum.float().exp()                                                   # start of the chunk .. token
        self.back = (tot[..., None] - cum).float().exp()                               # token .. end of the chunk
        self.tot = tot.float().exp()

    def heads(self, t):
        return t.repeat_interleave(self.H // self.G, 1)

    def states(self, S0=None):
        """The states that enter chunks 0 .. nc (the last one: the final state)."""
        w = (self.heads(self.b) * (self.back * self.d)[..., None]).transpose(-1, -2).contiguous()
        h = (self.E @ (w @ self.x).flatten(3)).unflatten(3, (self.N, self.P))
        return h if S0 is None else h + self.before[..., None, None] * S0[:, :, None]


def _plain_ssm_fwd(s):
    p = _Parts(s)
    h = p.states(s["S"])
    y = (p.heads(p.gm) * p.L * p.d[..., None, :]) @ p.x
    y += p.out[..., None] * (p.heads(p.c) @ h[:, :, :-1])
    y += s["D"][None, :, None, None, None] * p.x
    y = y.flatten(2, 3)[:, :, :p.T].to(s["x"].dtype)
    if "lens" not in s:
        return y, h[:, :, -1]
    s["y"].copy_(torch.where(_keep(s["lens"], p.T)[:, None, :, None], y, s["y"]))
    return s["y"], h[:, :, -1]


def _suffix(t):
    return t.flip(-1).cumsum(-1).flip(-1)


def _plain_ssm_bwd(s):
    p = _Parts(s)
    ty, A = s["x"].dtype, s["A"]
    dy = _chunks(s["dy"].float(), p.nc)
    hin = p.states()[:, :, :-1]
    # the adjoint arriving at the end of each chunk
    v = (p.heads(p.c) * p.out[..., None]).transpose(-1, -2).contiguous() @ dy
    r = p.E[:, :, 1:].transpose(-1, -2).contiguous() @ torch.nn.functional.pad(v[:, :, 1:], (0, 0, 0, 0, 0, 1)).flatten(3)
    dh = r.unflatten(3, (p.N, p.P)) + (p.E[:, :, -1, :, None, None] * s["dS"][:, :, None])
    gl = p.heads(p.gm) * p.L
    dm = dy @ p.x.transpose(-1, -2).contiguous()
    bh, ch = p.heads(p.b), p.heads(p.c)
    bdh = bh @ dh                                                          # [.., token, P]
    dx = (gl * p.d[..., None, :]).transpose(-1, -2).contiguous() @ dy
    dx += (p.d * p.back)[..., None] * bdh + s["D"][None, :, None, None, None] * dy
    dg = dm * p.L * p.d[..., None, :]
    dcm = dg @ bh + p.out[..., None] * (dy @ hin.transpose(-1, -2).contiguous())
    dbm = dg.transpose(-1, -2).contiguous() @ ch
    dbm += (p.d * p.back)[..., None] * (p.x @ dh.transpose(-1, -2).contiguous())
    q = gl * dm
    z = (q * p.d[..., None, :]).masked_fill(~p.low.tril(-1), 0.0).double()
    j = p.back * (p.x * bdh).sum(-1)
    i = p.out * ((ch @ hin) * dy).sum(-1)
    jd = (j * p.d).double()
    dl = _suffix(z.sum(-1) - z.sum(-2) + i.double()) + (jd.cumsum(-1) - jd)
    dl = dl + (p.tot * (hin * dh).sum((-1, -2)))[..., None]
    dd = q.sum(-2) + j + (A[None, :, None, None] * dl).float()
    ddt = dd.flatten(2)[:, :, :p.T] * torch.sigmoid(p.z)

    def rows(t):
        return t.flatten(2, 3)[:, :, :p.T]

    def groups(t):
        return rows(t).unflatten(1, (p.G, p.H // p.G)).sum(2).to(ty)

    return {"dx": rows(dx).to(ty), "dB": groups(dbm), "dC": groups(dcm), "ddt": ddt, "dA": (dl * p.d).sum((0, 2, 3)).float(),
            "dD": (p.x * dy).sum((0, 2, 3, 4)), "ddt_bias": ddt.sum((0, 2))}


def _plain_ssm_step(s):
    S, x = s["S"], s["x"].float()
    rep = S.shape[1] // s["Bm"].shape[1]
    b, c = s["Bm"].float().repeat_interleave(rep, 1), s["Cm"].float().repeat_interleave(rep, 1)
    d = _softplus(s["dt"] + s["dt_bias"][None])
    S.mul_(torch.exp(d * s["A"][None])[..., None, None])
    S.add_(b[..., :, None] * (d[..., None] * x)[..., None, :])
    y = (S * c[..., :, None]).sum(2) + s["D"][None, :, None] * x
    return y.to(s["x"].dtype), S


def _plain_norm_fwd(s):
    case, x = s["case"], s["x"]
    h = x.float() + s["residual"].float() if case["residual"] else x.float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    if case["gate"]:
        y = y * _silu_parts(s["gate"].float())[0]
    out = []
    if case["bits8"]:
        rows, D = y.shape
        blocks = torch.nn.functional.pad(y, (0, -D % BLOCK)).unflatten(1, (-1, BLOCK))
        amax = blocks.abs().amax(-1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        q = (blocks / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :D]
        out += [q.to(torch.float8_e4m3fn), scale]
    else:
        out.append(y.to(x.dtype))
    return out + ([h.to(x.dtype)] if case["residual"] else [])


def _plain_norm_bwd(s):
    case, ty = s["case"], s["x"].dtype
    h, dy, w = s["x"].float(), s["dy"].float(), s["w"]
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hat, out = h * rstd, {}
    if case["gate"]:
        silu, dsilu = _silu_parts(s["gate"].float())
        out["dgate"] = (dy * hat * w * dsilu).to(ty)
        dy = dy * silu
    g = dy * w
    dh = rstd * (g - hat * (g * hat).mean(-1, keepdim=True))
    if case["residual"]:
        dh = dh + s["residual"].float()
    return {"dh": dh.to(ty), "dw": (dy * hat).sum(0), **out}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def _own_run(s):
    import delta_rule_sequence_amd as prism
    case = s["case"]
    op = case["op"]
    if op == "conv_fwd":
        return prism.conv_fwd(s["x"], s["w"], bias=s["bias"], silu=True, lens=s.get("lens"), out=s.get("y"))
    if op == "conv_bwd":
        g = prism.conv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], silu=True)
        return g["dx"], g["dconv_w"], g["dbias"]
    if op == "conv_step":
        return prism.conv_step(s["state"], s["x"], s["w"], bias=s["bias"], silu=True), s["state"]
    if op == "ssm_fwd":
        return prism.ssm_fwd(s["x"], s["Bm"], s["Cm"], s["dt"], s["A"], D=s["D"], dt_bias=s["dt_bias"], softplus=True,
                             S0=s["S"], lens=s.get("lens"), out=s.get("y"))
    if op == "ssm_bwd":
        return prism.ssm_bwd(s["x"], s["Bm"], s["Cm"], s["dt"], s["A"], s["dy"], D=s["D"], dt_bias=s["dt_bias"],
                             softplus=True, dS_final=s["dS"])
    if op == "ssm_step":
        return prism.ssm_step(s["S"], s["x"], s["Bm"], s["Cm"], s["dt"], s["A"], D=s["D"], dt_bias=s["dt_bias"],
                              softplus=True), s["S"]
    if op == "norm_fwd":
        r = prism.norm_fwd(s["x"], s["w"], residual=s.get("residual"), gate=s.get("gate"), eps=EPS, bits8=case["bits8"])
        return [r[k] for k in ("y", "scales", "h") if k in r]
    g = prism.norm_bwd(s["x"], s["w"], s["dy"], gate=s.get("gate"), dh_in=s.get("residual"), eps=EPS)
    return g


def run(s):
    if own:
        return _own_run(s)
    return {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
            "ssm_fwd": _plain_ssm_fwd, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step,
            "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("conv"):
        B, T, D, K = (case[k] for k in "BTDK")
        n, par = B * T * D, 4 * D * (K + 1)
        if op == "conv_fwd":
            n = n // 2 if case["lens"] else n                # lengths are uniform over 0 .. T
            return {"bytes": 2 * n * e + par + B * D * (K - 1) * e, "flops": n * (2 * K + 4)}
        if op == "conv_step":
            return {"bytes": 2 * n * e + par + 2 * B * D * (K - 1) * e, "flops": n * (2 * K + 4)}
        return {"bytes": 3 * n * e + 2 * par, "flops": n * (6 * K + 10)}
    if op.startswith("ssm"):
        B, H, G, T, N, P = (case[k] for k in ("B", "H", "G", "T", "N", "P"))
        t = B * T // 2 if case["lens"] else B * T
        state = 4 * B * H * N * P
        if op == "ssm_fwd":
            return {"bytes": t * (2 * H * P * e + 2 * G * N * e + 4 * H) + 2 * state, "flops": 4 * t * H * N * P}
        if op == "ssm_step":
            return {"bytes": t * (2 * H * P * e + 2 * G * N * e + 4 * H) + 2 * state, "flops": 5 * t * H * N * P}
        return {"bytes": t * (3 * H * P * e + 4 * G * N * e + 8 * H) + state, "flops": 10 * t * H * N * P}
    rows, D = case["rows"], case["D"]
    n = rows * D
    if op == "norm_fwd":
        moved = e + (1 if case["bits8"] else e) + (2 * e if case["residual"] else 0) + (e if case["gate"] else 0)
        return {"bytes": n * moved + 4 * D + (4 * rows * -(-D // BLOCK) if case["bits8"] else 0), "flops": n * 8}
    moved = 3 * e + (e if case["residual"] else 0) + (2 * e if case["gate"] else 0)
    return {"bytes": n * moved + 8 * D, "flops": n * 12}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _exact_conv(s, op):
    x, w, b = s["x"].double(), s["w"].double(), s["bias"].double()
    K = w.shape[1]
    if op == "conv_step":
        past = torch.cat((s["state"].double(), x.unsqueeze(2)), 2)
        pre = torch.einsum("bhkd,hkd->bhd", past, w) + b
        return pre / (1 + torch.exp(-pre)), past[:, :, 1:]
    T = x.shape[2]
    hist = torch.cat((torch.zeros_like(x[:, :, :1]).expand(-1, -1, K - 1, -1), x), 2)
    windows = hist.unfold(2, K, 1)                                       # [B, H, T, D, K]
    pre = (windows * w.transpose(1, 2)[None, :, None]).sum(-1) + b[None, :, None]
    sig = 1 / (1 + torch.exp(-pre))
    if op == "conv_fwd":
        y, state = pre * sig, hist[:, :, T:]
        if "lens" in s:
            state = state.clone()
            for i, n in enumerate(s["lens"].tolist()):
                y[i, :, n:] = 0
                state[i] = hist[i, :, n:n + K - 1]
        return y, state
    g = s["dy"].double() * (sig + pre * sig * (1 - sig))
    dx = torch.zeros_like(hist)
    for j in range(K):
        dx[:, :, j:j + T] += g * w[:, j][None, :, None]
    return dx[:, :, K - 1:], (windows * g[..., None]).sum((0, 2)).transpose(1, 2), g.sum((0, 2))


def _exact_ssm(s, op):
    one = op == "ssm_step"
    x, Bm, Cm, raw = (s[k].double().unsqueeze(2) if one else s[k].double() for k in ("x", "Bm", "Cm", "dt"))
    B, H, T, P = x.shape
    N, rep = Bm.shape[3], H // Bm.shape[1]
    A, D = s["A"].double(), s["D"].double()
    z = raw + s["dt_bias"].double()[None, :, None]
    d = torch.logaddexp(z, torch.zeros_like(z))
    lens = s["lens"].tolist() if "lens" in s else [T] * B
    live = torch.tensor([[t < n for t in range(T)] for n in lens], device=DEV, dtype=torch.float64)
    d = d * live[:, None]                                                # a step of zero keeps the state
    a = torch.exp(d * A[None, :, None])
    head = torch.arange(H, device=DEV) // rep
    if op != "ssm_bwd":
        S, y = s["S"].double(), torch.empty_like(x)
        for t in range(T):
            S = a[:, :, t, None, None] * S + (d[:, :, t, None] * Bm[:, head, t])[..., :, None] * x[:, :, t, None, :]
            y[:, :, t] = (Cm[:, head, t].unsqueeze(2) @ S).squeeze(2) + D[:, None] * x[:, :, t]
        y = y * live[:, None, :, None]
        return (y[:, :, 0], S) if one else (y, S)
    if 8 * B * H * T * N * P > 60e9:
        return None
    dy, past = s["dy"].double(), torch.zeros(T + 1, B, H, N, P, dtype=torch.float64, device=DEV)
    for t in range(T):
        past[t + 1] = a[:, :, t, None, None] * past[t] + (d[:, :, t, None] * Bm[:, head, t])[..., :, None] * x[:, :, t, None, :]
    dx, dd, da = torch.empty_like(x), torch.empty_like(d), torch.empty_like(d)
    dB, dC = torch.zeros(B, H, T, N, dtype=torch.float64, device=DEV), torch.zeros(B, H, T, N, dtype=torch.float64, device=DEV)
    R = s["dS"].double()
    for t in range(T - 1, -1, -1):
        b, c, xt, g = Bm[:, head, t], Cm[:, head, t], x[:, :, t], dy[:, :, t]
        R = R + c[..., :, None] * g[..., None, :]
        dC[:, :, t] = (past[t + 1] @ g.unsqueeze(-1)).squeeze(-1)
        Rx = (R @ xt.unsqueeze(-1)).squeeze(-1)
        dB[:, :, t] = d[:, :, t, None] * Rx
        bR = (b.unsqueeze(2) @ R).squeeze(2)
        dx[:, :, t] = d[:, :, t, None] * bR + D[:, None] * g
        dd[:, :, t] = (bR * xt).sum(-1)
        da[:, :, t] = (R * past[t]).sum((-1, -2)) * a[:, :, t]
        R = a[:, :, t, None, None] * R
    ddt = (dd + A[None, :, None] * da) / (1 + torch.exp(-z))
    G = Bm.shape[1]
    return {"dx": dx, "dB": dB.view(B, G, rep, T, N).sum(2), "dC": dC.view(B, G, rep, T, N).sum(2), "ddt": ddt,
            "dA": (da * d).sum((0, 2)), "dD": (x * dy).sum((0, 2, 3)), "ddt_bias": ddt.sum((0, 2))}


def _exact_norm(s, case):
    x, w = s["x"].double(), s["w"].double()
    D = x.shape[1]
    z = s["gate"].double() if case["gate"] else None
    sig = None if z is None else 1 / (1 + torch.exp(-z))
    if case["op"] == "norm_fwd":
        h = x + s["residual"].double() if case["residual"] else x
        y = w * h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / D + EPS)
        y = y if z is None else y * z * sig
        out = [y]
        if case["bits8"]:
            scale = torch.stack([y[:, i:i + BLOCK].abs().amax(1) / E4M3_MAX for i in range(0, D, BLOCK)], 1)
            scale[scale == 0] = 1
            out = [y / scale.repeat_interleave(BLOCK, 1)[:, :D], scale]
        return out + ([h] if case["residual"] else [])
    dy = s["dy"].double()
    n = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
    up = dy * w if z is None else dy * w * z * sig
    dh = up / n - x * (up * x).sum(-1, keepdim=True) / (D * n ** 3)
    if case["residual"]:
        dh = dh + s["residual"].double()
    out = {"dh": dh, "dw": ((dy if z is None else dy * z * sig) * x / n).sum(0)}
    if z is not None:
        out["dgate"] = dy * w * x / n * (sig + z * sig * (1 - sig))
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("conv"):
        return _exact_conv(s, op)
    return _exact_ssm(s, op) if op.startswith("ssm") else _exact_norm(s, case)
