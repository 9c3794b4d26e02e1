"""The state space layer on the GPU against its float64 oracle.

Tolerances.  Each check is element-wise, |got - ref| <= a |ref| + b size, where `size` is the same sum over absolute
values (scan, gradients), so that it bounds what roundings of the terms can do:
* float32: sums of up to a few hundred terms in float32: b = 2e-5 (about 300 half steps of 2^-24), a = 0;
* bfloat16 outputs: the output's own rounding, a = 2^-8 (half a step); the score matrix and the state's readout (and, in
  the backward, the summed score gradients) enter a product rounded to bfloat16 once: b = 2^-8, plus 2^-12 for products of
  two roundings and float32 sums;
* float32 outputs of bfloat16 inputs (states, ddt, dA, ...): the operands keep at least 16 bits (two bfloat16 parts): an
  operand is off by at most 2^-17, two of them meet in a product and once more in the state itself: b = 2^-14;
* elementwise operators (conv, norm): float32 arithmetic throughout, b = 2e-5 of the row's scale.
"""
import numpy as np
import pytest

from oracle import layer
from tests.conftest import gpu_available

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def prism():
    if not gpu_available():
        pytest.skip("no GPU")
    import delta_rule_sequence_amd as m
    m.load_library()
    return m


def torch_dtype(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


class Rng:
    """Tensors on the GPU and the values they hold in float64."""

    def __init__(self, seed, dt):
        self.r, self.dt = np.random.default_rng(seed), torch_dtype(dt)

    def vec(self, *shape, scale=1.0):
        import torch
        return torch.tensor(scale * self.r.standard_normal(shape), dtype=torch.float32, device="cuda").to(self.dt)

    def flt(self, *shape, lo=None, hi=None, scale=1.0):
        import torch
        a = scale * self.r.standard_normal(shape) if lo is None else self.r.uniform(lo, hi, shape)
        return torch.tensor(a, dtype=torch.float32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, size, dt, kind=None):
    """kind: None = an output in dt; "f32" = a float32 output of the operator."""
    got, ref, size = f64(got) if not isinstance(got, np.ndarray) else got, np.asarray(ref), np.asarray(size)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    a, b = (0.0, 2e-5) if dt == "f32" else (0.0, 2.0 ** -14) if kind == "f32" else (2.0 ** -8, 2.0 ** -8 + 2.0 ** -12)
    lim = a * np.abs(ref) + b * np.abs(size) + 1e-30
    bad = ~(np.abs(got - ref) <= lim)
    worst = float(np.max(np.abs(got - ref) / lim)) if got.size else 0.0
    print(f"  {name}: worst {worst:.3f} of its tolerance", flush=True)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} values outside, worst {worst:.2f} of the tolerance"


# ---- convolution -------------------------------------------------------------------------------
def conv_inputs(seed, dt, B, H, T, D, K):
    r = Rng(seed, dt)
    return r, r.vec(B, H, T, D), r.flt(H, K, D), r.flt(H, D)


CONV = [("bf16", 2, 1, 300, 64, 4), ("bf16", 1, 3, 33, 24, 4), ("bf16", 2, 2, 1, 8, 3), ("bf16", 1, 1, 3, 7, 4),
        ("f32", 2, 1, 130, 20, 4), ("f32", 1, 2, 2, 5, 2), ("f32", 3, 1, 65, 1, 3), ("bf16", 1, 1, 1100, 40, 2)]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("silu", [True, False])
def test_conv_fwd_bwd(prism, case, silu):
    dt, B, H, T, D, K = case
    r, x, w, bias = conv_inputs(1, *case)
    y, end = prism.conv_fwd(x, w, bias, silu=silu)
    ref, ref_end = layer.conv(f64(x), f64(w), f64(bias), silu)
    size = 1 + layer.conv(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(bias)), False)[0]
    elementwise = 2e-5 / (2.0 ** -8 + 2.0 ** -12) if dt == "bf16" else 1.0
    close("y", y, ref, elementwise * size, dt)
    np.testing.assert_array_equal(f64(end), ref_end)
    dy = r.vec(B, H, T, D)
    g = prism.conv_bwd(x, w, dy, bias, silu=silu)
    ref = layer.conv_grad(f64(x), f64(w), f64(dy), f64(bias), silu)
    # |silu'| <= 1.1 and its argument is off by 2e-5 of its size at most
    size = layer.conv_grad(np.abs(f64(x)), np.abs(f64(w)), 1.1 * np.abs(f64(dy)) * size, None, False)
    for k in ("dx", "dconv_w", "dbias"):
        close(k, g[k], ref[k], (elementwise if k == "dx" else 2e-5 / 2.0 ** -14 if dt == "bf16" else 1.0) * size[k], dt,
              None if k == "dx" else "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_conv_lens_history_and_strides(prism, dt):
    import torch
    B, H, T, D, K = 6, 3, 70, 16, 4
    r = Rng(2, dt)
    rows = r.vec(B, T, H * D + 8)                          # heads of a token-major tensor
    x = rows[..., 8:].unflatten(-1, (H, D)).transpose(1, 2)
    w, past = r.flt(H, K, D), r.vec(B, H, K - 1, D)
    lens = torch.tensor([0, 1, 2, 69, 500, -4], dtype=torch.int32, device="cuda")
    for b, n in enumerate([0, 1, 2, 69, 70, 0]):
        rows[b, n:] = float("nan")                         # never read
    out = torch.full((B, T, H, D), 7.0, dtype=x.dtype, device="cuda").transpose(1, 2)
    y, end = prism.conv_fwd(x, w, conv_in=past, lens=lens, out=out)
    assert y is out
    for b, n in enumerate([0, 1, 2, 69, 70, 0]):
        ref, ref_end = layer.conv(f64(x[b:b + 1, :, :n]), f64(w), None, True, f64(past[b:b + 1]))
        size = 1 + layer.conv(np.abs(f64(x[b:b + 1, :, :n])), np.abs(f64(w)), None, False, np.abs(f64(past[b:b + 1])))[0]
        close(f"y[{b}]", y[b:b + 1, :, :n], ref, size * (2e-5 / 2.0 ** -8 if dt == "bf16" else 1.0), dt)
        np.testing.assert_array_equal(f64(end[b:b + 1]), ref_end)
        assert bool((y[b, :, n:] == 7.0).all())


@pytest.mark.parametrize("dt,K,D", [("bf16", 4, 40), ("f32", 2, 3), ("bf16", 3, 7)])
def test_conv_steps_continue_the_prompt(prism, dt, K, D):
    r, x, w, bias = conv_inputs(3, dt, 3, 2, 9, D, K)
    y, end = prism.conv_fwd(x, w, bias)
    _, state = prism.conv_fwd(x[:, :, :4], w, bias)
    for t in range(4, 9):
        step = prism.conv_step(state, x[:, :, t], w, bias)
        assert bool((step == y[:, :, t]).all()) or np.max(np.abs(f64(step) - f64(y[:, :, t]))) < 1e-2 * 2.0 ** -6
    np.testing.assert_array_equal(f64(state), f64(end))


# ---- scan --------------------------------------------------------------------------------------
def scan_inputs(seed, dt, B, H, G, T, N, P, layout="heads", A=None):
    r = Rng(seed, dt)
    if layout == "tokens":
        rows = r.vec(B, T, H * P + 2 * G * N)
        x = rows[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
        Bm = rows[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
        Cm = rows[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2)
    else:
        x, Bm, Cm = r.vec(B, H, T, P), r.vec(B, G, T, N), r.vec(B, G, T, N)
    dt_ = r.flt(B, T, H).transpose(1, 2) if layout == "tokens" else r.flt(B, H, T)
    a = r.flt(H, lo=-4.0, hi=-0.1) if A is None else r.flt(H, lo=A, hi=A)
    return r, x, Bm, Cm, dt_, a, r.flt(H), r.flt(H, lo=-4.0, hi=-1.0)


def sizes(x, Bm, Cm, dt, A, D, bias, softplus, S0=None):
    a = [np.abs(f64(t)) for t in (x, Bm, Cm)]
    z = f64(dt) + (0.0 if bias is None else f64(bias)[None, :, None])
    d = np.logaddexp(z, 0.0) if softplus else np.abs(z)
    return layer.ssm(*a, d, f64(A), None if D is None else np.abs(f64(D)), None, False, None if S0 is None else np.abs(f64(S0)),
                     decays=np.exp((np.logaddexp(z, 0.0) if softplus else z) * f64(A)[None, :, None]))


# every width pair, then lengths around the 64-token chunk and long enough for several segments
SCAN = [("bf16", 1, 2, 1, 70, n, p, "heads") for n in (16, 32, 64, 128) for p in (16, 32, 64, 128)] + \
       [("f32", 1, 2, 1, 70, n, p, "tokens") for n in (16, 32, 64, 128) for p in (16, 32, 64, 128)] + \
       [("bf16", 2, 4, 2, t, 64, 64, "tokens") for t in (1, 2, 63, 64, 65, 129)] + \
       [("f32", 2, 4, 2, t, 32, 64, "heads") for t in (1, 2, 63, 64, 65, 129)] + \
       [("bf16", 1, 3, 1, 1500, 128, 64, "tokens"), ("f32", 1, 3, 3, 777, 16, 32, "heads"), ("bf16", 2, 6, 2, 400, 32, 128, "heads")]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "_".join(map(str, c)))
def test_ssm_fwd_bwd(prism, case):
    dt, B, H, G, T, N, P, layout = case
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(10, *case)
    S0 = r.flt(B, H, N, P)
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias, S0=S0)
    ref, ref_S = layer.ssm(*(f64(t) for t in (x, Bm, Cm, dt_, A, D, bias)), True, f64(S0))
    size, size_S = sizes(x, Bm, Cm, dt_, A, D, bias, True, S0)
    close("y", y, ref, size, dt)
    close("S_final", S, ref_S, size_S, dt, "f32")
    dy, dS = r.vec(B, T, H, P).transpose(1, 2), r.flt(B, H, N, P)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, dy, D, bias, dS_final=dS)
    args = [f64(t) for t in (x, Bm, Cm, dt_, A, dy, D, bias)]
    ref = layer.ssm_grad(*args, True, f64(dS))
    size = layer.ssm_grad(*args, True, f64(dS), absolute=True)
    for k in ("dx", "dB", "dC", "ddt", "dA", "dD", "ddt_bias"):
        close(k, g[k], ref[k], size[k], dt, None if k in ("dx", "dB", "dC") else "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("A", [0.0, -1e4, -300.0])
def test_ssm_no_decay_and_total_decay(prism, dt, A):
    """A = 0 keeps everything (linear attention); A = -1e4 forgets within a token, exponents far below float32's range."""
    B, H, G, T, N, P = 1, 2, 1, 200, 32, 32
    r, x, Bm, Cm, dt_, A, _, _ = scan_inputs(11, dt, B, H, G, T, N, P, A=A)
    dt_ = dt_.abs() * 0.1
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, softplus=False)
    args = [f64(t) for t in (x, Bm, Cm, dt_, A)]
    ref, ref_S = layer.ssm(*args, None, None, False)
    size, size_S = sizes(x, Bm, Cm, dt_, A, None, None, False)
    close("y", y, ref, size, dt)
    close("S_final", S, ref_S, size_S, dt, "f32")
    dy = r.vec(B, H, T, P)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, dy, softplus=False)
    ref = layer.ssm_grad(*args, f64(dy), None, None, False)
    size = layer.ssm_grad(*args, f64(dy), None, None, False, absolute=True)
    assert "dD" not in g and "ddt_bias" not in g
    for k in ("dx", "dB", "dC", "ddt", "dA"):
        close(k, g[k], ref[k], size[k], dt, None if k in ("dx", "dB", "dC") else "f32")


@pytest.mark.parametrize("dt,T", [("bf16", 200), ("f32", 130), ("bf16", 1400)])
def test_ssm_lens(prism, dt, T):
    """A padded batch: rows past a length are neither read (NaN there) nor written, the state stops at the length."""
    import torch
    B, H, G, N, P = 7, 2, 1, 32, 64
    n = [0, 1, 64, 65, T, T, 0]
    lens = torch.tensor([0, 1, 64, 65, T, T + 9, -1], dtype=torch.int32, device="cuda")
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(12, dt, B, H, G, T, N, P)
    S0 = r.flt(B, H, N, P)
    clean = [t.clone() for t in (x, Bm, Cm, dt_)]
    for b in range(B):
        for t in (x, Bm, Cm):
            t[b, :, n[b]:] = float("nan")
        dt_[b, :, n[b]:] = float("inf")
    out = torch.full((B, H, T, P), 3.0, dtype=x.dtype, device="cuda")
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias, S0=S0, lens=lens, out=out)
    for b in range(B):
        part = [t[b:b + 1, :, :n[b]] for t in clean]
        ref, ref_S = layer.ssm(*(f64(t) for t in part), f64(A), f64(D), f64(bias), True, f64(S0[b:b + 1]))
        size, size_S = sizes(*part, A, D, bias, True, S0[b:b + 1])
        close(f"y[{b}]", y[b:b + 1, :, :n[b]], ref, size, dt)
        close(f"S[{b}]", S[b:b + 1], ref_S, size_S, dt, "f32")
        assert bool((y[b, :, n[b]:] == 3.0).all())


@pytest.mark.parametrize("dt,N,P", [("bf16", 128, 64), ("f32", 16, 16), ("bf16", 16, 128), ("bf16", 64, 32), ("f32", 128, 128),
                                    ("f32", 32, 16)])
def test_ssm_steps_continue_the_prompt(prism, dt, N, P):
    B, H, G, T = 3, 4, 2, 6
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(13, dt, B, H, G, T, N, P, "tokens")
    args = [f64(t) for t in (x, Bm, Cm, dt_, A, D, bias)]
    ref, ref_S = layer.ssm(*args)
    size, size_S = sizes(x, Bm, Cm, dt_, A, D, bias, True)
    _, S = prism.ssm_fwd(x[:, :, :3], Bm[:, :, :3], Cm[:, :, :3], dt_[:, :, :3], A, D, bias)
    for t in range(3, T):
        y = prism.ssm_step(S, x[:, :, t], Bm[:, :, t], Cm[:, :, t], dt_[:, :, t], A, D, bias)
        close(f"y{t}", y, ref[:, :, t], size[:, :, t], dt)
    close("S", S, ref_S, size_S, dt, "f32")


def test_ssm_final_state_may_be_the_entering_one(prism):
    """S_final and S0 in one buffer, with one segment and with several (through the C ABI: the binding returns a new
    state)."""
    import ctypes
    import torch
    lib = prism.load_library()
    for T in (64, 2000):
        B, H, G, N, P = 1, 2, 1, 32, 32
        r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(14, "bf16", B, H, G, T, N, P)
        S0 = r.flt(B, H, N, P)
        y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, S0=S0)
        y2, S2 = torch.empty_like(y), S0.clone()
        need = lib.prism_ssm_fwd_workspace_bytes(B, H, G, T, N, P, 1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        assert lib.prism_ssm_fwd(p(x), None, p(Bm), None, p(Cm), None, p(dt_), None, None, p(A), None, p(S2), None, B, H, G, T, N,
                                 P, 1, 1, p(y2), None, p(S2), p(ws), need, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(S, S2)


# ---- norm --------------------------------------------------------------------------------------
NORM = [("bf16", 5, 64), ("bf16", 33, 128), ("bf16", 3, 1536), ("bf16", 2, 8200), ("bf16", 4, 7), ("bf16", 3, 1), ("f32", 3, 20),
        ("f32", 5, 129), ("f32", 2, 5000), ("bf16", 600, 72), ("f32", 700, 4), ("bf16", 1, 24576), ("bf16", 9, 260), ("f32", 6, 256)]


@pytest.mark.parametrize("case", NORM, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("residual,gate,weight", [(False, False, True), (True, False, True), (False, True, False), (True, True, True)])
def test_norm_fwd_bwd(prism, case, residual, gate, weight):
    dt, rows, D = case
    r = Rng(20, dt)
    x, res, z = r.vec(rows, D), r.vec(rows, D) if residual else None, r.vec(rows, D) if gate else None
    w = 1 + 0.1 * r.flt(D) if weight else None
    v = lambda t: None if t is None else f64(t)  # noqa: E731
    elementwise = 2e-5 / (2.0 ** -8 + 2.0 ** -12) if dt == "bf16" else 1.0
    ref, ref_h = layer.norm(v(x), v(w), v(res), v(z))
    got = prism.norm_fwd(x, w, residual=res, gate=z)
    close("y", got["y"], ref, elementwise * (np.abs(ref) + 1e-3), dt)
    if residual:
        close("h", got["h"], ref_h, elementwise * (np.abs(v(x)) + np.abs(v(res))), dt)
    else:
        assert "h" not in got
    # 8 bits: the scales in float32, each byte the nearest e4m3 of y / scale (half a step: 2^-4 of the value, 2^-10 below 2^-6)
    q = prism.norm_fwd(x, w, residual=res, gate=z, bits8=True)
    nb = -(-D // 128)
    pad = np.pad(np.abs(ref), ((0, 0), (0, nb * 128 - D))).reshape(rows, nb, 128).max(-1)
    scale = np.where(pad > 0, pad / 448.0, 1.0)
    close("scales", q["scales"], scale, scale, "f32")
    full = np.repeat(scale, 128, 1)[:, :D]
    back = f64(q["y"].float()) * full
    assert np.all(np.abs(back - ref) <= (2.0 ** -4 + 1e-4) * np.abs(ref) + (2.0 ** -10 + 1e-4) * full)
    # backward, from the float32 or rounded row
    h = got["h"] if residual else x
    dy, dh_in = r.vec(rows, D), r.vec(rows, D) if residual else None
    g = prism.norm_bwd(h, w, dy, gate=z, dh_in=dh_in)
    ref = layer.norm_grad(v(h), v(dy), v(w), v(z), v(dh_in))
    zz = 1.0 if z is None else np.abs(v(z)) + 0.1
    rms = np.sqrt((v(h) ** 2).mean(-1, keepdims=True) + 1e-5)
    u = np.abs(v(dy)) * zz * (1.0 if w is None else np.abs(v(w)))
    size = u / rms + np.abs(v(h)) * (u * np.abs(v(h))).mean(-1, keepdims=True) / rms ** 3
    size = size if dh_in is None else size + np.abs(v(dh_in))
    close("dh", g["dh"], ref["dh"], elementwise * size, dt)
    if weight:
        close("dw", g["dw"], ref["dw"], (2e-5 / 2.0 ** -14 if dt == "bf16" else 1.0) * (np.abs(v(dy)) * zz * np.abs(v(h)) / rms).sum(0),
              dt, "f32")
    if gate:
        close("dgate", g["dgate"], ref["dgate"], elementwise * (np.abs(v(dy)) * 1.1 * np.abs(v(h)) / rms *
                                                               (1.0 if w is None else np.abs(v(w)))), dt)


def test_norm_strided_rows(prism):
    """x and gate as column slices of wider rows, aligned and not, and rows of one head of a scan's output."""
    r = Rng(21, "bf16")
    for off in (16, 3):
        wide = r.vec(2, 9, 200)
        x, z = wide[..., off:off + 64], wide[..., 100:164]
        got = prism.norm_fwd(x, gate=z)["y"]
        assert got.equal(prism.norm_fwd(x.contiguous(), gate=z.contiguous())["y"])
        dy = r.vec(2, 9, 64)
        a, b = prism.norm_bwd(x, None, dy, gate=z), prism.norm_bwd(x.contiguous(), None, dy, gate=z.contiguous())
        assert a["dh"].equal(b["dh"]) and a["dgate"].equal(b["dgate"])
    with pytest.raises(prism.PrismError):
        prism.norm_fwd(r.vec(4, 6, 32).transpose(0, 1)[:, :3])


def test_norm_special_rows(prism):
    """A row of zeros, of tiny and huge values, and one with an infinity."""
    import torch
    x = torch.zeros(5, 256, device="cuda")
    x[1], x[2], x[3] = 1e-30, 1e18, torch.linspace(-2, 2, 256, device="cuda")
    x[4, 7] = float("inf")
    got = prism.norm_fwd(x)["y"]
    ref = layer.norm(f64(x[:4]))[0]
    close("y", got[:4], ref, np.abs(ref), "f32")
    assert bool(torch.isnan(got[4, 7])) and bool((got[0] == 0).all())
    q = prism.norm_fwd(x, bits8=True)
    assert bool((q["scales"][0] == 1).all()) and bool((q["y"][0].float() == 0).all())
    assert bool(torch.isnan(q["y"][4, :128].float()).all())


# ---- together --------------------------------------------------------------------------------------
def the_layer(prism, rows, w, bias, dt_, A, D, dbias, z, weight, H, G, N, P, lens=None):
    """conv -> scan -> gated norm over one layer's rows [B, T, H P + 2 G N]."""
    y, conv_end = prism.conv_fwd(rows.unsqueeze(1), w, bias, lens=lens)
    y = y.squeeze(1)
    x = y[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
    Bm = y[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
    Cm = y[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2)
    o, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, dbias, lens=lens)
    o = o.transpose(1, 2)                                          # [B, T, H, P], dense
    n = prism.norm_fwd(o.flatten(2), weight, gate=z)["y"]
    return n, conv_end, S, (x, Bm, Cm, o)


def layer_inputs(dt, B, T, H, G, N, P, seed=30):
    r = Rng(seed, dt)
    C = H * P + 2 * G * N
    return (r.vec(B, T, C), r.flt(1, 4, C, scale=0.5), r.flt(1, C, scale=0.1), r.flt(B, T, H).transpose(1, 2), r.flt(H, lo=-4, hi=-0.5),
            r.flt(H), r.flt(H, lo=-3, hi=-1), r.vec(B, T, H * P), 1 + 0.1 * r.flt(H * P))


def test_layer_prompt_and_tokens(prism):
    """The three operators as a layer runs them: a prompt, then single tokens from its windows and states, equal to the
    whole sequence at once (float32: sums in another order only)."""
    import torch
    B, T, H, G, N, P = 2, 100, 4, 2, 32, 32
    rows, w, bias, dt_, A, D, db, z, nw = layer_inputs("f32", B, T, H, G, N, P)
    whole, end, S_end, _ = the_layer(prism, rows, w, bias, dt_, A, D, db, z, nw, H, G, N, P)
    first, conv, S, _ = the_layer(prism, rows[:, :90], w, bias, dt_[:, :, :90], A, D, db, z[:, :90].contiguous(), nw, H, G, N, P)
    assert torch.allclose(first, whole[:, :90], rtol=1e-4, atol=1e-4)
    for t in range(90, T):
        y = prism.conv_step(conv, rows[:, t].unsqueeze(1), w, bias).squeeze(1)
        x, Bm, Cm = y[:, :H * P].unflatten(-1, (H, P)), y[:, H * P:H * P + G * N].unflatten(-1, (G, N)), y[:, H * P + G * N:].unflatten(-1, (G, N))
        o = prism.ssm_step(S, x, Bm, Cm, dt_[:, :, t], A, D, db)
        n = prism.norm_fwd(o.flatten(1), nw, gate=z[:, t])["y"]
        assert torch.allclose(n, whole[:, t], rtol=1e-4, atol=1e-4), t
    assert torch.equal(conv, end) and torch.allclose(S, S_end, rtol=1e-4, atol=1e-5)


def test_layer_gradients_against_differences(prism):
    """The chained backward passes against central differences of the float64 oracle's layer along random directions."""
    import torch
    B, T, H, G, N, P = 1, 70, 2, 1, 16, 16
    rows, w, bias, dt_, A, D, db, z, nw = layer_inputs("f32", B, T, H, G, N, P, 31)
    r = Rng(32, "f32")
    out, _, _, (x, Bm, Cm, o) = the_layer(prism, rows, w, bias, dt_, A, D, db, z, nw, H, G, N, P)
    dn = r.vec(B, T, H * P)
    gn = prism.norm_bwd(o.flatten(2), nw, dn, gate=z)
    d_o = gn["dh"].unflatten(-1, (H, P)).transpose(1, 2)
    dy = torch.empty(B, T, H * P + 2 * G * N, device="cuda")       # the convolution's output gradient, filled in place
    parts = (dy[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2), dy[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2),
             dy[..., H * P + G * N:].unflatten(-1, (G, N)).transpose(1, 2))
    gs = prism.ssm_bwd(x, Bm, Cm, dt_, A, d_o, D, db, out=parts)
    gc = prism.conv_bwd(rows.unsqueeze(1), w, dy.unsqueeze(1), bias)

    def oracle(rows, w, bias, dt_, A, D, db, z, nw):
        y = layer.conv(rows[:, None], w, bias)[0][:, 0]
        cut = lambda a, n, k: a.reshape(B, T, n, k).transpose(0, 2, 1, 3)  # noqa: E731
        o = layer.ssm(cut(y[..., :H * P], H, P), cut(y[..., H * P:H * P + G * N], G, N), cut(y[..., H * P + G * N:], G, N), dt_, A, D, db)[0]
        return float((layer.norm(o.transpose(0, 2, 1, 3).reshape(B, T, H * P), nw, None, z)[0] * f64(dn)).sum())

    args = {k: f64(v) for k, v in zip(("rows", "w", "bias", "dt_", "A", "D", "db", "z", "nw"), (rows, w, bias, dt_, A, D, db, z, nw))}
    grads = {"rows": gc["dx"].squeeze(1), "w": gc["dconv_w"], "bias": gc["dbias"], "dt_": gs["ddt"], "A": gs["dA"], "D": gs["dD"],
             "db": gs["ddt_bias"], "z": gn["dgate"], "nw": gn["dw"]}
    rng = np.random.default_rng(33)
    for k, g in grads.items():
        v = rng.standard_normal(args[k].shape)
        hi, lo = dict(args), dict(args)
        hi[k], lo[k] = args[k] + 1e-5 * v, args[k] - 1e-5 * v
        num, ana = (oracle(**hi) - oracle(**lo)) / 2e-5, float((f64(g) * v).sum())
        # the norm of the gradient times the direction's sets the scale of the float32 sums (2e-5 each, three operators deep)
        assert abs(num - ana) <= 3e-4 * (np.linalg.norm(f64(g)) + 1.0), (k, num, ana)


def test_layer_side_stream_and_graph(prism):
    """On a non-default stream, and captured into a graph that is replayed three times on fresh inputs with eager calls in
    between: bit-identical to eager calls."""
    import torch
    B, T, H, G, N, P = 2, 700, 4, 2, 64, 64
    cut = dict(H=H, G=G, N=N, P=P)
    inp = layer_inputs("bf16", B, T, H, G, N, P, 40)
    lens = torch.tensor([T, 300], dtype=torch.int32, device="cuda")

    def both(inp):
        n, conv, S, (x, Bm, Cm, o) = the_layer(prism, *inp, lens=None, **cut)
        gn = prism.norm_bwd(o.flatten(2), inp[8], n, gate=inp[7])
        gs = prism.ssm_bwd(x, Bm, Cm, inp[3], inp[4], gn["dh"].unflatten(-1, (H, P)).transpose(1, 2), inp[5], inp[6], dS_final=S)
        gc = prism.conv_bwd(inp[0].unsqueeze(1), inp[1], inp[0].unsqueeze(1), inp[2])
        y = torch.zeros(B, H, T, P, dtype=torch.bfloat16, device="cuda")
        prism.ssm_fwd(x, Bm, Cm, inp[3], inp[4], lens=lens, out=y)
        S2, w2 = S.clone(), conv.clone()
        st = prism.ssm_step(S2, x[:, :, 0], Bm[:, :, 0], Cm[:, :, 0], inp[3][:, :, 0], inp[4])
        cs = prism.conv_step(w2, inp[0][:, 0].unsqueeze(1), inp[1])
        q = prism.norm_fwd(n, residual=inp[7], bits8=True)
        return [n, conv, S, y, S2, w2, st, cs, q["y"].view(torch.uint8), q["scales"], q["h"]] + [gn[k] for k in sorted(gn)] + \
            [gs[k] for k in sorted(gs)] + [gc[k] for k in sorted(gc)]

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    eager = both(inp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(inp)
    side.synchronize()
    assert same(eager, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(inp)
    for seed in (41, 42, 43):
        for dst, src in zip(inp, layer_inputs("bf16", B, T, H, G, N, P, seed)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, both(inp)), seed


def test_binding_refusals(prism):
    import torch
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    x, bc, dt_, A = z(2, 2, 4, 16), z(2, 1, 4, 16), z(2, 2, 4), z(2)
    bad = [lambda: prism.ssm_fwd(x, bc, bc, dt_, None), lambda: prism.ssm_fwd(x, bc, bc[:, :, :3], dt_, A),
           lambda: prism.ssm_fwd(x, bc.bfloat16(), bc, dt_, A), lambda: prism.ssm_fwd(x.half(), bc.half(), bc.half(), dt_, A),
           lambda: prism.ssm_fwd(x, bc, bc, dt_.double(), A), lambda: prism.ssm_fwd(x, bc, bc, dt_, A, lens=z(2, dtype=torch.int64)),
           lambda: prism.ssm_fwd(x, bc, bc, dt_, A, S0=z(2, 2, 16, 8)), lambda: prism.ssm_fwd(x[:1].expand(2, -1, -1, -1), bc, bc, dt_, A),
           lambda: prism.ssm_fwd(x, bc, bc, dt_, A, workspace=z(8, dtype=torch.uint8)),
           lambda: prism.ssm_fwd(x, bc, bc, dt_, A, out=x.transpose(2, 3)), lambda: prism.ssm_bwd(x, bc, bc, dt_, A, None),
           lambda: prism.ssm_bwd(x, bc, bc, dt_, A, x, out=(x,)), lambda: prism.ssm_step(None, x[:, :, 0], bc[:, :, 0], bc[:, :, 0], dt_[:, :, 0], A),
           lambda: prism.ssm_fwd(z(2, 2, 0, 16), z(2, 1, 0, 16), z(2, 1, 0, 16), z(2, 2, 0), A), lambda: prism.conv_fwd(x, z(2, 5, 16)),
           lambda: prism.conv_fwd(x, z(2, 4, 8)), lambda: prism.conv_fwd(x, None), lambda: prism.conv_bwd(x, z(2, 4, 16), None),
           lambda: prism.conv_step(None, x[:, :, 0], z(2, 4, 16)), lambda: prism.norm_fwd(x, z(8)), lambda: prism.norm_fwd(x, eps=-1.0),
           lambda: prism.norm_fwd(x, residual=x[:1]), lambda: prism.norm_fwd(z(0, 16)), lambda: prism.norm_bwd(x, None, None),
           lambda: prism.norm_fwd(x, gate=x.transpose(2, 3))]
    for k, f in enumerate(bad):
        with pytest.raises(prism.PrismError):
            f()
            pytest.fail(f"call {k} was not refused")
