"""Edges of the state space layer's operators on the GPU: long and large tensors (offsets past 32 bits), many segments, odd
head groups, streams, repeated calls.  Tolerances as in tests/test_layer_gpu.py."""
import numpy as np
import pytest

from oracle import layer
from tests import test_layer_gpu as base
from tests.conftest import gpu_available
from tests.test_layer_gpu import Rng, close, f64, scan_inputs, sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def prism():
    if not gpu_available():
        pytest.skip("no GPU")
    import delta_rule_sequence_amd as m
    m.load_library()
    return m


# (dtype, B, H, G, T, N, P): more than 8 and more than 16 segments (a scan over them), one to eight (none), an odd number of
# heads per group (one head per workgroup), two slices of 64 columns per head, groups of one head
LONG = [("bf16", 1, 1, 1, 3000, 16, 16), ("f32", 1, 1, 1, 3000, 16, 16), ("bf16", 1, 1, 1, 8200, 16, 32), ("f32", 1, 2, 2, 2100, 32, 16),
        ("bf16", 2, 9, 3, 450, 32, 64), ("bf16", 1, 5, 1, 700, 64, 32), ("bf16", 1, 3, 3, 330, 64, 128), ("f32", 1, 3, 1, 200, 128, 128),
        ("bf16", 40, 8, 1, 130, 16, 64)]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "_".join(map(str, c)))
def test_ssm_segments_and_groups(prism, case):
    dt, B, H, G, T, N, P = case
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(50, *case, layout="tokens")
    S0 = r.flt(B, H, N, P)
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias, S0=S0)
    ref, ref_S = layer.ssm(*(f64(t) for t in (x, Bm, Cm, dt_, A, D, bias)), True, f64(S0))
    size, size_S = sizes(x, Bm, Cm, dt_, A, D, bias, True, S0)
    close("y", y, ref, size, dt)
    close("S_final", S, ref_S, size_S, dt, "f32")
    dy, dS = r.vec(B, H, T, P), r.flt(B, H, N, P)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, dy, D, bias, dS_final=dS)
    args = [f64(t) for t in (x, Bm, Cm, dt_, A, dy, D, bias)]
    ref, size = layer.ssm_grad(*args, True, f64(dS)), layer.ssm_grad(*args, True, f64(dS), absolute=True)
    for k in ("dx", "dB", "dC", "ddt", "dA", "dD", "ddt_bias"):
        close(k, g[k], ref[k], size[k], dt, None if k in ("dx", "dB", "dC") else "f32")


def test_ssm_pieces_are_the_whole(prism):
    """A sequence in pieces of 1, 63, 64, 65 and 300 tokens, each from the state of the one before: float32, sums in another
    order only."""
    import torch
    B, H, G, N, P = 1, 2, 1, 32, 32
    T = 1 + 63 + 64 + 65 + 300
    _, x, Bm, Cm, dt_, A, D, bias = scan_inputs(51, "f32", B, H, G, T, N, P)
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias)
    state, at = None, 0
    for n in (1, 63, 64, 65, 300):
        cut = [t[:, :, at:at + n] for t in (x, Bm, Cm, dt_)]
        part, state = prism.ssm_fwd(*cut, A, D, bias, S0=state)
        assert torch.allclose(part, y[:, :, at:at + n], rtol=1e-4, atol=1e-4)
        at += n
    assert torch.allclose(state, S, rtol=1e-4, atol=1e-4)


def test_offsets_past_32_bits(prism):
    """Rows whose element offsets exceed 2^31 (and byte offsets 2^32), against the same rows in a small tensor."""
    import torch
    big = torch.empty(1, 300, 1 << 23, dtype=torch.bfloat16, device="cuda")              # 4.7 GiB, rows 16 MB apart
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(52, "bf16", 1, 1, 1, 300, 64, 64)
    xv, bv, cv, yv = (big[:, :, k * 64:(k + 1) * 64].unsqueeze(1) for k in (0, 1, 2, 131071))
    xv.copy_(x), bv.copy_(Bm), cv.copy_(Cm)
    y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias)
    got, got_S = prism.ssm_fwd(xv, bv, cv, dt_, A, D, bias, out=yv)
    assert torch.equal(got, y) and torch.equal(got_S, S)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, x, D, bias)
    outs = tuple(big[:, :, k * 64:(k + 1) * 64].unsqueeze(1) for k in (3, 4, 5))
    h = prism.ssm_bwd(xv, bv, cv, dt_, A, xv, D, bias, out=outs)
    assert all(torch.equal(g[k], h[k]) for k in g)
    w = r.flt(1, 4, 64)
    assert torch.equal(prism.conv_fwd(xv, w, out=yv)[0], prism.conv_fwd(x, w)[0])
    assert torch.equal(prism.conv_bwd(xv, w, yv)["dx"], prism.conv_bwd(x, w, yv.contiguous())["dx"])
    n, m = prism.norm_fwd(xv[:, 0])["y"], prism.norm_fwd(x[:, 0])["y"]
    assert torch.equal(n, m)
    with pytest.raises(prism.PrismError):                                                # rows more than 16 MB apart
        wide = big.view(1, 100, 3 << 23)[:, :, :64].unsqueeze(1)
        prism.ssm_fwd(wide, wide, wide, dt_[:, :, :100].contiguous(), A)
    del big, xv, bv, cv, yv, outs
    rows = torch.zeros((1 << 16) + 3, 1 << 15, dtype=torch.bfloat16, device="cuda")      # 2^31 elements and more
    rows[-3:] = r.vec(3, 1 << 15)
    ref = prism.norm_fwd(rows[-3:].contiguous(), bits8=True)
    got = prism.norm_fwd(rows, bits8=True)
    assert torch.equal(got["y"][-3:].view(torch.uint8), ref["y"].view(torch.uint8)) and torch.equal(got["scales"][-3:], ref["scales"])


def test_non_finite_rows_stay_causal(prism):
    """An infinity in one token of the convolution, and one in B, C or dt of the scan: earlier tokens are unaffected; and a
    non-finite x reaches no token before its chunk of 64."""
    import torch
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(53, "bf16", 1, 2, 1, 200, 32, 32)
    y, _ = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias)
    for t in (Bm, Cm, dt_):
        keep = t.clone()
        t[:, :, 100] = float("inf")
        got, _ = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias)
        assert torch.equal(got[:, :, :100], y[:, :, :100])
        t.copy_(keep)
    x2 = x.clone()
    x2[:, :, 100] = float("nan")
    got, _ = prism.ssm_fwd(x2, Bm, Cm, dt_, A, D, bias)
    assert torch.equal(got[:, :, :64], y[:, :, :64]) and bool(torch.isnan(got[:, :, 128:]).all())
    w = r.flt(2, 4, 32)
    c, c2 = prism.conv_fwd(x, w)[0], prism.conv_fwd(x2, w)[0]
    assert torch.equal(c2[:, :, :100], c[:, :, :100]) and torch.equal(c2[:, :, 104:], c[:, :, 104:])
    assert bool(torch.isnan(c2[:, :, 100:104]).all())


def test_two_streams_and_a_given_one(prism):
    """Calls on two streams at once, and on a stream given by its handle, with results bit-identical to one after another."""
    import torch
    cases = [scan_inputs(s, "bf16", 2, 4, 1, 600, 64, 64)[1:] for s in (54, 55)]

    def both(c, **kw):
        x, Bm, Cm, dt_, A, D, bias = c
        y, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias, **kw)
        g = prism.ssm_bwd(x, Bm, Cm, dt_, A, y, D, bias, dS_final=S, **kw)
        n = prism.norm_fwd(y, residual=y, bits8=True, **kw)
        return [y, S, n["y"].view(torch.uint8), n["scales"]] + [g[k] for k in sorted(g)]

    ref = [both(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = both(cases[k])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for k in (0, 1) for p, q in zip(got[k], ref[k]))
    got = both(cases[0], stream=streams[0].cuda_stream)
    streams[0].synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref[0]))
    got = both(cases[0], stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref[0]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeated_calls_are_identical(prism, dt):
    """Every sum has a fixed order: three calls on the same inputs, a used workspace among them, agree bit for bit."""
    import torch
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(56, dt, 2, 6, 2, 500, 32, 128)
    w, b = r.flt(6, 4, 128), r.flt(6, 128)
    lib = prism.load_library()
    ws = torch.full((lib.prism_ssm_bwd_workspace_bytes(2, 6, 2, 500, 32, 128, 1 if dt == "bf16" else 0),), 0xff, dtype=torch.uint8, device="cuda")

    def run():
        g = prism.ssm_bwd(x, Bm, Cm, dt_, A, x, D, bias, workspace=ws)
        c = prism.conv_bwd(x, w, x, b)
        n = prism.norm_bwd(x, torch.ones(128, device="cuda"), x, gate=x)
        return [d[k].clone() for d in (g, c, n) for k in sorted(d)]

    first = run()
    for _ in range(2):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))


# More channels than a wave's narrow form takes, not a multiple of a thread's group: (dtype, D)
WIDE = [("bf16", 129), ("bf16", 137), ("bf16", 1001), ("bf16", 519), ("f32", 65), ("f32", 263), ("bf16", 136), ("f32", 514)]


@pytest.mark.parametrize("dt,D", WIDE)
def test_conv_odd_widths_and_starts(prism, dt, D):
    """Rows that start at any element, with channels left over from the vector groups; the columns beside them stay."""
    import torch
    B, H, T, K = 2, 1, 45, 4
    r = Rng(60, dt)
    lens = torch.tensor([45, 2], dtype=torch.int32, device="cuda")
    for off in (0, 1):
        x, past = r.vec(B, H, T, D + 3)[..., off:off + D], r.vec(B, H, K - 1, D)
        w, bias, dy = r.flt(H, K, D), r.flt(H, D), r.vec(B, H, T, D + 2)[..., off:off + D]
        rows = torch.full((B, H, T, D + 3), 7.0, dtype=x.dtype, device="cuda")
        y, end = prism.conv_fwd(x, w, bias, conv_in=past, lens=lens, out=rows[..., off:off + D])
        assert bool((rows[..., :off] == 7.0).all()) and bool((rows[..., off + D:] == 7.0).all()) and bool((y[1, :, 2:] == 7.0).all())
        elementwise = 2e-5 / (2.0 ** -8 + 2.0 ** -12) if dt == "bf16" else 1.0
        for b, n in enumerate((45, 2)):
            ref, ref_end = layer.conv(f64(x[b:b + 1, :, :n]), f64(w), f64(bias), True, f64(past[b:b + 1]))
            size = 1 + layer.conv(np.abs(f64(x[b:b + 1, :, :n])), np.abs(f64(w)), np.abs(f64(bias)), False, np.abs(f64(past[b:b + 1])))[0]
            close(f"y[{b}]", y[b:b + 1, :, :n], ref, elementwise * size, dt)
            np.testing.assert_array_equal(f64(end[b:b + 1]), ref_end)
        dxr = torch.full((B, H, T, D + 3), 7.0, dtype=x.dtype, device="cuda")
        g = prism.conv_bwd(x, w, dy, bias, out=dxr[..., off:off + D])
        assert bool((dxr[..., :off] == 7.0).all()) and bool((dxr[..., off + D:] == 7.0).all())
        ref = layer.conv_grad(f64(x), f64(w), f64(dy), f64(bias))
        size = 1 + layer.conv(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(bias)), False)[0]
        size = layer.conv_grad(np.abs(f64(x)), np.abs(f64(w)), 1.1 * np.abs(f64(dy)) * size, None, False)
        for k in ("dx", "dconv_w", "dbias"):
            close(k, g[k], ref[k], (elementwise if k == "dx" else 2e-5 / 2.0 ** -14 if dt == "bf16" else 1.0) * size[k], dt,
                  None if k == "dx" else "f32")


@pytest.mark.parametrize("dt,D", [("bf16", 519), ("f32", 263), ("bf16", 1024)])
def test_conv_history_in_place(prism, dt, D):
    """conv_out in the buffer of conv_in: the same rows and the same history as apart, for lengths below and above the
    window's."""
    import ctypes
    import torch
    B, H, T, K = 3, 2, 40, 4
    lib = prism.load_library()
    r = Rng(61, dt)
    x, w, past = r.vec(B, H, T, D), r.flt(H, K, D), r.vec(B, H, K - 1, D)
    lens = torch.tensor([1, 40, 2], dtype=torch.int32, device="cuda")
    y, end = prism.conv_fwd(x, w, conv_in=past, lens=lens, out=torch.zeros_like(x))
    y2, state = torch.zeros_like(x), past.clone()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.prism_conv_fwd(p(x), None, p(w), None, p(state), p(lens), B, H, T, D, K, 1, 1 if dt == "bf16" else 0, p(y2), None,
                              p(state), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(end, state)


@pytest.mark.parametrize("dt,D", [("bf16", 1013), ("f32", 515), ("bf16", 131), ("bf16", 8191)])
def test_norm_odd_rows_and_starts(prism, dt, D):
    """Rows of any length that start at any element: what dense rows give, and the columns beside them are not read."""
    r = Rng(62, dt)
    nan = float("nan")
    wide = [r.vec(7, D + 9) for _ in range(4)]
    w = 1 + 0.1 * r.flt(D)
    x, res, z, dy = (t[:, 5:5 + D] for t in wide)
    dense = [t.contiguous() for t in (x, res, z, dy)]
    for t in wide:
        t[:, :5], t[:, 5 + D:] = nan, nan
    for bits8 in (False, True):
        a = prism.norm_fwd(x, w, residual=dense[1], gate=z, bits8=bits8)
        b = prism.norm_fwd(dense[0], w, residual=dense[1], gate=dense[2], bits8=bits8)
        assert all(a[k].float().equal(b[k].float()) for k in b)
    a, b = prism.norm_bwd(x, w, dense[3], gate=z), prism.norm_bwd(dense[0], w, dense[3], gate=dense[2])
    assert all(a[k].equal(b[k]) for k in b)
    ref = layer.norm(f64(dense[0]), f64(w), None, f64(dense[2]))[0]
    got = prism.norm_fwd(x, w, gate=z)["y"]
    close("y", got, ref, (2e-5 / (2.0 ** -8 + 2.0 ** -12) if dt == "bf16" else 1.0) * (np.abs(ref) + 1e-3), dt)


@pytest.mark.parametrize("dt,rows,D", [("bf16", (1 << 25) + 77, 5), ("bf16", (1 << 20) + 3, 8193)])
def test_norm_many_rows(prism, dt, rows, D):
    """More workgroups than one axis of the launch holds: every row as in a call of its own."""
    import torch
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    y = prism.norm_fwd(x)["y"]
    for at in (0, rows // 2, (1 << 20) - 100, rows - 200):
        assert torch.equal(y[at:at + 200], prism.norm_fwd(x[at:at + 200].clone())["y"])


def test_sizes_past_the_interface(prism):
    """More rows than the C interface can be told are refused, not cut off."""
    import torch
    x = torch.zeros(1, dtype=torch.bfloat16, device="cuda").expand((1 << 32) + 5, 1)
    with pytest.raises(prism.PrismError):
        prism.norm_fwd(x)
    with pytest.raises(prism.PrismError):
        prism.conv_fwd(x[None, None], torch.zeros(1, 4, 1, device="cuda"))


@pytest.mark.parametrize("dt,rows,D", [("bf16", 3, 8193), ("bf16", 2, 16384), ("bf16", 2, 16385), ("f32", 5, 4097), ("f32", 2, 8192),
                                       ("f32", 3, 8193), ("bf16", 1100, 8250)])
@pytest.mark.parametrize("residual,gate,weight", [(True, True, True), (False, False, False)])
def test_norm_long_rows(prism, dt, rows, D, residual, gate, weight):
    """On both sides of the lengths that a workgroup of 256, of 1024 lanes holds; more rows than workgroups."""
    base.test_norm_fwd_bwd(prism, (dt, rows, D), residual, gate, weight)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("step", [30.0, 3e3, 3e4, 1e6])
def test_ssm_decay_after_a_reset(prism, dt, step):
    """A token whose step wipes the state out: the log decays of its chunk pass 1e5, those between the tokens after it are
    small and keep their digits."""
    B, H, G, T, N, P = 1, 2, 1, 130, 32, 64
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(63, dt, B, H, G, T, N, P)
    A.fill_(-16.0)
    d = dt_.sigmoid() * 0.1
    d[:, :, 3], d[:, :, 70] = step, step
    x[:, :, 3], x[:, :, 70] = 0.0, 0.0
    y, S = prism.ssm_fwd(x, Bm, Cm, d, A, D, softplus=False)
    args = (x, Bm, Cm, d, A, D, None)
    ref, ref_S = layer.ssm(*(None if t is None else f64(t) for t in args), False)
    size, size_S = sizes(*args, False, None)
    close("y", y, ref, size, dt)
    close("S_final", S, ref_S, size_S, dt, "f32")
    dy = r.vec(B, H, T, P)
    g = prism.ssm_bwd(x, Bm, Cm, d, A, dy, D, softplus=False)
    args = [None if t is None else f64(t) for t in (x, Bm, Cm, d, A, dy, D, None)]
    ref, size = layer.ssm_grad(*args, False, None), layer.ssm_grad(*args, False, None, absolute=True)
    for k in ("dx", "dB", "dC", "ddt", "dA", "dD"):
        close(k, g[k], ref[k], size[k], dt, None if k in ("dx", "dB", "dC") else "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ssm_decay_gradient_has_independent_errors(prism, dt):
    """dA sums a term per token that cancels to a hundredth of itself.  A token's ddt is off by a few half steps, 2^-22 of
    their usual size; if those errors are independent, their sum over the tokens, d_t / A each, stays below 4 of its
    standard deviations (what a chunk's tokens share would add up 64 times)."""
    import torch
    worst = 0.0
    for seed in range(12):
        r = Rng(70 + seed, dt)
        B, H, G, T, N, P = 5, 2, 1, 343, 64, 32
        x, Bm, Cm, dy = r.vec(B, H, T, P), r.vec(B, G, T, N), r.vec(B, G, T, N), r.vec(B, H, T, P)
        d, A = torch.exp(0.4 * r.flt(B, H, T)) * 0.05, -r.flt(H, lo=1.0, hi=16.0)
        g = prism.ssm_bwd(x, Bm, Cm, d, A, dy, softplus=False)
        ref = layer.ssm_grad(f64(x), f64(Bm), f64(Cm), f64(d), f64(A), f64(dy), None, None, False)
        usual = np.sqrt((ref["ddt"] ** 2).mean((0, 2)))
        lim = 4 * 2.0 ** -22 * usual * np.sqrt((f64(d) ** 2).sum((0, 2))) / np.abs(f64(A))
        worst = max(worst, float(np.max(np.abs(f64(g["dA"]) - ref["dA"]) / lim)))
    print(f"  dA: worst {worst:.3f} of its tolerance", flush=True)
    assert worst <= 1.0
