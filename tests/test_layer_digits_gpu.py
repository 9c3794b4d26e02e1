"""What the state space layer's operators keep of their digits, on the GPU against definitions in 64 bits.

Tolerances of bfloat16 scans.  An output in bfloat16 is off by its own rounding, 2^-8 of the value (half a step), and by
what enters its products rounded: the scores, their gradients, the state and its adjoint pass as two bfloat16 parts, the
second a rounding (2^-8) of what the first leaves (2^-8): 2^-16 of a term; with float32 sums as in a scan of float32
tensors (2e-5 of the sum of absolute values) b = 2^-16 + 2e-5 of that sum.  A scan that rounds a score once is off by up to
2^-8 of its terms and exceeds this wherever they cancel.
"""
import numpy as np
import pytest

from oracle import layer
from tests.conftest import gpu_available
from tests.test_layer_gpu import f64, scan_inputs, sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def prism():
    if not gpu_available():
        pytest.skip("no GPU")
    import delta_rule_sequence_amd as m
    m.load_library()
    return m


# ---- silu of float32 tensors ---------------------------------------------------------------------------------------------
def test_silu_keeps_float32_digits(prism):
    """silu(z) over z from -80 to 80, in half steps of 2^-24, alone (a filter of one tap): the exponential 2, what corrects its
    argument and their product 1 each, the sum 1, the reciprocal 2, the product with z 1: 8.  Behind a norm 10 more: the row's sum
    of 64 squares (6 levels and 3 additions, halved by the root), its root, quotient and the two products of h r w."""
    import torch
    n = 20000
    z = torch.linspace(-80, 80, n, device="cuda")
    ref = f64(z) / (1 + np.exp(-f64(z)))
    w = torch.zeros(1, 2, 64, device="cuda")
    w[:, 1] = 1.0
    x = z[None, None, :, None].expand(1, 1, n, 64).contiguous()
    y = f64(prism.conv_fwd(x, w)[0])[0, 0]
    step = f64(prism.conv_step(torch.zeros(n, 1, 1, 64, device="cuda"), x[0, 0][:, None].contiguous(), w))[:, 0]
    dx = f64(prism.conv_bwd(x, w, torch.ones_like(x))["dx"])[0, 0]
    h = torch.linspace(0.5, 2.0, 64, device="cuda").expand(n, 64).contiguous()
    g = z[:, None].expand(n, 64).contiguous()
    got, dgate = f64(prism.norm_fwd(h, gate=g)["y"]), f64(prism.norm_bwd(h, None, torch.ones_like(h), gate=g)["dgate"])
    hat = f64(h) / np.sqrt((f64(h) ** 2).mean(-1, keepdims=True) + 1e-5)
    sig = 1 / (1 + np.exp(-f64(z)))
    slope = sig * (1 + f64(z) * (1 - sig))
    flat = sig * (1 + np.abs(f64(z)))
    worst = {}
    for name, a, b, scale, k in [("conv", y, ref[:, None], np.abs(ref)[:, None], 8), ("conv step", step, ref[:, None], np.abs(ref)[:, None], 8),
                                 # silu' = s (1 + z (1 - s)): s 7 half steps, 1 - s and its product with z, the sum and the product with s 5 more
                                 ("conv dx", dx, slope[:, None], flat[:, None], 12),
                                 ("norm", got, hat * ref[:, None], hat * np.abs(ref)[:, None], 18),
                                 ("norm dgate", dgate, hat * slope[:, None], hat * flat[:, None], 22)]:
        worst[name] = float(np.max(np.abs(a - b) / (k * 2.0 ** -24 * scale)))
    print("  " + ", ".join(f"{k}: worst {v:.3f} of its tolerance" for k, v in worst.items()), flush=True)
    assert max(worst.values()) <= 1.0, worst


# ---- scan of bfloat16 tensors -----------------------------------------------------------------------------------------------
def rounded_once(name, got, ref, size):
    got = f64(got)
    lim = 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + 2e-5) * np.abs(size) + 1e-30
    worst = float(np.max(np.abs(got - ref) / lim))
    print(f"  {name}: worst {worst:.3f} of its tolerance", flush=True)
    assert worst <= 1.0, (name, worst)


# every width pair with an even and an odd number of heads per group, one to many segments, lengths off the chunk
SCAN = [(1, h, 1, 70, n, p) for h in (2, 3) for n in (16, 32, 64, 128) for p in (16, 32, 64, 128)] + \
       [(2, 3, 1, 333, 64, 64), (1, 5, 1, 700, 128, 64), (2, 9, 3, 130, 16, 32), (1, 1, 1, 3000, 16, 16), (2, 6, 2, 400, 32, 128), (1, 2, 2, 1, 64, 64)]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "_".join(map(str, c)))
def test_scan_output_is_rounded_once(prism, case):
    B, H, G, T, N, P = case
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(82, "bf16", *case, layout="tokens")
    S0 = r.flt(B, H, N, P)
    y, _ = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias, S0=S0)
    ref = layer.ssm(*(f64(t) for t in (x, Bm, Cm, dt_, A, D, bias)), True, f64(S0))[0]
    rounded_once("y", y, ref, sizes(x, Bm, Cm, dt_, A, D, bias, True, S0)[0])


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "_".join(map(str, c)))
def test_scan_gradients_are_rounded_once(prism, case):
    B, H, G, T, N, P = case
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(83, "bf16", *case)
    dy, dS = r.vec(B, H, T, P), r.flt(B, H, N, P)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, dy, D, bias, dS_final=dS)
    args = [f64(t) for t in (x, Bm, Cm, dt_, A, dy, D, bias)]
    ref, size = layer.ssm_grad(*args, True, f64(dS)), layer.ssm_grad(*args, True, f64(dS), absolute=True)
    for k in ("dx", "dB", "dC"):
        rounded_once(k, g[k], ref[k], size[k])


@pytest.mark.parametrize("step", [30.0, 1e6])
def test_scan_is_rounded_once_after_a_reset(prism, step):
    """A token that wipes the state out puts the log decays of its chunk past 230: the scores behind it keep their digits."""
    B, H, G, T, N, P = 1, 2, 1, 130, 32, 64
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(84, "bf16", B, H, G, T, N, P)
    A.fill_(-16.0)
    d = dt_.sigmoid() * 0.1
    d[:, :, 3], d[:, :, 70] = step, step
    x[:, :, 3], x[:, :, 70] = 0.0, 0.0
    y, _ = prism.ssm_fwd(x, Bm, Cm, d, A, D, softplus=False)
    args = (x, Bm, Cm, d, A, D, None)
    ref = layer.ssm(*(None if t is None else f64(t) for t in args), False)[0]
    rounded_once("y", y, ref, sizes(*args, False, None)[0])


@pytest.mark.parametrize("case", [(2, 4, 1, 500, 128, 64), (1, 3, 1, 1100, 64, 32), (2, 2, 2, 300, 16, 128)], ids=lambda c: "_".join(map(str, c)))
def test_states_and_step_gradients_keep_float32_digits(prism, case):
    """S_final and ddt of bfloat16 tensors, root mean square of the error against that of the value.  Their operands pass as three
    parts (24 bits), so what is left are roundings of 2^-24: the weight and its product (3 half steps), a sum over 64 tokens per
    chunk and one per chunk.  Independent, a dozen of them make 2^-22; the limit is 2^-21.  Two parts (16 bits) leave
    1e-5 of S_final and 3e-6 of ddt (the oracle's formulas with operands cut to 16 bits)."""
    B, H, G, T, N, P = case
    r, x, Bm, Cm, dt_, A, D, bias = scan_inputs(85, "bf16", *case)
    _, S = prism.ssm_fwd(x, Bm, Cm, dt_, A, D, bias)
    dy, dS = r.vec(B, H, T, P), r.flt(B, H, N, P)
    g = prism.ssm_bwd(x, Bm, Cm, dt_, A, dy, D, bias, dS_final=dS)
    ref_S = layer.ssm(*(f64(t) for t in (x, Bm, Cm, dt_, A, D, bias)))[1]
    ref = layer.ssm_grad(*(f64(t) for t in (x, Bm, Cm, dt_, A, dy, D, bias)), True, f64(dS))
    rms = lambda a: float(np.sqrt((a ** 2).mean()))  # noqa: E731
    off = {"S_final": rms(f64(S) - ref_S) / rms(ref_S), "ddt": rms(f64(g["ddt"]) - ref["ddt"]) / rms(ref["ddt"])}
    print("  " + ", ".join(f"{k}: {v:.2e}" for k, v in off.items()), flush=True)
    assert max(off.values()) <= 2.0 ** -21, off
