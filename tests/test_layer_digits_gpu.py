"""What the state space layer's operators keep of their digits, on the GPU against definitions in 64 bits."""
import numpy as np
import pytest

from tests.conftest import gpu_available
from tests.test_layer_gpu import f64

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
