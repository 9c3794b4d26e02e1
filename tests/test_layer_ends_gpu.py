"""The ends of the state space layer's ranges on the GPU: the longest sequences, the last token."""
import pytest

from tests import test_layer_edges_gpu as edges
from tests.conftest import gpu_available
from tests.test_layer_gpu import Rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def prism():
    if not gpu_available():
        pytest.skip("no GPU")
    import delta_rule_sequence_amd as m
    m.load_library()
    return m


LONGEST = 2 ** 31 - 1 - 4096  # tokens that the convolution accepts


def test_conv_longest_sequence(prism):
    """The last rows of the longest sequence that is accepted, and of one whose last strip of tokens ends at 2^31, are what a
    call on the end of the sequence gives; the filter's gradient has their share."""
    import torch
    K, tail = 4, 40000
    r = Rng(80, "bf16")
    for T in (LONGEST, 2 ** 31 - 16384 + 5):
        x, y = torch.zeros(1, 1, T, 1, dtype=torch.bfloat16, device="cuda"), torch.full((1, 1, T, 1), 7.0, dtype=torch.bfloat16, device="cuda")
        x[:, :, -tail:] = r.vec(1, 1, tail, 1)
        w = r.flt(1, K, 1)
        print(f"  T = {T}, forward", flush=True)
        _, end = prism.conv_fwd(x, w, out=y)
        ref, ref_end = prism.conv_fwd(x[:, :, -tail:].clone(), w)
        assert torch.equal(y[:, :, -tail:], ref) and torch.equal(end, ref_end)
        dy = torch.zeros_like(x)
        dy[:, :, -tail + K:] = r.vec(1, 1, tail - K, 1)
        y.fill_(7.0)
        print(f"  T = {T}, backward", flush=True)
        g = prism.conv_bwd(x, w, dy, out=y)
        small = prism.conv_bwd(x[:, :, -tail:].clone(), w, dy[:, :, -tail:].clone())
        assert torch.equal(g["dx"][:, :, -tail:], small["dx"]) and bool((g["dx"][:, :, :-tail] == 0).all())
        # the same products, summed in float32 over strips of other lengths: 2e-5 of the sum of their absolute values
        size = float((x[:, :, -tail:].float().abs().max() * dy[:, :, -tail:].float().abs()).sum()) * 1.1
        assert float((g["dconv_w"] - small["dconv_w"]).abs().max()) <= 2e-5 * size


@pytest.mark.parametrize("dt,D", [("bf16", 7), ("bf16", 264), ("f32", 5), ("f32", 130)])
@pytest.mark.parametrize("T", [1, 2, 50, 256])
def test_conv_infinity_in_the_last_token(prism, dt, D, T):
    """Of dconv_w, the last token's row enters the last tap only; without silu the gradients of the others and all of
    dx stay what they are without the infinity."""
    import torch
    B, H, K = 2, 1, 4
    r = Rng(81, dt)
    x, w, bias, dy = r.vec(B, H, T, D), r.flt(H, K, D), r.flt(H, D), r.vec(B, H, T, D)
    x[:, :, -1] = 0.0
    ref = prism.conv_bwd(x, w, dy, bias, silu=False)
    for v in (float("inf"), float("nan")):
        x[:, :, -1] = v
        g = prism.conv_bwd(x, w, dy, bias, silu=False)
        assert torch.equal(g["dconv_w"][:, :-1], ref["dconv_w"][:, :-1])
        assert torch.equal(g["dx"], ref["dx"]) and torch.equal(g["dbias"], ref["dbias"])
        assert not bool(torch.isfinite(g["dconv_w"][:, -1]).any())


@pytest.mark.parametrize("dt,D", [("bf16", 256), ("bf16", 257), ("bf16", 264), ("f32", 128), ("f32", 129), ("f32", 132), ("bf16", 132)])
def test_conv_on_both_sides_of_the_narrow_form(prism, dt, D):
    """The last width whose lanes take a channel each, and the first ones that take a group, whole and with channels left over."""
    edges.test_conv_odd_widths_and_starts(prism, dt, D)
