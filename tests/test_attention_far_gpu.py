"""Scores of 10^4 and far beyond in the kernels of many rows: every row's p is 1 for one key, so the results are sums of inputs."""
import numpy as np
import pytest

from tests.test_attention_gpu import H, U, Rng, prism  # noqa: F401

pytestmark = pytest.mark.gpu

# workgroups of 128 rows and of 256, forward and backward
CASES = [("bf16", 1, 48, 513, 128), ("bf16", 2, 120, 513, 128), ("bf16", 1, 48, 513, 64), ("bf16", 1, 124, 2050, 64), ("bf16", 1, 48, 513, 32),
         ("f32", 1, 120, 513, 32), ("f32", 1, 120, 513, 64), ("f32", 1, 120, 513, 128)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("size", [1e2, 1e3, 1e6, 1e10])
@pytest.mark.parametrize("at", [5, 300])
def test_one_key_above_all_others(prism, case, size, at):  # noqa: F811
    """The rows in front of it have equal scores and a p of 1 / (i + 1)."""
    import torch
    dt, B, heads, T, D = case
    G, half = heads // 2, H if dt == "bf16" else 0.0
    r = Rng(85, dt)
    v, do = r.vec(B, G, T, D), r.vec(B, heads, T, D)
    q = torch.full((B, heads, T, D), size, device="cuda").to(v.dtype)
    k = torch.zeros_like(v)
    k[:, :, at] = size
    o, lse = prism.attn_fwd(q, k, v)
    top = v[:, :, at].repeat_interleave(2, 1)
    assert torch.equal(o[:, :, at:], top[:, :, None].expand(-1, -1, T - at, -1))
    score = float(q[0, 0, 0, 0]) * float(k[0, 0, at, 0]) * D ** 0.5
    assert bool(((lse[:, :, at:].double() - score).abs() <= (D + 8) * U * score).all())
    n = torch.arange(1, at + 1, device="cuda", dtype=torch.float64)
    assert bool(((lse[:, :, :at].double() - n.log()).abs() <= 32 * U).all())
    vd = v.repeat_interleave(2, 1)[:, :, :at].double()
    mean, size_o = vd.cumsum(2) / n[:, None], vd.abs().cumsum(2) / n[:, None]
    assert bool(((o[:, :, :at].double() - mean).abs() <= half * mean.abs() + (half + 8 * U + 3 * T * U) * size_o).all())
    g = prism.attn_bwd(q, k, v, o, lse, do)
    x = do.double()

    def summed(x):
        share = x[:, :, :at] / n[:, None]
        front = share.flip(2).cumsum(2).flip(2)                        # keys in front: the rows from each on
        y = torch.cat([front, x[:, :, at:].sum(2, keepdim=True), torch.zeros_like(x[:, :, at + 1:])], 2)
        return y.view(B, G, 2, T, D).sum(2)

    assert bool(((g["dv"].double() - summed(x)).abs() <= half * summed(x).abs() + (2 * T * U + 16 * U + half) * summed(x.abs())).all())
    # what is left of dp - <do, o> is the two sums' roundings, times key `at`; all other keys are zero
    left = 2.02 * D * U * (x.abs() * top[:, :, None].double().abs()).sum(-1, keepdim=True) * size * D ** -0.5 * (1 + half)
    assert bool((g["dq"][:, :, at:].double().abs() <= left[:, :, at:] * (1 + half)).all()) and bool((g["dq"][:, :, :at] == 0).all())
    assert bool(torch.isfinite(g["dk"]).all()) and bool((g["dk"][:, :, at + 1:] == 0).all())
