"""How far a row that is not finite reaches in the gradients of attention.

Row i of o sees the keys i - window + 1 .. i, so a key or value j enters the rows j .. j + window - 1, and through them the keys from
j - window + 1 to j + window - 1; a query's or an o's gradient i enters row i and the keys that it sees.  The kernels may spoil
tokens within 256 of these; all others are what they are without the value, within the tolerances of test_attention_gpu.
"""
import numpy as np
import pytest

from tests.test_attention_gpu import Rng, check_grads, f64, prism  # noqa: F401

pytestmark = pytest.mark.gpu
NEAR = 256

# workgroups of many rows and of 32 for each type and width; tokens in front of a workgroup's window, at its edges and in its middle
CASES = [("bf16", 128, 24, 12, 768, 2, 448), ("bf16", 128, 24, 12, 1000, 40, 420), ("bf16", 128, 24, 12, 800, 1, 511), ("bf16", 128, 2, 1, 800, 2, 448),
         ("bf16", 64, 40, 20, 900, 2, 448), ("bf16", 64, 40, 20, 900, 70, 300), ("bf16", 64, 2, 1, 900, 33, 448), ("bf16", 32, 40, 20, 900, 2, 448),
         ("bf16", 32, 3, 1, 700, 5, 383), ("f32", 64, 40, 20, 900, 2, 448), ("f32", 64, 2, 1, 700, 64, 320), ("f32", 128, 96, 48, 768, 2, 448),
         ("f32", 128, 2, 1, 700, 2, 448), ("f32", 32, 2, 1, 700, 9, 350)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_gradients_beyond_a_row_that_is_not_finite(prism, case, which, value):  # noqa: F811
    import torch
    dt, D, heads, G, T, window, at = case
    r = Rng(81, dt)
    q, k, v = r.heads(1, T, heads, G, G, D=D)
    do = r.vec(1, heads, T, D)
    x = {"q": q, "k": k, "v": v, "do": do}

    def run():
        o, lse = prism.attn_fwd(q, k, v, window=window)
        return prism.attn_bwd(q, k, v, o, lse, do, window=window)

    inputs = [f64(t) for t in (q[0, :heads // G], k[0, 0], v[0, 0], do[0, :heads // G])]
    clean = run()
    x[which][0, 0, at, 3] = value
    got = run()
    rows = (at, at + window - 1) if which in "kv" else (at, at)        # the rows that it enters, and the keys that these see
    keys = (rows[0] - window + 1, rows[1])
    t, group = np.arange(T), []
    for name, (lo, hi) in (("dq", rows), ("dk", keys), ("dv", keys)):
        far = torch.tensor((t < lo - NEAR) | (t > hi + NEAR), device="cuda")
        rep = heads // G if name == "dq" else 1
        ok = torch.isfinite(got[name][0, :rep]).all(-1) | ~far
        assert bool(far.any()) and bool(ok.all()), f"{name}: tokens {torch.nonzero(~ok)[:, 1].unique().tolist()}"
        assert torch.equal(got[name][:, rep:], clean[name][:, rep:]), f"{name}: another group"
        group.append(f64(torch.where(far[:, None], got[name][0, :rep], clean[name][0, :rep])))
    check_grads(name, dt, *inputs, float(np.float32(1 / np.sqrt(D))), [group[0], group[1][0], group[2][0]], window=window)
    if which == "k" and np.isnan(value):
        assert not torch.isfinite(got["dq"][0, 0, at:at + window]).any()
