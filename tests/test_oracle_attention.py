"""The attention layer's oracle against closed forms, library routines and finite differences."""
import numpy as np
import pytest
import torch

from oracle import attention as A


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    r = np.random.default_rng(0)
    x, freq, pos = r.standard_normal((2, 3, 5, 16)), r.uniform(0, 1, 6), r.integers(0, 1 << 20, (2, 5))
    y = A.rope(x, pos, freq, interleaved=interleaved, factor=1.5)
    a, b = (np.arange(0, 12, 2), np.arange(1, 12, 2)) if interleaved else (np.arange(6), np.arange(6, 12))
    z = 1.5 * (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None, :, None] * freq)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-9)
    np.testing.assert_array_equal(y[..., 12:], x[..., 12:])


def test_scores_depend_on_distance_only():
    r = np.random.default_rng(1)
    q, k, freq = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8)), r.uniform(0, 1, 4)
    s = [float((A.rope(q, [[i]], freq) * A.rope(k, [[j]], freq)).sum()) for i, j in ((7, 3), (104, 100), (4, 0))]
    np.testing.assert_allclose(s, s[0], rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_grad_by_differences(interleaved, norm):
    r = np.random.default_rng(2)
    x, dy, w = r.standard_normal((2, 2, 3, 8)), r.standard_normal((2, 2, 3, 8)), (r.standard_normal(8) if norm else None)
    freq, pos, h = r.uniform(0, 1, 3), r.integers(0, 100, (2, 3)), 1e-6
    f = lambda x, w: float((A.rope(x, pos, freq, w, 1e-3, interleaved, 0.7) * dy).sum())  # noqa: E731
    dx, dw = A.rope_grad(x, dy, pos, freq, w, 1e-3, interleaved, 0.7)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(8 if norm else 0):
        e = np.eye(8)[i] * h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (True, 1), (False, 0)])
def test_attention_and_grad(causal, window):
    r = np.random.default_rng(3)
    q, k, v, do = (r.standard_normal((9, 4)) for _ in range(4))
    leaves = [torch.tensor(t, requires_grad=True) for t in (q, k, v)]
    ok = torch.tensor(A.visible(9, 9, causal, window))
    o = torch.nn.functional.scaled_dot_product_attention(*(t[None, None] for t in leaves), attn_mask=ok, scale=0.3)[0, 0]
    np.testing.assert_allclose(A.attention(q, k, v, 0.3, causal, window)[0], o.detach().numpy(), atol=1e-12)
    for got, ref in zip(A.attention_grad(q, k, v, do, 0.3, causal, window), torch.autograd.grad(o, leaves, torch.tensor(do))):
        np.testing.assert_allclose(got, ref.numpy(), atol=1e-12)
    h = 1e-6
    for n in range(3):
        g = A.attention_grad(q, k, v, do, 0.3, causal, window)[n]
        for i in np.ndindex(3, 4):
            x = [q.copy(), k.copy(), v.copy()]
            f = []
            for s in (h, -2 * h):
                x[n][i] += s
                f.append(float((A.attention(*x, 0.3, causal, window)[0] * do).sum()))
            assert abs((f[0] - f[1]) / (2 * h) - g[i]) < 1e-7


def test_rows_that_see_nothing():
    q, k = np.ones((2, 4)), np.ones((3, 4))
    o, lse = A.attention(q, k, k, 1.0, past=-2)
    assert (o[0] == 0).all() and np.isneginf(lse[0])
    o, lse = A.attention(q, k[:0], k[:0], 1.0)
    assert (o == 0).all() and np.isneginf(lse).all()


def test_lse_of_equal_scores():
    q, k = np.zeros((5, 4)), np.ones((5, 4))
    np.testing.assert_allclose(A.attention(q, k, k, 1.0)[1], np.log(np.arange(1, 6)))


def test_positions_of_a_chunk():
    r = np.random.default_rng(4)
    q, k, v = (r.standard_normal((12, 4)) for _ in range(3))
    whole = A.attention(q, k, v, 0.5, window=5)[0]
    np.testing.assert_allclose(A.attention(q[7:10], k[:10], v[:10], 0.5, window=5, past=7)[0], whole[7:10])


def test_e4m3_values():
    v = A.e4m3_values()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(v, ref)
