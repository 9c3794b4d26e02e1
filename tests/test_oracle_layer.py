"""The state space layer's oracle against closed forms and finite differences (CPU)."""
import numpy as np
import pytest

from oracle import layer


def directional(f, args, name, grad, rng, eps=1e-6):
    """|central difference - <grad, direction>| relative to the gradient's norm along a random direction."""
    v = rng.standard_normal(args[name].shape)
    hi, lo = dict(args), dict(args)
    hi[name], lo[name] = args[name] + eps * v, args[name] - eps * v
    num = (f(**hi) - f(**lo)) / (2 * eps)
    ana = float((grad * v).sum())
    return abs(num - ana) / max(1.0, abs(ana))


@pytest.mark.parametrize("K,silu", [(2, True), (4, True), (3, False)])
def test_conv_gradients(K, silu):
    rng = np.random.default_rng(K)
    args = {"x": rng.standard_normal((2, 2, 7, 3)), "w": rng.standard_normal((2, K, 3)), "bias": rng.standard_normal((2, 3))}
    dy = rng.standard_normal((2, 2, 7, 3))
    g = layer.conv_grad(args["x"], args["w"], dy, args["bias"], silu)
    f = lambda x, w, bias: float((layer.conv(x, w, bias, silu)[0] * dy).sum())  # noqa: E731
    for name, key in (("x", "dx"), ("w", "dconv_w"), ("bias", "dbias")):
        assert directional(f, args, name, g[key], rng) < 1e-7


@pytest.mark.parametrize("softplus", [True, False])
def test_ssm_gradients(softplus):
    rng = np.random.default_rng(3)
    B, H, G, T, N, P = 2, 4, 2, 9, 3, 2
    args = {"x": rng.standard_normal((B, H, T, P)), "Bm": rng.standard_normal((B, G, T, N)),
            "Cm": rng.standard_normal((B, G, T, N)), "dt": 0.5 + 0.3 * rng.random((B, H, T)), "A": -rng.random(H),
            "D": rng.standard_normal(H), "bias": 0.1 * rng.standard_normal(H)}
    dy, dS = rng.standard_normal((B, H, T, P)), rng.standard_normal((B, H, N, P))
    g = layer.ssm_grad(args["x"], args["Bm"], args["Cm"], args["dt"], args["A"], dy, args["D"], args["bias"], softplus, dS)

    def f(**k):
        y, S = layer.ssm(k["x"], k["Bm"], k["Cm"], k["dt"], k["A"], k["D"], k["bias"], softplus)
        return float((y * dy).sum() + (S * dS).sum())

    for name, key in (("x", "dx"), ("Bm", "dB"), ("Cm", "dC"), ("dt", "ddt"), ("A", "dA"), ("D", "dD"), ("bias", "ddt_bias")):
        assert directional(f, args, name, g[key], rng) < 1e-7, name


@pytest.mark.parametrize("gate,weight", [(True, True), (False, True), (False, False)])
def test_norm_gradients(gate, weight):
    rng = np.random.default_rng(5)
    args = {"h": rng.standard_normal((4, 6))}
    if weight:
        args["weight"] = rng.standard_normal(6)
    if gate:
        args["gate"] = rng.standard_normal((4, 6))
    dy, dh = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))
    g = layer.norm_grad(dy=dy, dh_in=dh, **args)
    f = lambda h, weight=None, gate=None: float((layer.norm(h, weight, None, gate)[0] * dy).sum() + (h * dh).sum())  # noqa: E731
    assert directional(f, args, "h", g["dh"], rng) < 1e-7
    if weight:
        assert directional(f, args, "weight", g["dw"], rng) < 1e-7
    if gate:
        assert directional(f, args, "gate", g["dgate"], rng) < 1e-7


def test_ssm_is_the_delta_rule_without_erase():
    """With beta = 0 the recurrence's erase and its own write vanish; a write of d B x^T with decay exp(d A) is the
    scan, and with decay 1 it is linear attention: y_t = sum_{s<=t} (C_t . B_s) d_s x_s."""
    rng = np.random.default_rng(6)
    x, Bm, Cm = rng.standard_normal((1, 2, 8, 3)), rng.standard_normal((1, 1, 8, 4)), rng.standard_normal((1, 1, 8, 4))
    dt = rng.random((1, 2, 8))
    y, S = layer.ssm(x, Bm, Cm, dt, np.zeros(2), softplus=False)
    score = np.tril(Cm[0, 0] @ Bm[0, 0].T)
    for h in range(2):
        np.testing.assert_allclose(y[0, h], (score * dt[0, h][None]) @ x[0, h], atol=1e-12)
        np.testing.assert_allclose(S[0, h], (Bm[0, 0] * dt[0, h][:, None]).T @ x[0, h], atol=1e-12)


def test_ssm_continues_from_a_state():
    rng = np.random.default_rng(7)
    x, Bm, Cm = rng.standard_normal((2, 2, 10, 3)), rng.standard_normal((2, 2, 10, 4)), rng.standard_normal((2, 2, 10, 4))
    dt, A = rng.standard_normal((2, 2, 10)), -rng.random(2)
    y, S = layer.ssm(x, Bm, Cm, dt, A)
    y1, S1 = layer.ssm(x[:, :, :4], Bm[:, :, :4], Cm[:, :, :4], dt[:, :, :4], A)
    y2, S2 = layer.ssm(x[:, :, 4:], Bm[:, :, 4:], Cm[:, :, 4:], dt[:, :, 4:], A, S0=S1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 2), y, atol=1e-13)
    np.testing.assert_allclose(S2, S, atol=1e-13)


def test_conv_continues_from_its_rows():
    rng = np.random.default_rng(8)
    x, w = rng.standard_normal((2, 1, 9, 5)), rng.standard_normal((1, 4, 5))
    y, end = layer.conv(x, w)
    y1, mid = layer.conv(x[:, :, :2], w)
    y2, end2 = layer.conv(x[:, :, 2:], w, conv_in=mid)
    np.testing.assert_allclose(np.concatenate([y1, y2], 2), y, atol=1e-14)
    np.testing.assert_array_equal(end, end2)
