"""Float64 oracle of the state space layer: causal convolution, selective scan, root-mean-square norm, and
their gradients, stepped token by token in numpy from the definitions.  Shares no code with the library."""
import numpy as np


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(z, np.float64)))


def silu_grad(z):
    s = sigmoid(z)
    return s + z * s * (1.0 - s)


# ---- convolution: x [B, H, T, D], w [H, K, D], bias [H, D] ------------------------------------------
def conv(x, w, bias=None, silu=True, conv_in=None):
    """y and the last K - 1 rows of [conv_in; x]."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    B, H, T, D = x.shape
    K = w.shape[1]
    past = np.zeros((B, H, K - 1, D)) if conv_in is None else np.asarray(conv_in, np.float64)
    rows = np.concatenate([past, x], 2)
    y = np.empty((B, H, T, D))
    for t in range(T):
        pre = np.einsum("bhkd,hkd->bhd", rows[:, :, t:t + K], w)
        if bias is not None:
            pre = pre + bias[None]
        y[:, :, t] = pre * sigmoid(pre) if silu else pre
    return y, rows[:, :, T:]


def conv_grad(x, w, dy, bias=None, silu=True):
    x, w, dy = (np.asarray(v, np.float64) for v in (x, w, dy))
    B, H, T, D = x.shape
    K = w.shape[1]
    rows = np.concatenate([np.zeros((B, H, K - 1, D)), x], 2)
    drows, dw, db = np.zeros_like(rows), np.zeros_like(w), np.zeros((H, D))
    for t in range(T):
        win = rows[:, :, t:t + K]
        pre = np.einsum("bhkd,hkd->bhd", win, w) + (0.0 if bias is None else bias[None])
        g = dy[:, :, t] * (silu_grad(pre) if silu else 1.0)
        drows[:, :, t:t + K] += g[:, :, None] * w[None]
        dw += np.einsum("bhkd,bhd->hkd", win, g)
        db += g.sum(0)
    return {"dx": drows[:, :, K - 1:], "dconv_w": dw, "dbias": db}


# ---- scan: x [B, H, T, P], Bm / Cm [B, G, T, N], dt [B, H, T], A / D / bias [H] ------------------------
def _steps(dt, bias, softplus):
    z = np.asarray(dt, np.float64) + (0.0 if bias is None else np.asarray(bias, np.float64)[None, :, None])
    return z, (np.logaddexp(z, 0.0) if softplus else z)


def ssm(x, Bm, Cm, dt, A, D=None, bias=None, softplus=True, S0=None, decays=None):
    """y and the final state [B, H, N, P].  decays [B, H, T]: used in place of exp(d A) (for bounds on sums of
    absolute values)."""
    x, Bm, Cm = (np.asarray(v, np.float64) for v in (x, Bm, Cm))
    B, H, T, P = x.shape
    rep = H // Bm.shape[1]
    Bh, Ch = np.repeat(Bm, rep, 1), np.repeat(Cm, rep, 1)
    _, d = _steps(dt, bias, softplus)
    a = np.exp(d * np.asarray(A, np.float64)[None, :, None]) if decays is None else decays
    S = np.zeros((B, H, Bm.shape[3], P)) if S0 is None else np.array(S0, np.float64)
    y = np.empty((B, H, T, P))
    for t in range(T):
        S = a[:, :, t, None, None] * S + d[:, :, t, None, None] * Bh[:, :, t, :, None] * x[:, :, t, None, :]
        y[:, :, t] = np.einsum("bhnp,bhn->bhp", S, Ch[:, :, t])
        if D is not None:
            y[:, :, t] += np.asarray(D, np.float64)[None, :, None] * x[:, :, t]
    return y, S


def ssm_grad(x, Bm, Cm, dt, A, dy, D=None, bias=None, softplus=True, dS=None, absolute=False):
    """Gradients of <dy, y> + <dS, S_final> from a zero state.  absolute: every tensor and coefficient by its
    absolute value (the decays unchanged): the size of the sums behind each gradient, for error bounds."""
    x, Bm, Cm, dy, A = (np.asarray(v, np.float64) for v in (x, Bm, Cm, dy, A))
    z, d = _steps(dt, bias, softplus)
    a = np.exp(d * A[None, :, None])
    sg = sigmoid(z) if softplus else np.ones_like(z)
    if absolute:
        x, Bm, Cm, dy, d, A = (np.abs(v) for v in (x, Bm, Cm, dy, d, A))
        dS = None if dS is None else np.abs(dS)
        D = None if D is None else np.abs(D)
    B, H, T, P = x.shape
    G, N = Bm.shape[1], Bm.shape[3]
    rep = H // G
    Bh, Ch = np.repeat(Bm, rep, 1), np.repeat(Cm, rep, 1)
    S = np.zeros((T + 1, B, H, N, P))
    for t in range(T):
        S[t + 1] = a[:, :, t, None, None] * S[t] + d[:, :, t, None, None] * Bh[:, :, t, :, None] * x[:, :, t, None, :]
    R = np.zeros((B, H, N, P)) if dS is None else np.array(dS, np.float64)
    dx, dB, dC = np.zeros_like(x), np.zeros((B, H, T, N)), np.zeros((B, H, T, N))
    dd, dl = np.zeros((B, H, T)), np.zeros((B, H, T))
    for t in range(T - 1, -1, -1):
        R = R + Ch[:, :, t, :, None] * dy[:, :, t, None, :]
        dC[:, :, t] = np.einsum("bhnp,bhp->bhn", S[t + 1], dy[:, :, t])
        dB[:, :, t] = d[:, :, t, None] * np.einsum("bhnp,bhp->bhn", R, x[:, :, t])
        BR = np.einsum("bhnp,bhn->bhp", R, Bh[:, :, t])
        dx[:, :, t] = d[:, :, t, None] * BR + (0.0 if D is None else np.asarray(D)[None, :, None] * dy[:, :, t])
        dd[:, :, t] = (BR * x[:, :, t]).sum(-1)
        dl[:, :, t] = a[:, :, t] * (R * S[t]).sum((-1, -2))
        R = a[:, :, t, None, None] * R
    ddt = (dd + A[None, :, None] * dl) * sg
    return {"dx": dx, "dB": dB.reshape(B, G, rep, T, N).sum(2), "dC": dC.reshape(B, G, rep, T, N).sum(2), "ddt": ddt,
            "dA": (dl * d).sum((0, 2)), "dD": (x * dy).sum((0, 2, 3)), "ddt_bias": ddt.sum((0, 2))}


# ---- norm: rows in the last axis -----------------------------------------------------------------------
def norm(x, weight=None, residual=None, gate=None, eps=1e-5):
    """y and h."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if gate is not None:
        z = np.asarray(gate, np.float64)
        y = y * z * sigmoid(z)
    return y, h


def norm_grad(h, dy, weight=None, gate=None, dh_in=None, eps=1e-5):
    h, dy = np.asarray(h, np.float64), np.asarray(dy, np.float64)
    D = h.shape[-1]
    w = np.ones(D) if weight is None else np.asarray(weight, np.float64)
    rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    out, u = {}, dy
    if gate is not None:
        z = np.asarray(gate, np.float64)
        out["dgate"] = dy * w * h / rms * silu_grad(z)
        u = dy * z * sigmoid(z)
    out["dw"] = (u * h / rms).reshape(-1, D).sum(0)
    out["dh"] = u * w / rms - h * (u * w * h).mean(-1, keepdims=True) / rms ** 3
    if dh_in is not None:
        out["dh"] = out["dh"] + np.asarray(dh_in, np.float64)
    return out
