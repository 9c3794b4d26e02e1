"""Float64 oracle of the attention layer: norm and rotation of heads, softmax attention and its gradients, and the
8-bit rows of the cache, in numpy from the definitions.  Shares no code with the library."""
import numpy as np


# ---- norm and rotation: x [B, H, T, D], pos [B, T], freq [rot / 2] -----------------------------------------
def _channels(freq, interleaved):
    n = len(freq)
    i = np.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, n + i)


def _rotated(x, pos, freq, interleaved, factor, sign):
    angle = np.asarray(pos, np.float64)[:, None, :, None] * np.asarray(freq, np.float64)
    a, b = _channels(freq, interleaved)
    y = x.copy()
    y[..., a] = factor * (x[..., a] * np.cos(angle) - sign * x[..., b] * np.sin(angle))
    y[..., b] = factor * (x[..., b] * np.cos(angle) + sign * x[..., a] * np.sin(angle))
    return y


def rope(x, pos, freq, w=None, eps=1e-6, interleaved=False, factor=1.0):
    h = np.asarray(x, np.float64)
    if w is not None:
        h = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    return _rotated(h, pos, freq, interleaved, factor, 1.0)


def rope_grad(x, dy, pos, freq, w=None, eps=1e-6, interleaved=False, factor=1.0):
    """dx, dw (None without w) of <dy, y>."""
    g = _rotated(np.asarray(dy, np.float64), pos, freq, interleaved, factor, -1.0)
    if w is None:
        return g, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = g * w
    return u / rms - x * (u * x).mean(-1, keepdims=True) / rms ** 3, (g * x / rms).sum((0, 1, 2))


# ---- attention of one head: q [T, D], k, v [n, D]; token t has position past + t -------------------------------
def visible(T, n, causal=True, window=0, past=0):
    i, j = past + np.arange(T)[:, None], np.arange(n)[None]
    ok = np.ones((T, n), bool)
    if causal:
        ok &= j <= i
    if window:
        ok &= j > i - window
    return ok


def probabilities(q, k, scale, ok):
    """p and lse; a row that sees nothing: zeros and -inf."""
    with np.errstate(invalid="ignore"):
        s = np.where(ok, (q @ k.T) * scale, -np.inf)
    m = s.max(1, initial=-np.inf, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.where(ok, np.exp(s - m), 0.0)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        return e / np.where(total > 0, total, 1.0), (m + np.log(total))[:, 0]


def attention(q, k, v, scale, causal=True, window=0, past=0):
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    p, lse = probabilities(q, k, scale, visible(len(q), len(k), causal, window, past))
    return p @ v, lse


def attention_grad(q, k, v, do, scale, causal=True, window=0):
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    p, _ = probabilities(q, k, scale, visible(len(q), len(k), causal, window))
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdims=True))
    return scale * ds @ k, scale * ds.T @ q, p.T @ do


# ---- rows of the 8-bit cache -----------------------------------------------------------------------------------
def e4m3_values():
    """The value of each byte (OCP e4m3: 4 exponent bits of bias 7, 3 of mantissa, no infinities)."""
    b = np.arange(256)
    sign, ex, man = np.where(b & 128, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = sign * np.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * 2.0 ** (ex - 7.0))
    return np.where((b & 127) == 127, np.nan, v)
