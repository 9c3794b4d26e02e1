"""The attention layer on the GPU against its float64 oracle.

Tolerances are element-wise, |got - ref| <= a |ref| + b size, `size` being the same sum over absolute values.  A half step
is u = 2^-24 (float32), h = 2^-8 (bfloat16).
* scores: D products and their sum in float32 and three roundings of the exponent's argument: off by at most
  e_s = (D + 8) u max_j scale <|q|, |k_j|>, in the exponent; the hardware's 2^x adds 4 u: a probability is off by e_p = e_s + 8 u
  relative to itself, and once more that through the row's sum of n terms: 2 e_p + 2 n u.
* o: that times sum p |v|, the sum over n keys (n u), and for bfloat16 p's own rounding (h) and o's (a = h).
* lse: e_p + n u + 4 u (1 + |lse|).
* gradients: p by e_g = e_p + 4 u |lse| (lse is given in float32); dp and <do, o> by 2 D u of their sums of absolute values, o itself
  by h for bfloat16: with size_ds = p (<|do|, |v|> + <|do|, |o|>), ds is off by (e_g + 2 D u [+ h for o] [+ h for ds]) size_ds;
  dq, dk, dv add their sums over n terms (n u) and roundings (a = h); dv has p in place of ds.
* rotation: float32 arithmetic; angles within 2^-23, the row's sum of squares D u, a few roundings: (D + 32) u + 2^-22.
"""
import numpy as np
import pytest

from oracle import attention as A
from tests.conftest import gpu_available

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def prism():
    if not gpu_available():
        pytest.skip("no GPU")
    import delta_rule_sequence_amd as m
    m.load_library()
    return m


def torch_dtype(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


class Rng:
    """Tensors on the GPU and the values they hold in float64."""

    def __init__(self, seed, dt):
        self.r, self.dt = np.random.default_rng(seed), torch_dtype(dt)

    def vec(self, *shape, scale=1.0):
        import torch
        return torch.tensor(scale * self.r.standard_normal(shape), dtype=torch.float32, device="cuda").to(self.dt)

    def heads(self, B, T, *counts, D):
        """[B, heads, T, D] views of one token-major tensor, as a projection leaves them."""
        rows = self.vec(B, T, sum(counts), D)
        return [t.transpose(1, 2) for t in rows.split(counts, 2)]

    def flt(self, *shape, lo=0.0, hi=1.0):
        import torch
        return torch.tensor(self.r.uniform(lo, hi, shape), dtype=torch.float32, device="cuda")


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, size, b, a=0.0):
    got, ref = f64(got) if not isinstance(got, np.ndarray) else got, np.asarray(ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    lim = a * np.abs(ref) + b * np.asarray(size) + 1e-30
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= lim) & ~((got == ref) & np.isinf(ref))
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} values outside, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}"


def check_head(name, dt, q, k, v, scale, o, lse=None, causal=True, window=0, past=0, extra=0.0):
    """One head's rows [T, D] against the definition.  extra: relative error of the keys' and values' scales."""
    D, n = q.shape[1], len(k)
    ref, ref_lse = A.attention(q, k, v, scale, causal, window, past)
    ok = A.visible(len(q), n, causal, window, past)
    p, _ = A.probabilities(q, k, scale, ok)
    e_s = (D + 8) * U * (scale * np.abs(q) @ np.abs(k).T * ok).max(1, initial=0.0)[:, None]
    e_p = e_s + 8 * U + extra * (1 + e_s / ((D + 8) * U))
    rounding = H if dt == "bf16" else 0.0
    close(name + ".o", o, ref, p @ np.abs(v), 2 * e_p + 3 * n * U + extra + rounding, rounding)
    if lse is not None:
        close(name + ".lse", lse, ref_lse, np.ones(len(q)), (e_p + n * U)[:, 0] + 4 * U * (1 + np.where(np.isinf(ref_lse), 0, np.abs(ref_lse))))
    return ref


def check_grads(name, dt, q, k, v, do, scale, got, causal=True, window=0):
    """One group: q, do [rep, T, D], k, v [T, D]; got: dq [rep, T, D], dk, dv [T, D]."""
    rep, T, D = q.shape
    r = H if dt == "bf16" else 0.0
    ref_k, ref_v, size_k, size_v, worst = 0, 0, 0, 0, 0.0
    for i in range(rep):
        dq, dk, dv = A.attention_grad(q[i], k, v, do[i], scale, causal, window)
        ok = A.visible(T, T, causal, window)
        p, lse = A.probabilities(q[i], k, scale, ok)
        o = p @ v
        e_g = float(((D + 8) * U * (scale * np.abs(q[i]) @ np.abs(k).T * ok)).max() + 8 * U + 4 * U * np.abs(lse).max())
        ds = p * (np.abs(do[i]) @ np.abs(v).T + (np.abs(do[i]) * np.abs(o)).sum(1)[:, None])
        e_d = e_g + 2 * D * U + 2 * r + T * U
        close(f"{name}.dq[{i}]", got[0][i], dq, scale * ds @ np.abs(k), e_d, r)
        ref_k, ref_v = ref_k + dk, ref_v + dv
        size_k, size_v = size_k + scale * ds.T @ np.abs(q[i]), size_v + p.T @ np.abs(do[i])
        worst = max(worst, e_g)
    n = rep * T * U
    close(name + ".dk", got[1], ref_k, size_k, worst + 2 * D * U + 2 * r + n, r)
    close(name + ".dv", got[2], ref_v, size_v, worst + r + n, r)


def check_prompt(dt, q, k, v, o, lse, spans, scale, causal=True, window=0, do=None, grads=None):
    """spans: (batch, first token, tokens) of each sequence."""
    rep = q.shape[1] // k.shape[1]
    x = [f64(t) for t in (q, k, v)] + ([f64(do)] if do is not None else [])
    for b, lo, n in spans:
        for g in range(k.shape[1] if n else 0):
            for h in range(g * rep, (g + 1) * rep):
                check_head(f"[{b},{h}]", dt, x[0][b, h, lo:lo + n], x[1][b, g, lo:lo + n], x[2][b, g, lo:lo + n], scale,
                           f64(o[b, h, lo:lo + n]), f64(lse[b, h, lo:lo + n]), causal, window)
            if grads is not None:
                hs = slice(g * rep, (g + 1) * rep)
                check_grads(f"[{b},{g}]", dt, x[0][b, hs, lo:lo + n], x[1][b, g, lo:lo + n], x[2][b, g, lo:lo + n],
                            x[3][b, hs, lo:lo + n], scale, [f64(grads["dq"][b, hs, lo:lo + n]), f64(grads["dk"][b, g, lo:lo + n]),
                                                           f64(grads["dv"][b, g, lo:lo + n])], causal, window)


# ---- prompts -----------------------------------------------------------------------------------
PROMPT = [("bf16", 1, 1, 1, 1, 64, 0), ("bf16", 2, 3, 1, 2, 32, 0), ("bf16", 1, 2, 2, 31, 128, 0), ("bf16", 1, 4, 2, 32, 64, 0),
          ("bf16", 1, 2, 1, 33, 32, 1), ("bf16", 2, 2, 1, 63, 64, 5), ("bf16", 1, 1, 1, 65, 128, 64), ("bf16", 1, 8, 1, 127, 64, 0),
          ("bf16", 1, 6, 2, 129, 128, 0), ("bf16", 1, 2, 1, 257, 64, 100), ("bf16", 1, 2, 1, 300, 32, 1000), ("bf16", 1, 2, 1, 515, 128, 33),
          ("f32", 1, 1, 1, 1, 32, 0), ("f32", 2, 2, 1, 33, 64, 0), ("f32", 1, 3, 1, 95, 128, 0), ("f32", 1, 2, 2, 129, 32, 17),
          ("f32", 1, 4, 1, 200, 64, 64), ("f32", 1, 2, 1, 261, 128, 2)]


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(prism, case, causal):
    dt, B, heads, G, T, D, window = case
    window = window if causal else 0
    r = Rng(10 + T, dt)
    q, k, v = r.heads(B, T, heads, G, G, D=D)
    do, scale = r.vec(B, heads, T, D), 0.7 / np.sqrt(D)
    o, lse = prism.attn_fwd(q, k, v, scale=scale, causal=causal, window=window)
    g = prism.attn_bwd(q, k, v, o, lse, do, scale=scale, causal=causal, window=window)
    check_prompt(dt, q, k, v, o, lse, [(b, 0, T) for b in range(B)], float(np.float32(scale)), causal, window, do, g)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 40])
def test_padded_batch(prism, dt, window):
    import torch
    heads, G, T, D = 4, 2, 150, 64
    lens = [0, 1, 33, 149, 150, 500, -3]
    r = Rng(11, dt)
    q, k, v = r.heads(len(lens), T, heads, G, G, D=D)
    do = r.vec(len(lens), T, heads, D).transpose(1, 2)
    for b, n in enumerate(lens):                             # rows past a length are never read
        for t in (q, k, v, do):
            t[b, :, max(n, 0):] = float("nan")
    o = torch.full((len(lens), T, heads, D), 7.0, dtype=q.dtype, device="cuda").transpose(1, 2)
    lse = torch.full((len(lens), heads, T), 7.0, device="cuda")
    got = prism.attn_fwd(q, k, v, window=window, lens=i32(lens), out=(o, lse))
    assert got[0] is o and got[1] is lse
    out = [torch.full_like(t, 5.0) for t in (q, k, v)]
    g = prism.attn_bwd(q, k, v, o, lse, do, window=window, lens=i32(lens), out=out)
    z = prism.attn_bwd(q, k, v, o, lse, do, window=window, lens=i32(lens))
    spans = [(b, 0, min(max(n, 0), T)) for b, n in enumerate(lens)]
    check_prompt(dt, q, k, v, o, lse, spans, float(np.float32(1 / np.sqrt(D))), True, window, do, g)
    for b, _, n in spans:
        assert bool((o[b, :, n:] == 7).all()) and bool((lse[b, :, n:] == 7).all())
        for name in ("dq", "dk", "dv"):
            assert bool((g[name][b, :, n:] == 5).all()) and bool((z[name][b, :, n:] == 0).all()), name
            assert torch.equal(g[name][b, :, :n], z[name][b, :, :n])


STARTS = {"gaps": [3, 3, 40, 41, 200, 200, 290], "past the end": [0, 100, 310, 400], "many": list(range(0, 301, 2)),
          "none": [300, 300], "one": [0, 300], "negative": [-7, 20, 300]}


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", STARTS)
def test_packed(prism, dt, name):
    import torch
    heads, G, T, D, at = 4, 2, 300, 64, STARTS[name]
    r = Rng(12, dt)
    q, k, v = r.heads(1, T, heads, G, G, D=D)
    do = r.vec(1, heads, T, D)
    lo = np.clip(at, 0, T)
    outside = np.ones(T, bool)
    outside[lo[0]:lo[-1]] = False
    for t in (q, k, v, do):
        t[:, :, torch.tensor(outside, device="cuda")] = float("nan")
    o, lse = torch.full_like(q, 7.0), torch.full((1, heads, T), 7.0, device="cuda")
    prism.attn_fwd(q, k, v, starts=i32(at), out=(o, lse))
    out = [torch.full_like(t, 5.0) for t in (q, k, v)]
    g = prism.attn_bwd(q, k, v, o, lse, do, starts=i32(at), out=out)
    spans = [(0, a, b - a) for a, b in zip(lo, lo[1:])]
    check_prompt(dt, q, k, v, o, lse, spans, float(np.float32(1 / np.sqrt(D))), True, 0, do, g)
    sel = torch.tensor(outside, device="cuda")
    assert bool((o[:, :, sel] == 7).all()) and bool((lse[:, :, sel] == 7).all())
    assert all(bool((g[n][:, :, sel] == 5).all()) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_growing_scores(prism, dt):
    """Scores that rise and fall by hundreds from tile to tile move the running maximum every time."""
    import torch
    T, D = 400, 64
    r = Rng(13, dt)
    q, k, v = r.vec(1, 1, T, D), r.vec(1, 1, T, D), r.vec(1, 1, T, D)
    k *= torch.tensor(np.where(np.arange(T) // 32 % 3 == 1, 40.0, np.linspace(0.1, 20, T)), device="cuda").to(k.dtype)[:, None]
    do = r.vec(1, 1, T, D)
    o, lse = prism.attn_fwd(q, k, v)
    g = prism.attn_bwd(q, k, v, o, lse, do)
    check_prompt(dt, q, k, v, o, lse, [(0, 0, T)], 0.125, do=do, grads=g)


def test_equal_and_extreme_scores(prism):
    import torch
    T, D = 100, 32
    v = Rng(14, "f32").vec(1, 1, T, D)
    zero = torch.zeros(1, 1, T, D, device="cuda")
    o, lse = prism.attn_fwd(zero, zero, v)
    ref = np.cumsum(f64(v)[0, 0], 0) / np.arange(1, T + 1)[:, None]
    close("mean", o[0, 0], ref, np.cumsum(np.abs(f64(v)[0, 0]), 0) / np.arange(1, T + 1)[:, None], 4 * T * U)
    close("lse", lse[0, 0], np.log(np.arange(1, T + 1)), np.ones(T), 32 * U)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e4, 1e6, 1e10])
def test_one_key_above_all_others(prism, dt, size):
    """Scores of 10^6 to 10^20, where a rounding of the exponent's argument is worth thousands: the largest one's p is 1, all
    others' 0, so o, dq, dk and dv are sums of inputs."""
    import torch
    T, D = 100, 32
    r = Rng(18, dt)
    v, do = r.vec(1, 1, T, D), r.vec(1, 1, T, D)
    q = torch.full((1, 1, T, D), size, device="cuda").to(v.dtype)
    k = torch.zeros_like(q)
    k[:, :, 5] = size
    o, lse = prism.attn_fwd(q, k, v)
    assert torch.equal(o[0, 0, 5:], v[0, 0, 5].expand(T - 5, D))
    top = f64(q)[0, 0, 0] @ f64(k)[0, 0, 5] / np.sqrt(D)
    assert (np.abs(f64(lse)[0, 0, 5:] - top) <= (D + 8) * U * top).all()
    g = prism.attn_bwd(q, k, v, o, lse, do)
    x = f64(do)[0, 0]

    def summed(x):                                             # rows in front of it: equal scores
        mean = [x[i] / (i + 1) for i in range(5)]
        return np.array([sum(mean[j:]) if j < 5 else x[5:].sum(0) if j == 5 else 0 * x[0] for j in range(T)])

    half = H if dt == "bf16" else 0.0
    close("dv", g["dv"][0, 0], summed(x), summed(np.abs(x)), T * U + 8 * U + half, half)
    # what is left of dp - <do, o> are the two sums' roundings
    lim = 2 * D * U * (np.abs(x) @ np.abs(f64(v)[0, 0, 5])) * size / np.sqrt(D)
    assert (np.abs(f64(g["dq"])[0, 0, 5:]) <= 1.01 * lim[5:, None]).all() and (f64(g["dq"])[0, 0, :5] == 0).all()
    o = prism.attn_paged(q, *(t.reshape(1, 1, T, D).repeat(1, 1, 2, 1)[:, :, :128].contiguous() for t in (k, v)), i32([[0]]), i32([0]))
    assert torch.equal(o[0, 0, 5:], v[0, 0, 5].expand(T - 5, D))


def by_rows(dt, q, k, v, o, lse=None, window=0, past=0):
    """Each row against the definition over the keys that it sees, so that non-finite ones reach what they enter only."""
    for t in range(len(q)):
        lo, hi = max(0, past + t - window + 1) if window else 0, past + t + 1
        kk, vv = k[lo:hi], v[lo:hi]
        if np.isfinite(q[t]).all() and np.isfinite(kk).all() and np.isfinite(vv).all():
            check_head(f"row {t}", dt, q[t:t + 1], kk, vv, 1 / np.sqrt(q.shape[1]), o[t:t + 1], None if lse is None else lse[t:t + 1], past=hi)
        elif np.isfinite(q[t]).all() and np.isfinite(kk).all():            # values alone: their columns alone
            bad = ~np.isfinite(vv).all(0)
            assert (~np.isfinite(o[t]) == bad).all(), t
        else:
            assert np.isnan(o[t]).all(), t


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 20])
def test_non_finite_rows_reach_what_they_enter(prism, dt, window):
    import torch
    T, D = 200, 64
    r = Rng(15, dt)
    q, k, v = r.vec(2, 2, T, D), r.vec(2, 2, T, D), r.vec(2, 2, T, D)
    v[0, 1, 130, 5] = float("inf")
    v[0, 1, 131, 6] = float("nan")
    k[0, 0, 130] = float("nan")
    v[0, 0, 150] = -float("inf")
    q[1, 0, 7] = float("nan")
    v[1, 1, 0] = float("nan")
    o, lse = prism.attn_fwd(q, k, v, window=window)
    for b in range(2):
        for h in range(2):
            by_rows(dt, *(f64(t[b, h]) for t in (q, k, v, o, lse)), window=window)
    table, past = i32([[3, 1, 0, 2], [7, 4, 5, 6]]), i32([120, 0])         # the same rows from the cache, and a chunk of them
    ck, cv = (torch.zeros(8, 2, 64, D, dtype=q.dtype, device="cuda") for _ in range(2))
    prism.cache_write(ck, cv, k, v, table, i32([0, 0]))
    for n in (10, 70):
        c = prism.attn_paged(torch.stack([q[0, :, 120:120 + n], q[1, :, :n]]), ck, cv, table, past, window=window)
        for b in range(2):
            for h in range(2):
                first = [120, 0][b]
                by_rows(dt, f64(q[b, h, first:first + n]), f64(k[b, h]), f64(v[b, h]), f64(c[b, h]), window=window, past=first)


def test_far_strides(prism):
    """Rows further apart than 32-bit offsets reach."""
    import torch
    T, D, step = 300, 32, 1 << 23                              # bfloat16 rows 16 MB apart: 5 GB
    flat = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    r = Rng(16, "bf16")
    parts = [flat.as_strided((1, 1, T, D), (T * step, D, step, 1), i * D) for i in range(5)]
    dense = [r.vec(1, 1, T, D) for _ in range(4)]
    for p, d in zip(parts, dense):
        p.copy_(d)
    o, lse = prism.attn_fwd(*parts[:3], out=(parts[4], torch.empty(1, 1, T, device="cuda")))
    o2, lse2 = prism.attn_fwd(*dense[:3])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = prism.attn_bwd(*parts[:3], o, lse, parts[3])
    g2 = prism.attn_bwd(*dense[:3], o2, lse2, dense[3])
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_long_sequence(prism):
    """One row of many tiles against the sum over all keys; every row of a group's heads alike."""
    import torch
    T, D = 20000, 64
    r = Rng(17, "bf16")
    q, k, v = r.heads(1, T, 2, 1, 1, D=D)
    o, lse = prism.attn_fwd(q, k, v)
    for t in (0, 63, 64, 8191, T - 1):
        check_head(f"row {t}", "bf16", f64(q[0, 1, t:t + 1]), f64(k[0, 0, :t + 1]), f64(v[0, 0, :t + 1]), 0.125, f64(o[0, 1, t:t + 1]),
                   f64(lse[0, 1, t:t + 1]), past=t)


# Enough rows for the workgroups of 128 and 256: each type and width on both sides of their borders.
MANY = [("bf16", 4, 16, 8, 515, 64, 0), ("bf16", 2, 64, 32, 2050, 64, 0), ("bf16", 3, 24, 12, 400, 32, 70), ("bf16", 2, 32, 16, 450, 128, 0),
        ("bf16", 8, 32, 16, 500, 128, 130), ("f32", 8, 24, 12, 333, 32, 0), ("f32", 8, 24, 12, 333, 64, 50), ("f32", 4, 24, 12, 300, 128, 0)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "_".join(map(str, c)))
def test_many_rows(prism, case):
    """A padded batch whose padding holds NaN: the first and the last sequence's first and last group."""
    import torch
    dt, B, H, G, T, D, window = case
    r = Rng(23, dt)
    q, k, v = r.heads(B, T, H, G, G, D=D)
    do = r.vec(B, H, T, D)
    lens = [T] + [int(n) for n in r.r.integers(1, T, B - 2)] + [T - 67]
    for b, n in enumerate(lens):
        for t in (q, k, v, do):
            t[b, :, n:] = float("nan")
    out = (torch.full((B, H, T, D), 7.0, dtype=torch_dtype(dt), device="cuda"), torch.full((B, H, T), 7.0, device="cuda"))
    o, lse = prism.attn_fwd(q, k, v, lens=i32(lens), window=window, out=out)
    grads = prism.attn_bwd(q, k, v, o, lse, do, lens=i32(lens), window=window)
    for b in (0, B - 1):
        n = lens[b]
        for g in (0, G - 1):
            at = slice(2 * g, 2 * g + 2)                               # H = 2 G
            check_prompt(dt, q[b:b + 1, at], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], o[b:b + 1, at], lse[b:b + 1, at], [(0, 0, n)],
                         D ** -0.5, window=window, do=do[b:b + 1, at],
                         grads={"dq": grads["dq"][b:b + 1, at], "dk": grads["dk"][b:b + 1, g:g + 1], "dv": grads["dv"][b:b + 1, g:g + 1]})
    for b, n in enumerate(lens):
        assert (o[b, :, n:] == 7).all() and (lse[b, :, n:] == 7).all()
        assert all((grads[x][b, :, n:] == 0).all() for x in grads) and all(torch.isfinite(t[b, :, :n]).all() for t in grads.values())
    again = prism.attn_fwd(q, k, v, lens=i32(lens), window=window)
    assert all(torch.equal(again[0][b, :, :n], o[b, :, :n]) for b, n in enumerate(lens))


@pytest.mark.parametrize("case", [MANY[0], MANY[2], MANY[4], MANY[6]], ids=lambda c: "_".join(map(str, c)))
def test_many_rows_that_do_not_see_a_key(prism, case):
    """Keys and values that are not finite reach the rows behind them and no others."""
    import torch
    dt, B, H, G, T, D, window = case
    r = Rng(24, dt)
    q, k, v = r.heads(B, T, H, G, G, D=D)
    at = 301
    k[0, 0, at] = float("nan")
    v[B - 1, G - 1, at] = float("inf")
    o, lse = prism.attn_fwd(q, k, v, window=window)
    last = min(T, at + window) if window else T
    for b, g in ((0, 0), (B - 1, G - 1)):
        h = slice(2 * g, 2 * g + 2)
        check_prompt(dt, q[b:b + 1, h, :at], k[b:b + 1, g:g + 1, :at], v[b:b + 1, g:g + 1, :at], o[b:b + 1, h, :at], lse[b:b + 1, h, :at],
                     [(0, 0, at)], D ** -0.5, window=window)
        assert not torch.isfinite(o[b, h, at:last]).any() and torch.isfinite(o[b, h, last:]).all()
    assert torch.isfinite(o[1, 1:]).all() and torch.isfinite(o[0, 2:]).all()


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_many_rows_packed(prism, dt, D):
    import torch
    r = Rng(25, dt)
    H, G, lens = 48, 24, (700, 0, 1, 33, 1200)
    starts = np.cumsum((11,) + lens)
    T = int(starts[-1]) + 45
    q, k, v = r.heads(1, T, H, G, G, D=D)
    do = r.vec(1, H, T, D)
    out = (torch.full((1, H, T, D), 7.0, dtype=torch_dtype(dt), device="cuda"), torch.full((1, H, T), 7.0, device="cuda"))
    o, lse = prism.attn_fwd(q, k, v, starts=i32(starts), out=out)
    grads = prism.attn_bwd(q, k, v, o, lse, do, starts=i32(starts))
    for g in (0, G - 1):
        at = slice(2 * g, 2 * g + 2)
        check_prompt(dt, q[:, at], k[:, g:g + 1], v[:, g:g + 1], o[:, at], lse[:, at], [(0, int(a), n) for a, n in zip(starts, lens)],
                     D ** -0.5, do=do[:, at], grads={"dq": grads["dq"][:, at], "dk": grads["dk"][:, g:g + 1], "dv": grads["dv"][:, g:g + 1]})
    for lo, hi in ((0, 11), (int(starts[-1]), T)):
        assert (o[:, :, lo:hi] == 7).all() and (lse[:, :, lo:hi] == 7).all() and all((t[:, :, lo:hi] == 0).all() for t in grads.values())


# ---- norm and rotation --------------------------------------------------------------------------
ROPE = [("bf16", 2, 3, 1, 5, 64, 64, True), ("bf16", 1, 4, 2, 7, 128, 32, True), ("f32", 1, 2, 1, 9, 96, 24, True), ("f32", 3, 1, 1, 1, 32, 8, False),
        ("bf16", 1, 5, 3, 33, 256, 256, True), ("f32", 1, 2, 2, 3, 512, 500, True), ("bf16", 1, 1, 1, 4, 10, 6, True), ("f32", 2, 3, 2, 2, 2, 2, True),
        ("f32", 1, 2, 1, 6, 130, 130, True), ("bf16", 2, 24, 8, 700, 64, 16, True), ("f32", 1, 3, 1, 4, 510, 2, False), ("bf16", 1, 2, 1, 5, 48, 44, False)]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(prism, case, interleaved):
    import torch
    dt, B, heads, G, T, D, rot, norm = case
    r = Rng(21, dt)
    q, k = r.heads(B, T, heads, G, D=D)
    dq, dk = r.heads(B, T, heads, G, D=D)
    freq = r.flt(rot // 2, lo=1e-4, hi=1.0)
    pos = i32(r.r.integers(0, 1 << 20, (B, T)))
    wq, wk = (r.flt(D, lo=-2, hi=2), r.flt(D, lo=-2, hi=2)) if norm else (None, None)
    kw = dict(pos=pos, wq=wq, wk=wk, eps=1e-3, interleaved=interleaved, factor=1.25)
    y = prism.rope_fwd(q, k, freq, **kw)
    g = prism.rope_bwd(q, k, dq, dk, freq, **kw)
    b = (D + 32) * U + 2.0 ** -22
    a = H if dt == "bf16" else 0.0
    ch = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))

    def size_of(h):                                            # |a| + |b| of a pair for both channels, times factor
        s = np.abs(h).copy()
        s[..., ch[0]] = s[..., ch[1]] = 1.25 * (np.abs(h[..., ch[0]]) + np.abs(h[..., ch[1]]))
        return s

    for n, x, yy, dy, gg, w in (("q", q, y[0], dq, g["dq"], wq), ("k", k, y[1], dk, g["dk"], wk)):
        w64 = None if w is None else f64(w)
        h = f64(x)
        hn = h if w is None else h / np.sqrt((h * h).mean(-1, keepdims=True) + float(np.float32(1e-3))) * w64
        args = (f64(pos), f64(freq), w64, float(np.float32(1e-3)), interleaved, 1.25)
        close(n, yy, A.rope(h, *args), size_of(hn), b, a)
        rx, rw = A.rope_grad(h, f64(dy), *args)
        up = size_of(f64(dy))
        if w is not None:
            rms = np.sqrt((h * h).mean(-1, keepdims=True) + float(np.float32(1e-3)))
            hat = np.abs(h) / rms
            size = (up * np.abs(w64) + hat * (up * np.abs(w64) * hat).mean(-1, keepdims=True)) / rms
            close("d" + n, gg, rx, size, 2 * b, a)
            close("dw" + n, g["dw" + n], rw, (up * hat).sum((0, 1, 2)), 2 * b + x[..., 0].numel() * U)
        else:
            close("d" + n, gg, rx, up, b, a)
            assert set(g) == {"dq", "dk"}
    assert y[0].stride() == q.stride() or y[0].is_contiguous() or y[0].transpose(1, 2).is_contiguous()
    y2 = prism.rope_fwd(q, k, freq, **kw, out=(q, k))           # in place
    assert y2[0] is q and torch.equal(q, y[0]) and torch.equal(k, y[1])
    g2 = prism.rope_bwd(q, k, dq, dk, freq, **{**kw, "wq": None, "wk": None}, out=(dq, dk))
    assert g2["dq"] is dq


def test_rope_positions(prism):
    """The token's index where no positions are given; the largest and negative positions."""
    import torch
    r = Rng(22, "f32")
    q, k, freq = r.vec(2, 2, 50, 64), r.vec(2, 1, 50, 64), r.flt(32, lo=1e-3, hi=1)
    own = prism.rope_fwd(q, k, freq)
    given = prism.rope_fwd(q, k, freq, pos=i32(np.tile(np.arange(50), (2, 1))))
    assert torch.equal(own[0], given[0]) and torch.equal(own[1], given[1])
    pos = r.r.integers(-2 ** 31, 2 ** 31 - 1, (2, 50))
    y = prism.rope_fwd(q, k, freq, pos=i32(pos))
    for x, yy in ((q, y[0]), (k, y[1])):
        h = f64(x)
        s = np.abs(h[..., :32]) + np.abs(h[..., 32:])
        # angles of up to 2^31: three roundings of 2^-53 in the kernel (1 / 2 pi, two products), one in the oracle's product:
        # 4 x 2^31 x 2^-53 = 2^-20, beside the 2^-21 of near ones
        close("far", yy, A.rope(h, pos, f64(freq)), np.concatenate([s, s], -1), 2.0 ** -20 + 2.0 ** -21)
    q[0, 0, 3] = float("nan")
    z = prism.rope_fwd(q, k, freq)
    assert torch.isnan(z[0][0, 0, 3]).all() and torch.equal(z[0][1], own[0][1]) and torch.equal(z[1], own[1])


# ---- paged cache --------------------------------------------------------------------------------
def pages_of(r, G, page, counts, D, dt, bits8=False, spare=3):
    """Caches full of rows nobody has written (NaN), and a table of distinct pages in a random order."""
    import torch
    each = max(counts)
    n = sum(counts) + spare
    ids = r.r.permutation(n)
    table, at = np.full((len(counts), each), -1), 0
    for s, c in enumerate(counts):
        table[s, :c] = ids[at:at + c]
        at += c
    if bits8:
        c = [torch.full((n, G, page, D), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        return c, [torch.full((n, G, page), float("nan"), device="cuda") for _ in range(2)], table
    return [torch.full((n, G, page, D), float("nan"), dtype=torch_dtype(dt), device="cuda") for _ in range(2)], None, table


def rows_of(cache, scales, table, n):
    """The first n rows of a sequence's pages, [G, n, D] float64."""
    page = cache.shape[2]
    ids = [int(i) for i in table[:-(-n // page)]]
    x = np.concatenate([f64(cache[i].float()) * (1.0 if scales is None else f64(scales[i])[..., None]) for i in ids], 1)
    return x[:, :n]


WRITE = [("bf16", 2, 20, 64, 16, False), ("f32", 1, 1, 32, 32, False), ("f32", 3, 70, 128, 64, False), ("bf16", 4, 45, 128, 16, True),
         ("bf16", 1, 130, 32, 64, True), ("bf16", 2, 1, 64, 1024, True)]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("packed", [False, True])
def test_cache_write(prism, case, packed):
    import torch
    dt, G, T, D, page, bits8 = case
    r = Rng(31, dt)
    past, lens = [0, 5, page - 1, 2 * page + 3], [T, max(T - 1, 0), T, 0]
    S = len(past)
    counts = [-(-(p + T) // page) for p in past]
    (ck, cv), sc, table = pages_of(r, G, page, counts, D, dt, bits8)
    table[2, counts[2] - 1] = 10 ** 6                          # a page outside the cache: its rows are not written
    before = [t.clone() for t in (ck, cv)]
    if packed:
        k, v = r.heads(1, S * T, G, G, D=D)
        starts = np.concatenate([[0], np.cumsum(lens)])
        at = [(0, int(a)) for a in starts]
        kw = dict(starts=i32(starts))
    else:
        k, v = r.heads(S, T, G, G, D=D)
        at, kw = [(s, 0) for s in range(S)], dict(lens=i32(lens))
    if T > 8:
        k[0, 0, 3] = 0
        v[0, 0, 4] = 1e-35
        k[0, 0, 5, 1] = float("inf")
    prism.cache_write(ck, cv, k, v, i32(table), i32(past), scales=sc, **kw)
    seen = torch.zeros(ck.shape[0], page, dtype=torch.bool)
    for s in range(S):
        for t in range(lens[s]):
            p = past[s] + t
            i = int(table[s, p // page])
            if not 0 <= i < ck.shape[0]:
                continue
            seen[i, p % page] = True
            b, first = at[s]
            for x, c, j in ((k, ck, 0), (v, cv, 1)):
                row, held = x[b, :, first + t], c[i, :, p % page]
                if not bits8:
                    assert torch.equal(row, held)
                    continue
                row, held, scale = f64(row), f64(held.float()), f64(sc[j][i, :, p % page])
                for g in range(G):
                    top = np.abs(row[g]).max()
                    if not np.isfinite(top):
                        assert np.isnan(held[g]).all() and not np.isfinite(scale[g])
                    elif top < 2.0 ** -100:
                        assert scale[g] == 1 and (held[g] == 0).all()
                    else:                                      # half a step of e4m3, and of its smallest values
                        assert abs(scale[g] - top / 448) <= 2.0 ** -22 * scale[g]
                        assert (np.abs(held[g] * scale[g] - row[g]) <= (2.0 ** -4 * np.abs(row[g]) + 2.0 ** -10 * scale[g]) * (1 + 2.0 ** -20)).all()
    for c, old in zip((ck, cv), before):                       # everything else stays
        keep = ~seen.cuda()
        c, old = c.view(torch.uint8), old.view(torch.uint8)
        assert torch.equal(c.transpose(1, 2)[keep], old.transpose(1, 2)[keep])


PAGED = [("bf16", 4, 1, 1, 64, 64, 0, False), ("bf16", 4, 2, 1, 128, 16, 0, False), ("f32", 2, 1, 1, 32, 32, 0, False), ("bf16", 8, 1, 5, 64, 64, 30, False),
         ("bf16", 6, 2, 33, 32, 16, 0, False), ("bf16", 2, 2, 65, 128, 64, 0, False), ("bf16", 4, 1, 130, 64, 128, 100, False),
         ("f32", 3, 1, 17, 128, 16, 0, False), ("f32", 2, 1, 140, 64, 64, 50, False), ("f32", 4, 2, 1, 128, 256, 0, False),
         ("bf16", 4, 1, 1, 128, 64, 0, True), ("bf16", 8, 2, 3, 64, 16, 9, True), ("bf16", 2, 1, 100, 32, 32, 0, True), ("bf16", 2, 1, 150, 128, 64, 0, True),
         ("bf16", 40, 1, 1, 32, 64, 1, True)]


@pytest.mark.parametrize("case", PAGED, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("room", [0, 3000])
def test_paged(prism, case, room):
    """room: positions that the table could hold beyond what is used (the key ranges are split by it)."""
    import torch
    dt, heads, G, T, D, page, window, bits8 = case
    r = Rng(41, dt)
    past = [0, 1, 31, 200, 700]
    lens = [T, T, max(T - 1, 1), T, 0]
    S = len(past)
    counts = [-(-(p + T) // page) for p in past]
    (ck, cv), sc, table = pages_of(r, G, page, counts, D, dt, bits8)
    table = np.concatenate([table, np.full((S, room // page), -1)], 1)
    n = max(p + t for p, t in zip(past, lens))
    k, v = r.heads(S, n, G, G, D=D)
    prism.cache_write(ck, cv, k, v, i32(table), i32([0] * S), lens=i32([p + t for p, t in zip(past, lens)]), scales=sc)
    q = r.heads(S, T, heads, 2, D=D)[0]
    out = torch.full((S, T, heads, D), 7.0, dtype=q.dtype, device="cuda").transpose(1, 2)
    o = prism.attn_paged(q, ck, cv, i32(table), i32(past), lens=i32(lens), scales=sc, window=window, out=out)
    assert o is out
    scale, rep = float(np.float32(1 / np.sqrt(D))), heads // G
    for s in range(S):
        assert bool((o[s, :, lens[s]:] == 7).all())
        if lens[s] == 0:
            continue
        m = past[s] + lens[s]
        kk, vv = rows_of(ck, sc and sc[0], table[s], m), rows_of(cv, sc and sc[1], table[s], m)
        for h in range(heads):
            check_head(f"[{s},{h}]", dt, f64(q[s, h, :lens[s]]), kk[h // rep], vv[h // rep], scale, f64(o[s, h, :lens[s]]), window=window,
                       past=past[s], extra=4 * U if bits8 else 0.0)


@pytest.mark.parametrize("T", [1, 100])
def test_paged_bad_tables(prism, T):
    """Pages outside the cache read as zeros, positions past the table are not there, nothing else is touched."""
    import torch
    G, D, page = 1, 64, 16
    r = Rng(42, "bf16")
    ck, cv = r.vec(4, G, page, D), r.vec(4, G, page, D)
    q = r.vec(2, 2, T, D)
    table, past = np.array([[0, -5, 2, 1 << 30], [3, 1, 0, 2]]), [40, 60]
    o = prism.attn_paged(q, ck, cv, i32(table), i32(past))
    for s in range(2):
        n = min(past[s] + T, 64)
        kk, vv = np.zeros((64, D)), np.zeros((64, D))
        for j, i in enumerate(table[s]):
            if 0 <= i < 4:
                kk[16 * j:16 * j + 16], vv[16 * j:16 * j + 16] = f64(ck[i, 0]), f64(cv[i, 0])
        for h in range(2):
            check_head(f"[{s},{h}]", "bf16", f64(q[s, h]), kk[:n], vv[:n], 0.125, f64(o[s, h]), past=past[s])
    o = prism.attn_paged(q, ck, cv, i32(table), i32([-9, 1 << 30]))         # negative, and past the table
    check_head("start", "bf16", f64(q[0, 0, :1]), f64(ck[0, 0, :1]), f64(cv[0, 0, :1]), 0.125, f64(o[0, 0, :1]))
    assert torch.isfinite(o).all()


def test_window_that_sees_nothing(prism):
    """Positions past the table with a window that ends behind it: rows of zeros."""
    r = Rng(43, "bf16")
    ck, cv, q = r.vec(2, 1, 16, 32), r.vec(2, 1, 16, 32), r.vec(1, 2, 40, 32)
    o = f64(prism.attn_paged(q, ck, cv, i32([[0, 1]]), i32([30]), window=4))
    for t in range(40):
        assert (o[0, :, t] == 0).all() == (30 + t - 4 + 1 >= 32), t


# ---- together -----------------------------------------------------------------------------------
@pytest.mark.parametrize("bits8", [False, True])
def test_prompt_chunks_and_tokens_agree(prism, bits8):
    """A layer's prompt in one call, and the same tokens through the cache: a chunk, another one, then token by token."""
    import torch
    heads, G, T, D, page, S = 4, 2, 90, 64, 16, 2
    r = Rng(51, "bf16")
    q, k, v = r.heads(S, T, heads, G, G, D=D)
    freq, w = r.flt(16, lo=0.01, hi=1), [r.flt(D, lo=0.5, hi=1.5) for _ in range(2)]
    counts = [-(-T // page)] * S
    (ck, cv), sc, table = pages_of(r, G, page, counts, D, "bf16", bits8)
    pos = np.tile(np.arange(T), (S, 1))
    qq, kk = prism.rope_fwd(q, k, freq, pos=i32(pos), wq=w[0], wk=w[1])
    whole, _ = prism.attn_fwd(qq, kk, v, window=50)
    steps = [(0, 40), (40, 80)] + [(t, t + 1) for t in range(80, T)]
    for lo, hi in steps:
        a, b = prism.rope_fwd(q[:, :, lo:hi], k[:, :, lo:hi], freq, pos=i32(pos[:, lo:hi]), wq=w[0], wk=w[1])
        assert torch.equal(a, qq[:, :, lo:hi]) and torch.equal(b, kk[:, :, lo:hi])
        prism.cache_write(ck, cv, b, v[:, :, lo:hi], i32(table), i32([lo] * S), scales=sc)
        o = prism.attn_paged(a, ck, cv, i32(table), i32([lo] * S), scales=sc, window=50)
        for s in range(S):
            kc, vc = rows_of(ck, sc and sc[0], table[s], hi), rows_of(cv, sc and sc[1], table[s], hi)
            for h in range(heads):
                check_head(f"{lo} [{s},{h}]", "bf16", f64(a[s, h]), kc[h // 2], vc[h // 2], 0.125, f64(o[s, h]), window=50, past=lo,
                           extra=4 * U if bits8 else 0.0)
                if not bits8:                                  # and with the prompt's own pass: a rounding of o on each side, one of p
                    size = A.attention(f64(a[s, h]), kc[h // 2], np.abs(vc[h // 2]), 0.125, window=50, past=lo)[0]
                    assert (np.abs(f64(o[s, h]) - f64(whole[s, h, lo:hi])) <= 4 * H * size).all()


def layer_calls(prism, dt="bf16", seed=61):
    """Calls of every operator on fixed inputs, each returning the tensors it wrote."""
    import torch
    r = Rng(seed, dt)
    heads, G, T, D, page, S = 4, 2, 130, 64, 16, 3
    q, k, v = r.heads(S, T, heads, G, G, D=D)
    do, freq, w = r.vec(S, heads, T, D), r.flt(32), [r.flt(D), r.flt(D)]
    lens, past = i32([130, 64, 7]), i32([0, 3, 100])
    (ck, cv), sc, table = pages_of(r, G, page, [20] * S, D, dt)
    for t in (ck, cv):
        t.zero_()
    t, tok = i32(table), r.vec(S, heads, 1, D)
    o, lse = prism.attn_fwd(q, k, v, lens=lens)
    need = max(prism.load_library().prism_attn_bwd_workspace_bytes(S, heads, G, T, D, 1 if dt == "bf16" else 0),
               prism.load_library().prism_attn_paged_workspace_bytes(S, heads, G, T, D, page, 20, 1 if dt == "bf16" else 0),
               prism.load_library().prism_attn_paged_workspace_bytes(S, heads, G, 1, D, page, 20, 1 if dt == "bf16" else 0), 1 << 22)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = dict(o=torch.zeros_like(o), lse=torch.zeros_like(lse), g=[torch.zeros_like(x) for x in (q, k, v)], y=[torch.zeros_like(q), torch.zeros_like(k)],
               c=torch.zeros_like(q), t=torch.zeros_like(tok))

    def run(**kw):
        a, b = prism.rope_fwd(q, k, freq, wq=w[0], wk=w[1], out=out["y"], **kw)
        prism.attn_fwd(a, b, v, lens=lens, out=(out["o"], out["lse"]), **kw)
        g = prism.attn_bwd(a, b, v, out["o"], out["lse"], do, lens=lens, out=out["g"], workspace=ws, **kw)
        d = prism.rope_bwd(q, k, g["dq"], g["dk"], freq, wq=w[0], wk=w[1], workspace=ws, **kw)
        prism.cache_write(ck, cv, b, v, t, past, lens=lens, **kw)
        prism.attn_paged(a, ck, cv, t, past, lens=lens, out=out["c"], workspace=ws, **kw)
        prism.attn_paged(tok, ck, cv, t, past, out=out["t"], workspace=ws, **kw)
        return [out["o"], out["lse"], *out["g"], *out["y"], d["dq"], d["dk"], d["dwq"], d["dwk"], ck, cv, out["c"], out["t"]]

    return run, (q, k, v, do, tok)


def test_graph_replays(prism):
    """One captured pass through every operator with a shared workspace, replayed on changing inputs between eager calls."""
    import torch
    run, inputs = layer_calls(prism)
    run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = run()
    r = Rng(62, "bf16")
    for _ in range(4):
        for x in inputs:
            x.copy_(r.vec(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_streams_and_repeats(prism):
    """The same bits again, and on a stream given by its handle."""
    import torch
    for dt in ("bf16", "f32"):
        run, _ = layer_calls(prism, dt)
        first = [x.clone() for x in run()]
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = run(stream=s.cuda_stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_refusals_of_the_binding(prism):
    import torch
    r = Rng(71, "bf16")
    q, k = r.vec(1, 4, 8, 64), r.vec(1, 2, 8, 64)
    c, t, p, f = r.vec(4, 2, 16, 64), i32([[0, 1]]), i32([0]), r.flt(32)
    bad = [lambda: prism.attn_fwd(q, k, k[:, :, :7]), lambda: prism.attn_fwd(q, k.float(), k), lambda: prism.attn_fwd(q, k[:, :1].expand(1, 3, 8, 64), k),
           lambda: prism.attn_fwd(q, k, k, lens=torch.tensor([3], device="cuda")), lambda: prism.attn_fwd(q, k, k, starts=i32([0])),
           lambda: prism.attn_fwd(q, k, k, causal=False, window=3), lambda: prism.attn_fwd(q, k, k, scale=-1.0),
           lambda: prism.attn_fwd(q.expand(2, 4, 8, 64), k.repeat(2, 1, 1, 1), k.repeat(2, 1, 1, 1)), lambda: prism.attn_fwd(q, k, k, out=q),
           lambda: prism.attn_bwd(q, k, k, q, None, q), lambda: prism.attn_bwd(q, k, k, q, q[..., 0].float(), q, workspace=torch.empty(8, device="cuda")),
           lambda: prism.rope_fwd(q, k, r.flt(33)), lambda: prism.rope_fwd(q, k, f, wq=r.flt(64)), lambda: prism.rope_fwd(q, k, f, pos=i32([1])),
           lambda: prism.rope_fwd(q.half(), k.half(), f), lambda: prism.cache_write(c, c[:3], k, k, t, p), lambda: prism.cache_write(c, c, k, k, t, None),
           lambda: prism.cache_write(c, c, k, k, t, p, scales=(f, f)), lambda: prism.attn_paged(q, c, c, t, i32([0, 1])),
           lambda: prism.attn_paged(q, c, c, t.long(), p), lambda: prism.attn_paged(q, c, c, t, p, out=q), lambda: prism.attn_paged(q, c.float(), c.float(), t, p)]
    for i, call in enumerate(bad):
        with pytest.raises(prism.PrismError):
            call()
            pytest.fail(f"call {i} was not refused")
