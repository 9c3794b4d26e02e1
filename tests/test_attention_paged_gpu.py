"""Chunks of new tokens over the paged cache with enough rows for the workgroups of 128 and 256: every type, width and page
size on either side of a tile of keys, against the float64 oracle (tolerances: test_attention_gpu)."""
import numpy as np
import pytest

from tests import test_attention_gpu as base
from tests.test_attention_gpu import U, Rng, check_head, f64, i32, pages_of, prism, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu

# type, heads, G, tokens, width, page, window, 8 bits: more than 256 rows of a group's heads; 256 tokens or more of 128 wide bfloat16 heads
# have workgroups of 256 rows
FORMS = [("bf16", 4, 2, 300, 128, 16, 0, False), ("bf16", 2, 2, 513, 128, 64, 100, False), ("bf16", 4, 2, 300, 128, 64, 0, True),
         ("bf16", 2, 1, 256, 128, 32, 70, True), ("bf16", 4, 2, 200, 128, 16, 0, False), ("bf16", 4, 1, 100, 128, 128, 30, False),
         ("bf16", 4, 2, 255, 128, 16, 40, True), ("bf16", 4, 2, 140, 64, 16, 0, False), ("bf16", 3, 1, 140, 64, 64, 65, False),
         ("bf16", 4, 2, 140, 64, 32, 0, True), ("bf16", 1, 1, 300, 64, 256, 128, True), ("bf16", 2, 1, 150, 32, 16, 0, False),
         ("bf16", 2, 1, 150, 32, 128, 33, False), ("bf16", 4, 2, 150, 32, 16, 20, True), ("bf16", 2, 1, 290, 32, 64, 0, True),
         ("f32", 4, 2, 140, 32, 16, 0, False), ("f32", 2, 1, 150, 32, 64, 50, False), ("f32", 4, 2, 140, 64, 16, 31, False),
         ("f32", 2, 1, 150, 64, 32, 0, False), ("f32", 4, 2, 140, 128, 16, 0, False), ("f32", 2, 1, 150, 128, 64, 90, False)]


def name(case):
    return "_".join(map(str, case))


@pytest.mark.parametrize("case", FORMS, ids=name)
@pytest.mark.parametrize("room", [0, 3000])
def test_chunks_of_many_rows(prism, case, room):  # noqa: F811
    base.test_paged(prism, case, room)


@pytest.mark.parametrize("case", FORMS, ids=name)
@pytest.mark.parametrize("room", [0, 3000])
def test_rows_that_do_not_see_a_row_of_the_cache(prism, case, room):  # noqa: F811
    """Keys and values that are not finite reach the tokens that see them and no others: behind them, in front of their window,
    in another page of the tile, and what nobody has written."""
    import torch
    dt, heads, G, T, D, page, window, bits8 = case
    r = Rng(82, dt)
    past, lens = [0, 37, 460], [T, T - 5, T]
    n = [p + t for p, t in zip(past, lens)]
    (ck, cv), sc, table = pages_of(r, G, page, [-(-(p + T) // page) for p in past], D, dt, bits8)
    table = np.concatenate([table, np.full((3, room // page), -1)], 1)
    k, v = r.heads(3, max(n), G, G, D=D)
    k[0, 0, 71, 5] = float("nan")
    v[0, G - 1, T - 9, 2] = float("inf")
    v[1, 0, 40] = -float("inf")
    k[1, G - 1, 90] = float("nan")
    v[2, 0, 470, 7] = float("nan")
    prism.cache_write(ck, cv, k, v, i32(table), i32([0] * 3), lens=i32(n), scales=sc)
    q = r.heads(3, T, heads, 2, D=D)[0]
    q[2, 0, 11] = float("nan")
    o = prism.attn_paged(q, ck, cv, i32(table), i32(past), lens=i32(lens), scales=sc, window=window)
    rep, scale, finite = heads // G, float(np.float32(1 / np.sqrt(D))), 0
    for s in range(3):
        kk, vv = rows_of(ck, sc and sc[0], table[s], n[s]), rows_of(cv, sc and sc[1], table[s], n[s])
        for h in range(heads):
            kh, vh, qh, oh = kk[h // rep], vv[h // rep], f64(q[s, h]), f64(o[s, h])
            bad_k, bad_v = ~np.isfinite(kh).all(1), ~np.isfinite(vh)
            rows = []
            for t in range(lens[s]):
                lo, hi = max(0, past[s] + t - window + 1) if window else 0, past[s] + t + 1
                if bad_k[lo:hi].any() or not np.isfinite(qh[t]).all():
                    assert np.isnan(oh[t]).all(), (s, h, t)
                elif bad_v[lo:hi].any():                               # their columns alone
                    assert (~np.isfinite(oh[t]) == bad_v[lo:hi].any(0)).all(), (s, h, t)
                else:
                    rows.append(t)
            finite += len(rows)
            # what they do not see is nothing to them
            kz, vz = np.where(bad_k[:, None], 0.0, kh), np.where(bad_v, 0.0, vh)
            runs = np.split(np.array(rows), np.flatnonzero(np.diff(rows) != 1) + 1) if rows else []
            for run in runs:
                check_head(f"[{s},{h}] from {run[0]}", dt, qh[run], kz, vz, scale, oh[run], window=window, past=past[s] + int(run[0]),
                           extra=4 * U if bits8 else 0.0)
    assert finite > 0 and torch.isfinite(o[2, heads - 1, :5]).all()


@pytest.mark.parametrize("bits8", [False, True])
def test_pages_beyond_32_bit_offsets(prism, bits8):  # noqa: F811
    """Pages on both sides of 2^32 values of a cache hold what they hold in a small one, and are read alike."""
    import torch
    G, page, D, n, pages = 8, 64, 128, 450, 70000                      # 2^16 values to a page
    r = Rng(84, "bf16")
    k, v = r.heads(1, n, G, G, D=D)
    ids = [pages - 1, 3, 65535, 65536, 40000, 32768, 16383, pages - 2]
    near, far = i32([list(range(8))]), i32([ids])

    def caches(count):
        c = [torch.empty(count, G, page, D, dtype=torch.float8_e4m3fn if bits8 else torch.bfloat16, device="cuda") for _ in range(2)]
        return c, [torch.empty(count, G, page, device="cuda") for _ in range(2)] if bits8 else None

    (a, sa), (b, sb) = caches(8), caches(pages)
    prism.cache_write(*a, k, v, near, i32([0]), scales=sa)
    prism.cache_write(*b, k, v, far, i32([0]), scales=sb)
    for x, y in zip(a + (sa or []), b + (sb or [])):
        x, y = (t.view(torch.uint8) if t.dtype.itemsize == 1 else t for t in (x, y))
        for i, j in enumerate(ids):
            rows = min(page, max(0, n - i * page))
            assert torch.equal(x[i, :, :rows], y[j, :, :rows])
    for T, heads in ((1, 16), (40, 8), (200, 16), (300, 8)):           # one tile of rows, several, workgroups of 128 and of 256
        q = r.vec(1, heads, T, D)
        got = [prism.attn_paged(q, *c, t, i32([n - T]), scales=s) for c, t, s in ((a, near, sa), (b, far, sb))]
        assert bool(torch.isfinite(got[0]).all()) and torch.equal(*got)
