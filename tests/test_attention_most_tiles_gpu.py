"""The attention layer at 2^23 tiles of 32 tokens times heads, the most that its calls take: their launches have to hold
less than 2^32 threads."""
import pytest

from tests.test_attention_gpu import H, U, prism  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(128, 1), (64, 8), (32, 8)])
def test_prompts(prism, D, G):  # noqa: F811
    """2^20 sequences of one token and 8 heads: p is 1, so o is v and dv the sum of a group's do; dq and dk are what is left of
    two equal sums of D products, each off by D u of their absolute values."""
    import torch
    B, heads = 1 << 20, 8
    torch.manual_seed(91)
    q, do = (torch.randn(B, heads, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.randn(B, G, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o, lse = prism.attn_fwd(q, k, v)
    for lo in range(0, B, B // 8):                             # batch by batch of them: memory
        at, rep = slice(lo, lo + B // 8), heads // G
        each = lambda t: t[at, :, 0].float().repeat_interleave(rep, 1)
        assert torch.equal(o[at, :, 0], v[at, :, 0].repeat_interleave(rep, 1))
        x, y = q[at, :, 0].float(), each(k)
        size = (x.abs() * y.abs()).sum(-1) * D ** -0.5
        assert bool(((lse[at, :, 0] - (x * y).sum(-1) * D ** -0.5).abs() <= 2 * (D + 8) * U * size + 16 * U).all())
    g = prism.attn_bwd(q, k, v, o, lse, do)
    for lo in range(0, B, B // 8):
        at = slice(lo, lo + B // 8)
        d, y, x, w = do[at, :, 0].float(), each(k), q[at, :, 0].float(), each(v)
        left = 2.02 * D * U * (d.abs() * w.abs()).sum(-1, keepdim=True) * D ** -0.5 * (1 + H)
        assert bool((g["dq"][at, :, 0].float().abs() <= left * y.abs() * (1 + H) + 1e-30).all())
        group = lambda t: t.view(B // 8, G, rep, D).sum(2)
        assert bool((g["dk"][at, :, 0].float().abs() <= group(left * x.abs()) * (1 + H) + 1e-30).all())
        ref, most = group(d), group(d.abs())
        assert bool(((g["dv"][at, :, 0].float() - ref).abs() <= H * ref.abs() + 2 * rep * U * most).all())


def test_cache_write(prism):  # noqa: F811
    """2^23 sequences of 32 tokens, two tiles of the write each, whose rows overlap in memory; four of them have pages."""
    import torch
    B, T, D, page = 1 << 23, 32, 32, 16
    k, v = (torch.randn(8 * B + T * D, device="cuda").to(torch.bfloat16).as_strided((B, 1, T, D), (8, T * D, D, 1)) for _ in range(2))
    ck, cv = (torch.full((9, 1, page, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    written = [0, 12345, (1 << 22) + 3, B - 1]
    for i, s in enumerate(written):
        table[s] = torch.tensor([2 * i, 2 * i + 1])
    prism.cache_write(ck, cv, k, v, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    for x, c in ((k, ck), (v, cv)):
        for i, s in enumerate(written):
            assert torch.equal(c[2 * i:2 * i + 2, 0].reshape(T, D), x[s, 0]), s
        assert bool((c[8] == 7).all())
