"""The attention layer at 2^23 tiles of 32 tokens times heads, the most that its calls take: their launches have to hold
less than 2^32 threads."""
import pytest

from tests.test_attention_gpu import prism  # noqa: F401

pytestmark = pytest.mark.gpu


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
