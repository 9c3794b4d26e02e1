"""Argument checks of the attention layer's entry points.  Every call here fails on the host before anything is
enqueued, so no GPU is needed."""
import ctypes
import os

import pytest

import delta_rule_sequence_amd as prism
from delta_rule_sequence_amd.layer import _Strides

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
BIG = 1 << 40
P = 1 << 20          # aligned stand-ins for device pointers
Q = 1 << 21


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(prism.LIB_PATH):
        pytest.fail("libprism.so is not built (run __graft_entry__.build())")
    return prism.load_library()


def st(b, h, t):
    return ctypes.byref(_Strides(b, h, t))


def rope_fwd(lib, q=P, qs=None, k=P, ks=None, freq=P, pos=None, wq=None, wk=None, B=1, H=2, G=1, T=8, D=64, rot=64, factor=1.0,
             eps=1e-6, dt=1, yq=Q, ys=None, yk=Q):
    return lib.prism_rope_fwd(q, qs, k, ks, freq, pos, wq, wk, B, H, G, T, D, rot, 0, factor, eps, dt, yq, ys, yk, None, None)


def rope_bwd(lib, q=P, qs=None, k=P, dyq=P, dyk=P, freq=P, wq=P, wk=P, B=1, H=2, G=1, T=8, D=64, rot=64, factor=1.0, eps=1e-6, dt=1,
             dq=Q, dqs=None, dk=Q, dwq=P, dwk=P, ws=P, ws_bytes=BIG):
    return lib.prism_rope_bwd(q, qs, k, None, dyq, None, dyk, None, freq, None, wq, wk, B, H, G, T, D, rot, 0, factor, eps, dt, dq,
                              dqs, dk, None, dwq, dwk, ws, ws_bytes, None)


def attn_fwd(lib, q=P, qs=None, k=P, ks=None, v=P, lens=None, starts=None, S=0, B=1, H=2, G=1, T=8, D=64, scale=1.0, causal=1,
             window=0, dt=1, o=Q, os_=None):
    return lib.prism_attn_fwd(q, qs, k, ks, v, None, lens, starts, S, B, H, G, T, D, scale, causal, window, dt, o, os_, None, None)


def attn_bwd(lib, q=P, qs=None, k=P, ks=None, v=P, o=P, lse=P, do=P, lens=None, starts=None, S=0, B=1, H=2, G=1, T=8, D=64,
             scale=1.0, causal=1, window=0, dt=1, dq=Q, dqs=None, dk=Q, dv=Q, ws=P, ws_bytes=BIG):
    return lib.prism_attn_bwd(q, qs, k, ks, v, None, o, None, lse, do, None, lens, starts, S, B, H, G, T, D, scale, causal, window, dt,
                              dq, dqs, dk, None, dv, None, ws, ws_bytes, None)


def cache_write(lib, k=P, ks=None, v=P, table=P, past=P, lens=None, starts=None, S=0, B=1, G=1, T=8, D=64, pages=4, page=16,
                most=4, dt=1, ck=Q, cv=Q, sk=None, sv=None):
    return lib.prism_cache_write(k, ks, v, None, table, past, lens, starts, S, B, G, T, D, pages, page, most, dt, ck, cv, sk, sv, None)


def attn_paged(lib, q=P, qs=None, ck=P, cv=P, sk=None, sv=None, table=P, past=P, lens=None, B=1, H=2, G=1, T=1, D=64, pages=4,
               page=16, most=4, scale=1.0, window=0, dt=1, o=Q, os_=None, ws=P, ws_bytes=BIG):
    return lib.prism_attn_paged(q, qs, ck, cv, sk, sv, table, past, lens, B, H, G, T, D, pages, page, most, scale, window, dt, o, os_,
                                ws, ws_bytes, None)


ALL = [rope_fwd, rope_bwd, attn_fwd, attn_bwd, cache_write, attn_paged]


@pytest.mark.parametrize("call,names", [
    (rope_fwd, ["q", "k", "freq", "yq", "yk"]), (rope_bwd, ["q", "k", "dyq", "dyk", "freq", "dq", "dk"]),
    (attn_fwd, ["q", "k", "v", "o"]), (attn_bwd, ["q", "k", "v", "o", "lse", "do", "dq", "dk", "dv"]),
    (cache_write, ["k", "v", "table", "past", "ck", "cv"]), (attn_paged, ["q", "ck", "cv", "table", "past", "o"])])
def test_null_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == INVALID, n


@pytest.mark.parametrize("call", ALL)
def test_sizes(lib, call):
    for k in ("B", "G", "T", "D") + (() if call is cache_write else ("H",)):
        assert call(lib, **{k: 0}) == INVALID and call(lib, **{k: -1}) == INVALID, k
    assert call(lib, dt=2) == INVALID and call(lib, dt=-7) == INVALID
    assert call(lib, B=1 << 20, T=1 << 20) == UNSUPPORTED
    if call not in (rope_fwd, rope_bwd):
        for D in (16, 48, 96, 256):
            assert call(lib, D=D) == UNSUPPORTED, D
        assert call(lib, T=2 ** 31 - 1) == UNSUPPORTED


@pytest.mark.parametrize("call", [attn_fwd, attn_bwd, attn_paged])
def test_attention_arguments(lib, call):
    assert call(lib, H=3, G=2) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(lib, scale=scale) == INVALID, scale
    assert call(lib, window=-1) == INVALID


@pytest.mark.parametrize("call", [attn_fwd, attn_bwd])
def test_prompt_arguments(lib, call):
    assert call(lib, causal=0, window=4) == INVALID
    assert call(lib, starts=P, S=0) == INVALID and call(lib, starts=None, S=2) == INVALID
    assert call(lib, starts=P, S=2, B=2) == INVALID and call(lib, starts=P, S=2, lens=P) == INVALID
    assert call(lib, starts=P, S=2 ** 31 - 1) == UNSUPPORTED


@pytest.mark.parametrize("call", [attn_fwd, attn_bwd, attn_paged])
def test_strides(lib, call):
    assert call(lib, B=2, qs=st(0, 512, 64)) == INVALID                # a broadcast input
    assert call(lib, qs=st(1024, -512, 64)) == INVALID
    assert call(lib, T=8, qs=st(1024, 512, 68)) == UNSUPPORTED         # rows off the 16-byte boundary
    assert call(lib, T=8, qs=st(1024, 512, 1 << 25)) == UNSUPPORTED    # rows over 16 MB apart
    assert call(lib, T=8, qs=st(1024, 512, 32)) == UNSUPPORTED         # rows that overlap
    assert call(lib, q=P + 2) == UNSUPPORTED
    out = {"dqs" if call is attn_bwd else "os_": st(1024, 64, 64)}
    assert call(lib, T=8, **out) == INVALID                            # rows of the output overlap


def test_attention_outputs_over_inputs(lib):
    for name in ("dq", "dk", "dv"):
        assert attn_bwd(lib, **{name: P}) == INVALID, name
    assert attn_paged(lib, o=P) == INVALID
    assert attn_fwd(lib, k=Q) == INVALID and attn_fwd(lib, v=Q) == INVALID


def test_outputs_apart(lib):
    R, S = 1 << 22, 1 << 23
    assert attn_fwd(lib, o=P) == INVALID                               # a query's buffer: its rows may still be read
    assert attn_fwd(lib, q=Q) == INVALID
    for two in (("dq", "dk"), ("dq", "dv"), ("dk", "dv")):
        at = {"dq": Q, "dk": R, "dv": S}
        at[two[1]] = at[two[0]]
        assert attn_bwd(lib, **at) == INVALID, two
    # rotation: an output over its own input has its strides; never over the other one
    assert rope_fwd(lib, q=P, k=R, yq=Q, yk=Q) == INVALID
    assert rope_fwd(lib, q=P, k=R, yq=R, yk=Q) == INVALID and rope_fwd(lib, q=P, k=R, yq=Q, yk=P) == INVALID
    assert rope_fwd(lib, q=P, k=R, yq=P, ys=st(2048, 64, 128), yk=Q) == INVALID
    assert rope_bwd(lib, dyq=P, dyk=R, dq=P, dqs=st(2048, 64, 128), dk=Q) == INVALID
    assert rope_bwd(lib, dyq=P, dyk=R, dq=R, dk=Q) == INVALID and rope_bwd(lib, dyq=P, dyk=R, dq=Q, dk=Q) == INVALID
    assert rope_bwd(lib, q=S, k=P, dyq=R, dyk=R, dq=S, dk=Q) == INVALID
    assert cache_write(lib, ck=Q, cv=Q) == INVALID
    assert cache_write(lib, ck=Q, cv=R, sk=S, sv=S) == INVALID


def test_workspaces(lib):
    need = lib.prism_attn_bwd_workspace_bytes(1, 2, 1, 8, 64, 1)
    assert need > 0 and attn_bwd(lib, ws_bytes=need - 1) == WORKSPACE and attn_bwd(lib, ws=None) == WORKSPACE
    assert attn_bwd(lib, ws=P + 4) == INVALID
    need = lib.prism_rope_bwd_workspace_bytes(1, 2, 1, 8, 64, 64, 1)
    assert need > 0 and rope_bwd(lib, ws_bytes=need - 1) == WORKSPACE and rope_bwd(lib, ws=None) == WORKSPACE
    assert rope_bwd(lib, ws=P + 4) == INVALID
    need = lib.prism_attn_paged_workspace_bytes(1, 2, 1, 1, 64, 64, 1000, 1)
    assert need > 256 and attn_paged(lib, page=64, most=1000, ws_bytes=need - 1) == WORKSPACE
    assert attn_paged(lib, ws=None) == WORKSPACE and attn_paged(lib, ws=P + 4) == INVALID
    assert lib.prism_attn_bwd_workspace_bytes(1, 3, 2, 8, 64, 1) == 0 and lib.prism_attn_bwd_workspace_bytes(1, 2, 1, 8, 65, 1) == 0
    assert lib.prism_rope_bwd_workspace_bytes(1, 2, 1, 8, 63, 62, 1) == 0
    assert lib.prism_attn_paged_workspace_bytes(1, 2, 1, 1, 64, 48, 1, 1) == 0


@pytest.mark.parametrize("call", [rope_fwd, rope_bwd])
def test_rope_arguments(lib, call):
    assert call(lib, rot=0) == INVALID and call(lib, rot=66) == INVALID
    assert call(lib, rot=31) == UNSUPPORTED and call(lib, D=63, rot=62) == UNSUPPORTED and call(lib, D=514, rot=64) == UNSUPPORTED
    assert call(lib, eps=-1.0) == INVALID and call(lib, eps=float("nan")) == INVALID
    assert call(lib, factor=float("inf")) == INVALID
    assert call(lib, wq=P, wk=None) == INVALID and call(lib, wq=None, wk=P) == INVALID
    assert call(lib, B=2, qs=st(0, 512, 64)) == INVALID
    assert call(lib, **{"ys" if call is rope_fwd else "dqs": st(1024, 64, 64)}) == INVALID
    assert call(lib, H=65536) == UNSUPPORTED
    if call is rope_bwd:
        assert call(lib, wq=None, wk=None) == INVALID                  # gradients of weights that are not there


@pytest.mark.parametrize("call", [cache_write, attn_paged])
def test_cache_arguments(lib, call):
    for k in ("pages", "page", "most"):
        assert call(lib, **{k: 0}) == INVALID and call(lib, **{k: -1}) == INVALID, k
    for page in (8, 24, 2048):
        assert call(lib, page=page) == UNSUPPORTED, page
    assert call(lib, sk=P) == INVALID and call(lib, sv=P) == INVALID
    assert call(lib, sk=P, sv=P, dt=0) == UNSUPPORTED                  # 8 bits beside float32 rows
    assert call(lib, ck=P + 8) == UNSUPPORTED and call(lib, cv=P + 8) == UNSUPPORTED
    assert call(lib, page=1024, most=1 << 21) == UNSUPPORTED           # positions past 2^31
    if call is cache_write:
        assert call(lib, starts=P, S=0) == INVALID and call(lib, starts=P, S=2, B=2) == INVALID


def test_binding_refusals():
    import torch
    x, c, i, f = torch.zeros(1, 1, 4, 64), torch.zeros(2, 1, 16, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(32)
    for call in (lambda: prism.rope_fwd(x, x, f), lambda: prism.rope_bwd(x, x, x, x, f), lambda: prism.attn_fwd(x, x, x),
                 lambda: prism.attn_bwd(x, x, x, x, x[..., 0], x), lambda: prism.cache_write(c, c, x, x, i, i[:, 0]),
                 lambda: prism.attn_paged(x, c, c, i, i[:, 0]), lambda: prism.attn_fwd(None, x, x), lambda: prism.rope_fwd(None, x, f)):
        with pytest.raises(prism.PrismError):
            call()
