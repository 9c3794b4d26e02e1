"""The attention layer: norm and rotation of queries and keys, softmax attention of prompts with its gradients, the
paged cache and the attention of new tokens over it.

Argument marshalling only, as the rest of the binding; the operators are described in include/prism.h.  Tensors, views,
streams and devices as in the state space layer's calls (layer.py).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import PrismError
from .layer import _F32, _I32, _Strides, _dense, _dtype, _gpu, _like, _need, _on_stream, _run, _scratch, _sizes, _strides, _tensor


def declare(lib) -> None:
    """Argument types of the layer's functions."""
    p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    st = ctypes.POINTER(_Strides)
    prompt = [p, st, p, st, p, st]                              # q, k, v with strides
    turn = [p, p, p, p] + [i] * 7 + [f, f, i]                   # freq, pos, wq, wk; B, H, G, T, D, rot, interleaved; factor, eps, dt
    sigs = {
        "prism_rope_fwd": [p, st, p, st] + turn + [p, st, p, st, p],
        "prism_rope_bwd": [p, st, p, st, p, st, p, st] + turn + [p, st, p, st, p, p, p, sz, p],
        "prism_cache_write": [p, st, p, st, p, p, p, p, i] + [i] * 8 + [p, p, p, p, p],
        "prism_attn_paged": [p, st, p, p, p, p, p, p, p] + [i] * 8 + [f, i, i, p, st, p, sz, p],
        "prism_attn_fwd": prompt + [p, p, i] + [i] * 5 + [f, i, i, i, p, st, p, p],
        "prism_attn_bwd": prompt + [p, st, p, p, st, p, p, i] + [i] * 5 + [f, i, i, i, p, st, p, st, p, st, p, sz, p],
    }
    for name, args in sigs.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    for name, n in (("prism_rope_bwd", 7), ("prism_attn_bwd", 6), ("prism_attn_paged", 8)):
        fn = getattr(lib, name + "_workspace_bytes")
        fn.argtypes, fn.restype = [i] * n, sz


# ---- norm and rotation -------------------------------------------------------------------------
def _turned(q, k, freq, pos, wq, wk, factor, eps, interleaved):
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise PrismError("q must have 4 axes")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise PrismError("k must be a tensor [B, G, T, D]")
    B, H, T, D = q.shape
    G = k.shape[1]
    _sizes(B, H, G, T, D)
    _tensor("q", q, q.shape, q.dtype, dev)
    _tensor("k", k, (B, G, T, D), q.dtype, dev)
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise PrismError("freq must be a tensor [rot / 2]")
    if (wq is None) != (wk is None):
        raise PrismError("wq and wk are given together")
    n = freq.shape[0]
    if 2 * n > D:
        raise PrismError(f"freq holds {n} values, the heads {D // 2} pairs")
    return dev, (B, H, T, D), (B, G, T, D), (
        _dense("freq", freq, (n,), _F32, dev), _dense("pos", pos, (B, T), _I32, dev), _dense("wq", wq, (D,), _F32, dev),
        _dense("wk", wk, (D,), _F32, dev), B, H, G, T, D, 2 * n, bool(interleaved), factor, eps, _dtype(q))


def _pair(out, names, likes, shapes, dtype, dev):
    """Two outputs: new ones, or the caller's after checking them."""
    if out is None:
        return _like(likes[0]), _like(likes[1])
    if not isinstance(out, (tuple, list)) or len(out) != 2:
        raise PrismError(f"out must be two tensors ({', '.join(names)})")
    return tuple(_tensor(n, t, s, dtype, dev) for n, t, s in zip(names, out, shapes))


@_on_stream
def rope_fwd(q, k, freq, pos=None, wq=None, wk=None, eps=1e-6, interleaved=False, factor=1.0, out=None):
    """q', k' = rope_fwd(q, k, freq): rotation of q [B,H,T,D] and k [B,G,T,D] by the angles pos freq[i], i < rot / 2 =
    len(freq): pairs of channels (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved; channels from rot on stay.  pos [B,T]
    int32: positions (the token's index if not given); freq float32; factor: on the rotated channels.  With wq, wk [D]
    float32 each head's row is first normalised: w x / sqrt(mean x^2 + eps).  out: two tensors, q and k among them."""
    dev, sq, sk, args = _turned(q, k, freq, pos, wq, wk, factor, eps, interleaved)
    yq, yk = _pair(out, ("q", "k"), (q, k), (sq, sk), q.dtype, dev)
    _run("prism_rope_fwd", dev, q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), *args, yq.data_ptr(), _strides(yq),
         yk.data_ptr(), _strides(yk))
    return yq, yk


@_on_stream
def rope_bwd(q, k, dq, dk, freq, pos=None, wq=None, wk=None, eps=1e-6, interleaved=False, factor=1.0, out=None, workspace=None):
    """Gradients of <dq, q'> + <dk, k'> for rope_fwd with the same arguments: a dict of dq, dk (the dtype of q; out: two
    tensors, the given dq and dk among them) and, with weights, dwq, dwk (float32)."""
    dev, sq, sk, args = _turned(q, k, freq, pos, wq, wk, factor, eps, interleaved)
    _tensor("dq", dq, sq, q.dtype, dev)
    _tensor("dk", dk, sk, q.dtype, dev)
    gq, gk = _pair(out, ("dq", "dk"), (q, k), (sq, sk), q.dtype, dev)
    g, ws = {"dq": gq, "dk": gk}, None
    if wq is not None:
        g["dwq"], g["dwk"] = torch.empty_like(wq), torch.empty_like(wk)
        ws = _scratch(workspace, _need("prism_rope_bwd", *args[4:10], args[-1]), dev)
    _run("prism_rope_bwd", dev, q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), dq.data_ptr(), _strides(dq), dk.data_ptr(),
         _strides(dk), *args, gq.data_ptr(), _strides(gq), gk.data_ptr(), _strides(gk), None if ws is None else g["dwq"].data_ptr(),
         None if ws is None else g["dwk"].data_ptr(), None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return g


# ---- prompts -----------------------------------------------------------------------------------
def _count(starts):
    """Sequences of a packed batch (0: not packed)."""
    if starts is None:
        return 0
    if not isinstance(starts, torch.Tensor) or starts.dim() != 1 or starts.shape[0] < 2:
        raise PrismError("starts must be a tensor [S + 1]")
    _sizes(starts.shape[0])
    return starts.shape[0] - 1


def _prompt(q, k, v, lens, starts, scale, causal, window):
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise PrismError("q must have 4 axes")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise PrismError("k must be a tensor [B, G, T, D]")
    B, H, T, D = q.shape
    G = k.shape[1]
    _sizes(B, H, G, T, D)
    _tensor("q", q, q.shape, q.dtype, dev)
    _tensor("k", k, (B, G, T, D), q.dtype, dev)
    _tensor("v", v, (B, G, T, D), q.dtype, dev)
    S = _count(starts)
    p_lens, p_starts = _dense("lens", lens, (B,), _I32, dev), _dense("starts", starts, (S + 1,), _I32, dev)
    scale = 1 / math.sqrt(D) if scale is None and D else scale
    return dev, B, H, G, T, D, (p_lens, p_starts, S, B, H, G, T, D, scale, bool(causal), window, _dtype(q))


@_on_stream
def attn_fwd(q, k, v, scale=None, causal=True, window=0, lens=None, starts=None, out=None):
    """o, lse = attn_fwd(q, k, v): softmax attention of q [B,H,T,D] over k, v [B,G,T,D], each group of H / G heads sharing
    a key head; o [B,H,T,D] in q's dtype, lse [B,H,T] float32.  scale: 1 / sqrt(D) if not given.  causal: token i
    sees tokens up to i; window: the last `window` of them only (0: all).  lens [B] int32: tokens of each sequence; or
    starts [S + 1] int32 with B = 1: sequence s is tokens starts[s] .. starts[s + 1] - 1.  Rows of no sequence keep what
    out = (o, lse) holds (new tensors hold nothing defined there)."""
    dev, B, H, G, T, D, args = _prompt(q, k, v, lens, starts, scale, causal, window)
    if out is None:
        o, lse = _like(q), torch.empty((B, H, T), dtype=_F32, device=dev)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 2:
            raise PrismError("out must be two tensors (o, lse)")
        o, lse = _tensor("o", out[0], (B, H, T, D), q.dtype, dev), out[1]
    _run("prism_attn_fwd", dev, q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), *args,
         o.data_ptr(), _strides(o), _dense("lse", lse, (B, H, T), _F32, dev))
    return o, lse


def _zeros_like(t):
    return _like(t).zero_()


@_on_stream
def attn_bwd(q, k, v, o, lse, do, scale=None, causal=True, window=0, lens=None, starts=None, out=None, workspace=None):
    """Gradients of <do, o> for attn_fwd with the same arguments, from its o and lse: a dict of dq, dk, dv in q's dtype
    (out: three tensors to write them to).  Rows of no sequence keep what `out` holds (new gradients: zero)."""
    dev, B, H, G, T, D, args = _prompt(q, k, v, lens, starts, scale, causal, window)
    _tensor("o", o, (B, H, T, D), q.dtype, dev)
    _tensor("do", do, (B, H, T, D), q.dtype, dev)
    if lse is None:
        raise PrismError("lse is required")
    if out is None:
        new = _like if lens is None and starts is None else _zeros_like
        dq, dk, dv = new(q), new(k), new(v)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 3:
            raise PrismError("out must be three tensors (dq, dk, dv)")
        dq, dk, dv = (_tensor(n, t, s.shape, q.dtype, dev) for n, t, s in zip(("dq", "dk", "dv"), out, (q, k, v)))
    ws = _scratch(workspace, _need("prism_attn_bwd", B, H, G, T, D, args[-1]), dev)
    _run("prism_attn_bwd", dev, q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), o.data_ptr(),
         _strides(o), _dense("lse", lse, (B, H, T), _F32, dev), do.data_ptr(), _strides(do), *args, dq.data_ptr(), _strides(dq),
         dk.data_ptr(), _strides(dk), dv.data_ptr(), _strides(dv), ws.data_ptr(), ws.numel())
    return {"dq": dq, "dk": dk, "dv": dv}


# ---- paged cache -------------------------------------------------------------------------------
def _cache(cache_k, cache_v, scales, table, past, S, G, D, dtype, dev):
    """The cache's arguments after checking them: pointers of the caches, of their scales, of table and past; pages, page, max_pages."""
    if not isinstance(cache_k, torch.Tensor) or cache_k.dim() != 4:
        raise PrismError("the caches must be tensors [pages, G, page, D]")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise PrismError("table must be a tensor [sequences, pages of a sequence]")
    if table.shape[0] != S:
        raise PrismError(f"table has {table.shape[0]} rows for {S} sequences")
    pages, page, most = cache_k.shape[0], cache_k.shape[2], table.shape[1]
    _sizes(pages, page, most)
    held = dtype if scales is None else torch.float8_e4m3fn
    ptrs = [_dense(n, t, (pages, G, page, D), held, dev) for n, t in (("cache_k", cache_k), ("cache_v", cache_v))]
    if scales is None:
        ptrs += [None, None]
    else:
        if not isinstance(scales, (tuple, list)) or len(scales) != 2:
            raise PrismError("scales must be two tensors (of the keys, of the values)")
        ptrs += [_dense(n, t, (pages, G, page), _F32, dev) for n, t in zip(("scales of the keys", "scales of the values"), scales)]
    ptrs += [_dense("table", table, (S, most), _I32, dev), _dense("past", past, (S,), _I32, dev)]
    if None in ptrs[:2] + ptrs[4:] or (scales is not None and None in ptrs):
        raise PrismError("caches, scales, table and past are required")
    return ptrs, pages, page, most


@_on_stream
def cache_write(cache_k, cache_v, k, v, table, past, lens=None, starts=None, scales=None):
    """Writes k, v [B,G,T,D] to the paged caches [pages,G,page,D]: token t of sequence s at position past[s] + t, which
    lies in page table[s, position // page].  table [S, pages of a sequence], past [S]: int32.  lens [B] int32: tokens of each
    sequence; or starts [S + 1] int32 with B = 1 (else S = B).  scales: two float32 tensors [pages,G,page] for
    float8_e4m3fn caches (the value is byte value * scale), whose rows are written too."""
    dev = _gpu(k, "k")
    if k.dim() != 4:
        raise PrismError("k must have 4 axes")
    B, G, T, D = k.shape
    _sizes(B, G, T, D)
    _tensor("k", k, k.shape, k.dtype, dev)
    _tensor("v", v, (B, G, T, D), k.dtype, dev)
    S = _count(starts)
    p_lens, p_starts = _dense("lens", lens, (B,), _I32, dev), _dense("starts", starts, (S + 1,), _I32, dev)
    (ck, cv, sk, sv, pt, pp), pages, page, most = _cache(cache_k, cache_v, scales, table, past, S or B, G, D, k.dtype, dev)
    _run("prism_cache_write", dev, k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), pt, pp, p_lens, p_starts, S, B, G, T, D,
         pages, page, most, _dtype(k), ck, cv, sk, sv)


@_on_stream
def attn_paged(q, cache_k, cache_v, table, past, lens=None, scales=None, scale=None, window=0, out=None, workspace=None):
    """o = attn_paged(q, cache_k, cache_v, table, past): softmax attention of new tokens q [B,H,T,D] over the paged
    caches [pages,G,page,D] (cache_write), which hold the tokens' own keys and values already: token t of sequence b has
    position past[b] + t and sees the positions up to its own (window: the last `window` of them only).  lens [B] int32: new
    tokens of each sequence; rows past them keep what `out` holds.  scale: 1 / sqrt(D) if not given."""
    dev = _gpu(q, "q")
    if q.dim() != 4:
        raise PrismError("q must have 4 axes")
    if not isinstance(cache_k, torch.Tensor) or cache_k.dim() != 4:
        raise PrismError("the caches must be tensors [pages, G, page, D]")
    B, H, T, D = q.shape
    G = cache_k.shape[1]
    _sizes(B, H, G, T, D)
    _tensor("q", q, q.shape, q.dtype, dev)
    (ck, cv, sk, sv, pt, pp), pages, page, most = _cache(cache_k, cache_v, scales, table, past, B, G, D, q.dtype, dev)
    o = _like(q) if out is None else _tensor("out", out, (B, H, T, D), q.dtype, dev)
    code = _dtype(q)
    ws = _scratch(workspace, _need("prism_attn_paged", B, H, G, T, D, page, most, code), dev)
    _run("prism_attn_paged", dev, q.data_ptr(), _strides(q), ck, cv, sk, sv, pt, pp, _dense("lens", lens, (B,), _I32, dev), B, H, G, T,
         D, pages, page, most, 1 / math.sqrt(D) if scale is None and D else scale, window, code, o.data_ptr(), _strides(o),
         ws.data_ptr(), ws.numel())
    return o
