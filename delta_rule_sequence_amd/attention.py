"""The attention layer: norm and rotation of queries and keys, softmax attention of prompts with its gradients, the
paged cache and the attention of new tokens over it.

Argument marshalling only, as the rest of the binding; the operators are described in include/prism.h.  Tensors, views,
streams and devices as in the state space layer's calls (layer.py).
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import PrismError
from .layer import _DTYPES, _F32, _I32, _Strides, _dense, _gpu, _need, _on_stream, _run, _scratch, _sizes, _stride_arg


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


# ---- shapes ------------------------------------------------------------------------------------
# What a call's shapes, strides and dtypes decide is checked and prepared once for each combination of them (half of the
# binding's time for a small call).
def _meta(name, t):
    if not isinstance(t, torch.Tensor):
        raise PrismError(f"{name} is required")
    return t.shape, t.stride(), t.dtype


def _same_device(dev, *tensors):
    index = dev.index
    for t in tensors:
        if t.get_device() != index:
            raise PrismError(f"all tensors must be on {dev}")


def _rows(name, meta, shape, dtype):
    """The strides argument of a tensor [B, heads, T, D] after checking it (None: dense)."""
    got, stride, kind = meta
    if got != shape:
        raise PrismError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
    if kind is not dtype:
        raise PrismError(f"{name} must have dtype {dtype}")
    B, H, T, D = shape
    if stride[3] != 1 and D > 1:
        raise PrismError(f"{name} must have a unit stride in its last axis")
    if all(n == 1 or s == d for n, s, d in zip((B, H, T), stride, (H * T * D, T * D, D))):
        return None
    return _stride_arg(*stride[:3])


def _new_stride(meta):
    """Strides of a new dense tensor, heads or tokens outermost as in the one of this kind."""
    (B, H, T, D), stride, _ = meta
    return (T * H * D, D, H * D, 1) if H > 1 and stride[1] < stride[2] else (H * T * D, T * D, D, 1)


def _new_rows(stride, shape):
    """The strides argument of a new tensor."""
    B, H, T, D = shape
    return None if stride[2] == D or T == 1 and stride[1] == D else _stride_arg(*stride[:3])


def _code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise PrismError(f"unsupported dtype {dtype}: bfloat16 or float32")
    return code


def _axes(name, meta, what):
    if len(meta[0]) != 4:
        raise PrismError(f"{name} must be a tensor {what}")
    return meta[0]


def _given(out, names):
    if not isinstance(out, (tuple, list)) or len(out) != len(names):
        raise PrismError(f"out must be {len(names)} tensors ({', '.join(names)})")
    return out


_ints = ctypes.c_int


# ---- norm and rotation -------------------------------------------------------------------------
@functools.lru_cache(maxsize=4096)
def _turned(mq, mk, n, interleaved, factor, eps):
    B, H, T, D = sq = _axes("q", mq, "[B, H, T, D]")
    G = _axes("k", mk, "[B, G, T, D]")[1]
    _sizes(B, H, G, T, D)
    sk, dtype = (B, G, T, D), mq[2]
    if 2 * n > D:
        raise PrismError(f"freq holds {n} values, the heads {D // 2} pairs")
    sizes = (B, H, G, T, D, 2 * n)
    tail = tuple(map(_ints, (*sizes, interleaved))) + (ctypes.c_float(factor), ctypes.c_float(eps), _ints(_code(dtype)))
    new = _new_stride(mq), _new_stride(mk)
    return (sq, sk, dtype, _rows("q", mq, sq, dtype), _rows("k", mk, sk, dtype), tail, (*sizes, _code(dtype)), new,
            _new_rows(new[0], sq), _new_rows(new[1], sk))


def _vectors(dev, freq, pos, wq, wk, B, T, D):
    if (wq is None) != (wk is None):
        raise PrismError("wq and wk are given together")
    return (_dense("freq", freq, (freq.shape[0],), _F32, dev), _dense("pos", pos, (B, T), _I32, dev),
            _dense("wq", wq, (D,), _F32, dev), _dense("wk", wk, (D,), _F32, dev))


def _frequencies(freq):
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise PrismError("freq must be a tensor [rot / 2]")
    return freq.shape[0]


def _pair(out, names, plan, dev):
    """Two outputs and their strides arguments: new ones, or the caller's after checking them."""
    sq, sk, dtype = plan[:3]
    if out is None:
        yq = torch.empty_strided(sq, plan[7][0], dtype=dtype, device=dev)
        return yq, plan[8], torch.empty_strided(sk, plan[7][1], dtype=dtype, device=dev), plan[9]
    yq, yk = _given(out, names)
    st = _rows(names[0], _meta(names[0], yq), sq, dtype), _rows(names[1], _meta(names[1], yk), sk, dtype)
    _same_device(dev, yq, yk)
    return yq, st[0], yk, st[1]


@_on_stream
def rope_fwd(q, k, freq, pos=None, wq=None, wk=None, eps=1e-6, interleaved=False, factor=1.0, out=None):
    """q', k' = rope_fwd(q, k, freq): rotation of q [B,H,T,D] and k [B,G,T,D] by the angles pos freq[i], i < rot / 2 =
    len(freq): pairs of channels (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved; channels from rot on stay.  pos [B,T]
    int32: positions (the token's index if not given); freq float32; factor: on the rotated channels.  With wq, wk [D]
    float32 each head's row is first normalised: w x / sqrt(mean x^2 + eps).  out: two tensors, q and k among them."""
    dev = _gpu(q, "q")
    plan = _turned(_meta("q", q), _meta("k", k), _frequencies(freq), bool(interleaved), float(factor), float(eps))
    _same_device(dev, k)
    B, _, T, D = plan[0]
    yq, tq, yk, tk = _pair(out, ("q", "k"), plan, dev)
    _run("prism_rope_fwd", dev, q.data_ptr(), plan[3], k.data_ptr(), plan[4], *_vectors(dev, freq, pos, wq, wk, B, T, D), *plan[5],
         yq.data_ptr(), tq, yk.data_ptr(), tk)
    return yq, yk


@_on_stream
def rope_bwd(q, k, dq, dk, freq, pos=None, wq=None, wk=None, eps=1e-6, interleaved=False, factor=1.0, out=None, workspace=None):
    """Gradients of <dq, q'> + <dk, k'> for rope_fwd with the same arguments: a dict of dq, dk (the dtype of q; out: two
    tensors, the given dq and dk among them) and, with weights, dwq, dwk (float32)."""
    dev = _gpu(q, "q")
    plan = _turned(_meta("q", q), _meta("k", k), _frequencies(freq), bool(interleaved), float(factor), float(eps))
    sq, sk, dtype = plan[:3]
    st = _rows("dq", _meta("dq", dq), sq, dtype), _rows("dk", _meta("dk", dk), sk, dtype)
    _same_device(dev, k, dq, dk)
    vectors = _vectors(dev, freq, pos, wq, wk, sq[0], sq[2], sq[3])
    gq, tq, gk, tk = _pair(out, ("dq", "dk"), plan, dev)
    g, sums = {"dq": gq, "dk": gk}, (None, None, None, 0)
    if wq is not None:
        g["dwq"], g["dwk"] = torch.empty_like(wq), torch.empty_like(wk)
        ws = _scratch(workspace, _need("prism_rope_bwd", *plan[6]), dev)
        sums = g["dwq"].data_ptr(), g["dwk"].data_ptr(), ws.data_ptr(), ws.numel()
    _run("prism_rope_bwd", dev, q.data_ptr(), plan[3], k.data_ptr(), plan[4], dq.data_ptr(), st[0], dk.data_ptr(), st[1], *vectors,
         *plan[5], gq.data_ptr(), tq, gk.data_ptr(), tk, *sums)
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


@functools.lru_cache(maxsize=4096)
def _prompt(mq, mk, mv, scale, causal, window, S):
    B, H, T, D = sq = _axes("q", mq, "[B, H, T, D]")
    G = _axes("k", mk, "[B, G, T, D]")[1]
    _sizes(B, H, G, T, D, window)
    sk, dtype, sizes = (B, G, T, D), mq[2], (B, H, G, T, D)
    scale = 1 / math.sqrt(D) if scale is None and D else scale
    tail = tuple(map(_ints, (S, *sizes))) + (ctypes.c_float(scale), _ints(causal), _ints(window), _ints(_code(dtype)))
    new = _new_stride(mq), _new_stride(mk), _new_stride(mv)
    return (sq, sk, dtype, _rows("q", mq, sq, dtype), _rows("k", mk, sk, dtype), _rows("v", mv, sk, dtype), tail, new,
            (_new_rows(new[0], sq), _new_rows(new[1], sk), _new_rows(new[2], sk)), (*sizes, _code(dtype)))


def _scale(scale):
    return None if scale is None else float(scale)


def _spans(dev, lens, starts, B, S):
    return (None if lens is None else _dense("lens", lens, (B,), _I32, dev),
            None if starts is None else _dense("starts", starts, (S + 1,), _I32, dev))


@_on_stream
def attn_fwd(q, k, v, scale=None, causal=True, window=0, lens=None, starts=None, out=None):
    """o, lse = attn_fwd(q, k, v): softmax attention of q [B,H,T,D] over k, v [B,G,T,D], each group of H / G heads sharing
    a key head; o [B,H,T,D] in q's dtype, lse [B,H,T] float32.  scale: 1 / sqrt(D) if not given.  causal: token i
    sees tokens up to i; window: the last `window` of them only (0: all).  lens [B] int32: tokens of each sequence; or
    starts [S + 1] int32 with B = 1: sequence s is tokens starts[s] .. starts[s + 1] - 1.  Rows of no sequence keep what
    out = (o, lse) holds (new tensors hold nothing defined there)."""
    dev, S = _gpu(q, "q"), _count(starts)
    plan = _prompt(_meta("q", q), _meta("k", k), _meta("v", v), _scale(scale), bool(causal), window, S)
    _same_device(dev, k, v)
    sq, _, dtype, tq, tk, tv, tail, new, new_rows, _ = plan
    if out is None:
        o, lse = torch.empty_strided(sq, new[0], dtype=dtype, device=dev), torch.empty(sq[:3], dtype=_F32, device=dev)
        to, pl = new_rows[0], lse.data_ptr()
    else:
        o, lse = _given(out, ("o", "lse"))
        to, pl = _rows("o", _meta("o", o), sq, dtype), _dense("lse", lse, sq[:3], _F32, dev)
        _same_device(dev, o)
    _run("prism_attn_fwd", dev, q.data_ptr(), tq, k.data_ptr(), tk, v.data_ptr(), tv, *_spans(dev, lens, starts, sq[0], S), *tail,
         o.data_ptr(), to, pl)
    return o, lse


@_on_stream
def attn_bwd(q, k, v, o, lse, do, scale=None, causal=True, window=0, lens=None, starts=None, out=None, workspace=None):
    """Gradients of <do, o> for attn_fwd with the same arguments, from its o and lse: a dict of dq, dk, dv in q's dtype
    (out: three tensors to write them to).  Rows of no sequence keep what `out` holds (new gradients: zero)."""
    dev, S = _gpu(q, "q"), _count(starts)
    plan = _prompt(_meta("q", q), _meta("k", k), _meta("v", v), _scale(scale), bool(causal), window, S)
    sq, sk, dtype, tq, tk, tv, tail, new, new_rows, sizes = plan
    to, td = _rows("o", _meta("o", o), sq, dtype), _rows("do", _meta("do", do), sq, dtype)
    _same_device(dev, k, v, o, do)
    if lse is None:
        raise PrismError("lse is required")
    if out is None:
        g = [torch.empty_strided(shape, stride, dtype=dtype, device=dev) for shape, stride in zip((sq, sk, sk), new)]
        tg = new_rows
        if lens is not None or starts is not None:
            for t in g:
                t.zero_()
    else:
        g = _given(out, ("dq", "dk", "dv"))
        tg = [_rows(n, _meta(n, t), shape, dtype) for n, t, shape in zip(("dq", "dk", "dv"), g, (sq, sk, sk))]
        _same_device(dev, *g)
    ws = _scratch(workspace, _need("prism_attn_bwd", *sizes), dev)
    dq, dk, dv = g
    _run("prism_attn_bwd", dev, q.data_ptr(), tq, k.data_ptr(), tk, v.data_ptr(), tv, o.data_ptr(), to,
         _dense("lse", lse, sq[:3], _F32, dev), do.data_ptr(), td, *_spans(dev, lens, starts, sq[0], S), *tail, dq.data_ptr(), tg[0],
         dk.data_ptr(), tg[1], dv.data_ptr(), tg[2], ws.data_ptr(), ws.numel())
    return {"dq": dq, "dk": dk, "dv": dv}


# ---- paged cache -------------------------------------------------------------------------------
def _flat(name, meta, shape, dtype):
    """Checks a dense tensor."""
    got, stride, kind = meta
    if got != shape:
        raise PrismError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
    if kind is not dtype:
        raise PrismError(f"{name} must have dtype {dtype}")
    want = 1
    for n, s in zip(reversed(shape), reversed(stride)):
        if n > 1 and s != want:
            raise PrismError(f"{name} must be contiguous")
        want *= n


@functools.lru_cache(maxsize=4096)
def _cache(mk, mv, ms, mt, mp, S, G, D, dtype):
    """Checks of the cache's arguments; pages, page, pages of a sequence."""
    if len(mk[0]) != 4:
        raise PrismError("the caches must be tensors [pages, G, page, D]")
    if len(mt[0]) != 2:
        raise PrismError("table must be a tensor [sequences, pages of a sequence]")
    pages, page, most = mk[0][0], mk[0][2], mt[0][1]
    _sizes(pages, page, most)
    held = dtype if ms is None else torch.float8_e4m3fn
    _flat("cache_k", mk, (pages, G, page, D), held)
    _flat("cache_v", mv, (pages, G, page, D), held)
    for n, m in zip(("scales of the keys", "scales of the values"), ms or ()):
        _flat(n, m, (pages, G, page), _F32)
    _flat("table", mt, (S, most), _I32)
    _flat("past", mp, (S,), _I32)
    return pages, page, most


def _cached(dev, cache_k, cache_v, scales, table, past, S, G, D, dtype):
    """Pointers of the caches, of their scales, of table and past; pages, page, pages of a sequence."""
    ms, sk, sv = None, None, None
    if scales is not None:
        sk, sv = _given(scales, ("of the keys", "of the values"))
        ms = _meta("scales", sk), _meta("scales", sv)
        _same_device(dev, sk, sv)
        sk, sv = sk.data_ptr(), sv.data_ptr()
    sizes = _cache(_meta("cache_k", cache_k), _meta("cache_v", cache_v), ms, _meta("table", table), _meta("past", past), S, G, D, dtype)
    _same_device(dev, cache_k, cache_v, table, past)
    return cache_k.data_ptr(), cache_v.data_ptr(), sk, sv, table.data_ptr(), past.data_ptr(), sizes


@functools.lru_cache(maxsize=4096)
def _new_tokens(mk, mv):
    B, G, T, D = sk = _axes("k", mk, "[B, G, T, D]")
    _sizes(B, G, T, D)
    return sk, _rows("k", mk, sk, mk[2]), _rows("v", mv, sk, mk[2]), _code(mk[2])


@_on_stream
def cache_write(cache_k, cache_v, k, v, table, past, lens=None, starts=None, scales=None):
    """Writes k, v [B,G,T,D] to the paged caches [pages,G,page,D]: token t of sequence s at position past[s] + t, which
    lies in page table[s, position // page].  table [S, pages of a sequence], past [S]: int32.  lens [B] int32: tokens of each
    sequence; or starts [S + 1] int32 with B = 1 (else S = B).  scales: two float32 tensors [pages,G,page] for
    float8_e4m3fn caches (the value is byte value * scale), whose rows are written too."""
    dev, S = _gpu(k, "k"), _count(starts)
    (B, G, T, D), tk, tv, code = _new_tokens(_meta("k", k), _meta("v", v))
    _same_device(dev, v)
    ck, cv, sk, sv, pt, pp, sizes = _cached(dev, cache_k, cache_v, scales, table, past, S or B, G, D, k.dtype)
    _run("prism_cache_write", dev, k.data_ptr(), tk, v.data_ptr(), tv, pt, pp, *_spans(dev, lens, starts, B, S), S, B, G, T, D,
         *sizes, code, ck, cv, sk, sv)


@functools.lru_cache(maxsize=4096)
def _queries(mq):
    B, H, T, D = sq = _axes("q", mq, "[B, H, T, D]")
    _sizes(B, H, T, D)
    new = _new_stride(mq)
    return sq, _rows("q", mq, sq, mq[2]), new, _new_rows(new, sq), _code(mq[2])


@_on_stream
def attn_paged(q, cache_k, cache_v, table, past, lens=None, scales=None, scale=None, window=0, out=None, workspace=None):
    """o = attn_paged(q, cache_k, cache_v, table, past): softmax attention of new tokens q [B,H,T,D] over the paged
    caches [pages,G,page,D] (cache_write), which hold the tokens' own keys and values already: token t of sequence b has
    position past[b] + t and sees the positions up to its own (window: the last `window` of them only).  lens [B] int32: new
    tokens of each sequence; rows past them keep what `out` holds.  scale: 1 / sqrt(D) if not given."""
    dev = _gpu(q, "q")
    sq, tq, new, to, code = _queries(_meta("q", q))
    B, H, T, D = sq
    G = _axes("cache_k", _meta("cache_k", cache_k), "[pages, G, page, D]")[1]
    ck, cv, sk, sv, pt, pp, sizes = _cached(dev, cache_k, cache_v, scales, table, past, B, G, D, q.dtype)
    _sizes(window)
    if out is None:
        o = torch.empty_strided(sq, new, dtype=q.dtype, device=dev)
    else:
        o, to = out, _rows("out", _meta("out", out), sq, q.dtype)
        _same_device(dev, o)
    ws = _scratch(workspace, _need("prism_attn_paged", B, H, G, T, D, *sizes[1:], code), dev)
    _run("prism_attn_paged", dev, q.data_ptr(), tq, ck, cv, sk, sv, pt, pp, None if lens is None else _dense("lens", lens, (B,), _I32, dev),
         B, H, G, T, D, *sizes, 1 / math.sqrt(D) if scale is None and D else scale, window, code, o.data_ptr(), to, ws.data_ptr(),
         ws.numel())
    return o
