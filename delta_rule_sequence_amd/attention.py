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
    sigs = {
        "prism_attn_fwd": prompt + [p, p, i] + [i] * 5 + [f, i, i, i, p, st, p, p],
        "prism_attn_bwd": prompt + [p, st, p, p, st, p, p, i] + [i] * 5 + [f, i, i, i, p, st, p, st, p, st, p, sz, p],
    }
    for name, args in sigs.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    for name, n in (("prism_attn_bwd", 6),):
        fn = getattr(lib, name + "_workspace_bytes")
        fn.argtypes, fn.restype = [i] * n, sz


# ---- prompts -----------------------------------------------------------------------------------
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
    S = 0
    if starts is not None:
        if not isinstance(starts, torch.Tensor) or starts.dim() != 1 or starts.shape[0] < 2:
            raise PrismError("starts must be a tensor [S + 1]")
        S = starts.shape[0] - 1
        _sizes(S)
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
