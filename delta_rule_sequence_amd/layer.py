"""The state space layer: causal convolution, selective scan and root-mean-square norm.

Argument marshalling only, as the rest of the binding; the operators are described in
include/prism.h.  Tensors of shape [B, H, T, width] may have any positive strides with a unit
stride in the last axis, so that the heads of a token-major projection output are passed as
views; new outputs take the axis order of the matching input (heads outermost, or tokens).
Calls run on the device of their tensors, on its current stream unless `stream` (a raw
stream handle of that device) is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import PRISM_BF16, PRISM_F32, PrismError, _ptr, _workspace, load_library, status_string

_DTYPES = {torch.bfloat16: PRISM_BF16, torch.float32: PRISM_F32}


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


def declare(lib) -> None:
    """Argument types of the layer's functions."""
    p, i, ll, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    scan_in = [p, p, p, p, p, p, p, p, p, p, p]                 # x, Bm, Cm, dt with strides; dt_bias, A, D
    sigs = {
        "prism_conv_fwd": [p] * 6 + [i] * 7 + [p, p, p, p],
        "prism_conv_bwd": [p] * 6 + [i] * 7 + [p, p, p, p, p, sz, p],
        "prism_conv_step": [p] * 4 + [i] * 6 + [p, p, p],
        "prism_ssm_fwd": scan_in + [p, p] + [i] * 8 + [p, p, p, p, sz, p],
        "prism_ssm_bwd": scan_in + [p, p, p] + [i] * 8 + [p] * 10 + [p, sz, p],
        "prism_ssm_step": scan_in + [i] * 7 + [p, p, p],
        "prism_norm_fwd": [p, ll, p, p, p, ll, i, i, f, i, p, p, p, p],
        "prism_norm_bwd": [p, ll, p, p, ll, p, p, i, i, f, i, p, p, p, p, sz, p],
    }
    for name, args in sigs.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    for name, n in (("prism_conv_bwd", 6), ("prism_ssm_fwd", 7), ("prism_ssm_bwd", 7), ("prism_norm_bwd", 3)):
        fn = getattr(lib, name + "_workspace_bytes")
        fn.argtypes, fn.restype = [i] * n, sz


def _dtype(t) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise PrismError(f"unsupported dtype {t.dtype}: bfloat16 or float32") from None


def _tensor(name, t, shape, dtype, dev):
    """A tensor argument of this shape, dtype and device with a unit stride in the last axis."""
    if not isinstance(t, torch.Tensor):
        raise PrismError(f"{name} is required")
    if t.device != dev:
        raise PrismError(f"{name} must be on {dev}")
    if t.dtype != dtype:
        raise PrismError(f"{name} must have dtype {dtype}")
    if tuple(t.shape) != shape:
        raise PrismError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise PrismError(f"{name} must have a unit stride in its last axis")
    return t


def _dense(name, t, shape, dtype, dev):
    if t is not None and not _tensor(name, t, shape, dtype, dev).is_contiguous():
        raise PrismError(f"{name} must be contiguous")
    return t


def _strides(t, scalar=False):
    """The strides argument of a [B, H, T, width] tensor (scalar: [B, H, T]; without a token axis: t = 0)."""
    if t.is_contiguous():
        return None
    s = t.stride() if scalar else t.stride()[:-1]
    return ctypes.byref(_Strides(s[0], s[1], s[2] if len(s) > 2 else 0))


def _like(t):
    """A new dense tensor of t's shape and dtype, heads or tokens outermost as in t."""
    if t.dim() == 4 and t.shape[1] > 1 and t.stride(1) < t.stride(2):
        B, H, T, W = t.shape
        return torch.empty((B, T, H, W), dtype=t.dtype, device=t.device).transpose(1, 2)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise PrismError(f"{name} is required")
    if t.device.type != "cuda":
        raise PrismError("inputs must be on a GPU")
    return t.device


def _run(name, dev, stream, *args):
    lib = load_library()
    if torch.cuda.current_device() != dev.index:      # kernels launch on the current device
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
            st = getattr(lib, name)(*args, s)
    else:
        s = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        st = getattr(lib, name)(*args, s)
    if st != 0:
        raise PrismError(f"{name} failed: {status_string(st)}")


# ---- convolution -------------------------------------------------------------------------------
def _conv_shape(x, conv_w, bias, dim):
    dev = _gpu(x, "x")
    if x.dim() != dim:
        raise PrismError(f"x must have {dim} axes")
    if not isinstance(conv_w, torch.Tensor) or conv_w.dim() != 3:
        raise PrismError("conv_w must be a tensor [H, K, D]")
    B, H, D, K = x.shape[0], x.shape[1], x.shape[-1], conv_w.shape[1]
    _tensor("x", x, tuple(x.shape), x.dtype, dev)
    _dense("conv_w", conv_w, (H, K, D), torch.float32, dev)
    _dense("bias", bias, (H, D), torch.float32, dev)
    return dev, B, H, D, K


def conv_fwd(x, conv_w, bias=None, silu=True, conv_in=None, lens=None, out=None, want_conv=True, stream=None):
    """y, conv_out = conv_fwd(x, conv_w, bias): the depthwise causal convolution of x [B,H,T,D] with conv_w
    [H,K,D] and bias [H,D] (float32).  conv_in [B,H,K-1,D]: the rows before the first token.  lens [B] int32:
    tokens of each sequence; y rows past them keep what `out` holds (a new y holds nothing defined there).
    conv_out [B,H,K-1,D]: the rows that continue the sequence (None if want_conv is False).  A token-major
    [B,T,C] tensor is x.unsqueeze(1)."""
    dev, B, H, D, K = _conv_shape(x, conv_w, bias, 4)
    T = x.shape[2]
    _dense("conv_in", conv_in, (B, H, K - 1, D), x.dtype, dev)
    _dense("lens", lens, (B,), torch.int32, dev)
    y = _like(x) if out is None else _tensor("out", out, (B, H, T, D), x.dtype, dev)
    conv_out = torch.empty((B, H, max(K - 1, 0), D), dtype=x.dtype, device=dev) if want_conv else None
    _run("prism_conv_fwd", dev, stream, _ptr(x), _strides(x), _ptr(conv_w), _ptr(bias), _ptr(conv_in), _ptr(lens),
         B, H, T, D, K, int(silu), _dtype(x), _ptr(y), _strides(y), _ptr(conv_out))
    return y, conv_out


def conv_bwd(x, conv_w, dy, bias=None, silu=True, out=None, workspace=None, stream=None):
    """Gradients of <dy, y> for conv_fwd(x, conv_w, bias, silu) from a sequence start: a dict of dx (dtype of x; out:
    a tensor to write it to), dconv_w and dbias (float32; dbias only with a bias)."""
    dev, B, H, D, K = _conv_shape(x, conv_w, bias, 4)
    T = x.shape[2]
    _tensor("dy", dy, (B, H, T, D), x.dtype, dev)
    dx = _like(x) if out is None else _tensor("out", out, (B, H, T, D), x.dtype, dev)
    dw = torch.empty_like(conv_w)
    db = torch.empty_like(bias) if bias is not None else None
    ws = _workspace(workspace, load_library().prism_conv_bwd_workspace_bytes(B, H, T, D, K, _dtype(x)), dev)
    _run("prism_conv_bwd", dev, stream, _ptr(x), _strides(x), _ptr(conv_w), _ptr(bias), _ptr(dy), _strides(dy),
         B, H, T, D, K, int(silu), _dtype(x), _ptr(dx), _strides(dx), _ptr(dw), _ptr(db), _ptr(ws), ws.numel())
    return {"dx": dx, "dconv_w": dw} if db is None else {"dx": dx, "dconv_w": dw, "dbias": db}


def conv_step(conv_state, x, conv_w, bias=None, silu=True, stream=None):
    """y = conv_step(conv_state, x, conv_w, bias): one token x [B,H,D]; conv_state [B,H,K-1,D] is updated in place."""
    dev, B, H, D, K = _conv_shape(x, conv_w, bias, 3)
    if conv_state is None:
        raise PrismError("conv_state is required")
    _dense("conv_state", conv_state, (B, H, K - 1, D), x.dtype, dev)
    y = torch.empty((B, H, D), dtype=x.dtype, device=dev)
    _run("prism_conv_step", dev, stream, _ptr(x), _strides(x), _ptr(conv_w), _ptr(bias), B, H, D, K, int(silu),
         _dtype(x), _ptr(conv_state), _ptr(y))
    return y


# ---- scan --------------------------------------------------------------------------------------
def _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, token):
    dev = _gpu(x, "x")
    if x.dim() != (3 if token else 4):
        raise PrismError(f"x must have {3 if token else 4} axes")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != x.dim():
        raise PrismError("Bm must be a tensor with the axes of x")
    B, H, P = x.shape[0], x.shape[1], x.shape[-1]
    T = () if token else (x.shape[2],)
    G, N = Bm.shape[1], Bm.shape[-1]
    _tensor("x", x, (B, H) + T + (P,), x.dtype, dev)
    _tensor("Bm", Bm, (B, G) + T + (N,), x.dtype, dev)
    _tensor("Cm", Cm, (B, G) + T + (N,), x.dtype, dev)
    if not isinstance(dt, torch.Tensor) or dt.device != dev or dt.dtype != torch.float32 or tuple(dt.shape) != (B, H) + T:
        raise PrismError(f"dt must be a float32 tensor of shape {(B, H) + T} on {dev}")
    if A is None:
        raise PrismError("A is required")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        _dense(name, t, (H,), torch.float32, dev)
    return dev, B, H, G, (T[0] if T else 1), N, P


def _scan_args(x, Bm, Cm, dt, dt_bias, A, D):
    return (_ptr(x), _strides(x), _ptr(Bm), _strides(Bm), _ptr(Cm), _strides(Cm), _ptr(dt), _strides(dt, True),
            _ptr(dt_bias), _ptr(A), _ptr(D))


def ssm_fwd(x, Bm, Cm, dt, A, D=None, dt_bias=None, softplus=True, S0=None, lens=None, out=None, workspace=None,
            stream=None):
    """y, S_final = ssm_fwd(x, Bm, Cm, dt, A, D, dt_bias): the selective state space scan of x [B,H,T,P] with Bm, Cm
    [B,G,T,N] (one dtype, bfloat16 or float32) and dt [B,H,T], A, D, dt_bias [H] (float32).  S0 [B,H,N,P] float32:
    the state before the first token.  lens [B] int32: tokens of each sequence; y rows past them keep what `out`
    holds (a new y holds nothing defined there).  S_final [B,H,N,P] float32 is the state after the last token."""
    dev, B, H, G, T, N, P = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, False)
    _dense("S0", S0, (B, H, N, P), torch.float32, dev)
    _dense("lens", lens, (B,), torch.int32, dev)
    y = _like(x) if out is None else _tensor("out", out, (B, H, T, P), x.dtype, dev)
    S = torch.empty((B, H, N, P), dtype=torch.float32, device=dev)
    code = _dtype(x)
    ws = _workspace(workspace, load_library().prism_ssm_fwd_workspace_bytes(B, H, G, T, N, P, code), dev)
    _run("prism_ssm_fwd", dev, stream, *_scan_args(x, Bm, Cm, dt, dt_bias, A, D), _ptr(S0), _ptr(lens),
         B, H, G, T, N, P, int(softplus), code, _ptr(y), _strides(y), _ptr(S), _ptr(ws), ws.numel())
    return y, S


def ssm_bwd(x, Bm, Cm, dt, A, dy, D=None, dt_bias=None, softplus=True, dS_final=None, out=None, workspace=None,
            stream=None):
    """Gradients of <dy, y> + <dS_final, S_final> for ssm_fwd from a zero state: a dict of dx, dB, dC (dtype of x; out:
    three tensors to write them to), ddt, dA (float32) and, where the argument is given, dD and ddt_bias."""
    dev, B, H, G, T, N, P = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, False)
    _tensor("dy", dy, (B, H, T, P), x.dtype, dev)
    _dense("dS_final", dS_final, (B, H, N, P), torch.float32, dev)
    if out is None:
        dx, dB, dC = _like(x), _like(Bm), _like(Cm)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 3:
            raise PrismError("out must be three tensors (dx, dB, dC)")
        dx, dB, dC = (_tensor(n, t, tuple(s.shape), x.dtype, dev) for n, t, s in zip(("dx", "dB", "dC"), out, (x, Bm, Cm)))
    g = {"dx": dx, "dB": dB, "dC": dC, "ddt": torch.empty((B, H, T), dtype=torch.float32, device=dev),
         "dA": torch.empty_like(A)}
    if D is not None:
        g["dD"] = torch.empty_like(D)
    if dt_bias is not None:
        g["ddt_bias"] = torch.empty_like(dt_bias)
    code = _dtype(x)
    ws = _workspace(workspace, load_library().prism_ssm_bwd_workspace_bytes(B, H, G, T, N, P, code), dev)
    _run("prism_ssm_bwd", dev, stream, *_scan_args(x, Bm, Cm, dt, dt_bias, A, D), _ptr(dy), _strides(dy), _ptr(dS_final),
         B, H, G, T, N, P, int(softplus), code, _ptr(dx), _strides(dx), _ptr(dB), _strides(dB), _ptr(dC), _strides(dC),
         _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g.get("dD")), _ptr(g.get("ddt_bias")), _ptr(ws), ws.numel())
    return g


def ssm_step(S, x, Bm, Cm, dt, A, D=None, dt_bias=None, softplus=True, stream=None):
    """y = ssm_step(S, x, Bm, Cm, dt, A, D, dt_bias): one token x [B,H,P], Bm, Cm [B,G,N], dt [B,H]; S [B,H,N,P] float32
    is updated in place."""
    dev, B, H, G, _, N, P = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, True)
    if S is None:
        raise PrismError("S is required")
    _dense("S", S, (B, H, N, P), torch.float32, dev)
    y = torch.empty((B, H, P), dtype=x.dtype, device=dev)
    _run("prism_ssm_step", dev, stream, *_scan_args(x, Bm, Cm, dt, dt_bias, A, D), B, H, G, N, P, int(softplus),
         _dtype(x), _ptr(S), _ptr(y))
    return y


# ---- norm --------------------------------------------------------------------------------------
def _rows(name, t, shape, dtype, dev):
    """Rows of the last axis and their stride; the axes before it must merge into one."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise PrismError(f"{name} must be a tensor")
    if t.device != dev or t.dtype != dtype:
        raise PrismError(f"{name} must have dtype {dtype} on {dev}")
    if tuple(t.shape) != shape:
        raise PrismError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    D = shape[-1]
    if t.is_contiguous():
        return D
    if t.stride(-1) != 1 and D > 1:
        raise PrismError(f"{name} must have a unit stride in its last axis")
    stride, span = None, None
    for n, s in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride, span = s, s * n
        elif s != span:
            raise PrismError(f"the rows of {name} must be evenly spaced (its axes before the last do not merge)")
        else:
            span = s * n
    return D if stride is None else stride


def norm_fwd(x, weight=None, residual=None, gate=None, eps=1e-5, bits8=False, stream=None):
    """Root-mean-square norm over the last axis of x, with h = x + residual before it and y * silu(gate) after: a dict
    of y (the dtype of x, or with bits8 torch.float8_e4m3fn), scales (bits8: float32, one per 128 values of a row,
    y.float() * scale is the value) and h (with residual; the dtype of x).  weight [D] float32; gate like x; both
    x and gate may be views with evenly spaced rows."""
    dev = _gpu(x, "x")
    if x.dim() < 1:
        raise PrismError("x must have at least one axis")
    shape, D = tuple(x.shape), x.shape[-1]
    rows = x.numel() // D if D else 0
    xs = _rows("x", x, shape, x.dtype, dev)
    gs = _rows("gate", gate, shape, x.dtype, dev) if gate is not None else 0
    _dense("weight", weight, (D,), torch.float32, dev)
    _dense("residual", residual, shape, x.dtype, dev)
    code = _dtype(x)
    r = {"y": torch.empty(shape, dtype=torch.float8_e4m3fn if bits8 else x.dtype, device=dev)}
    if bits8:
        r["scales"] = torch.empty(shape[:-1] + (-(-D // 128),), dtype=torch.float32, device=dev)
    if residual is not None:
        r["h"] = torch.empty(shape, dtype=x.dtype, device=dev)
    _run("prism_norm_fwd", dev, stream, _ptr(x), xs, _ptr(residual), _ptr(weight), _ptr(gate), gs, rows, D, eps, code,
         _ptr(r["y"]), _ptr(r.get("scales")), _ptr(r.get("h")))
    return r


def norm_bwd(h, weight, dy, gate=None, dh_in=None, eps=1e-5, workspace=None, stream=None):
    """Gradients of <dy, y> + <dh_in, h> for norm_fwd, with h the row that was normalised: a dict of dh (the gradient of x
    and of residual), dw (float32; with a weight) and dgate (with a gate)."""
    dev = _gpu(h, "h")
    if h.dim() < 1:
        raise PrismError("h must have at least one axis")
    shape, D = tuple(h.shape), h.shape[-1]
    rows = h.numel() // D if D else 0
    hs = _rows("h", h, shape, h.dtype, dev)
    gs = _rows("gate", gate, shape, h.dtype, dev) if gate is not None else 0
    _dense("weight", weight, (D,), torch.float32, dev)
    if dy is None:
        raise PrismError("dy is required")
    _dense("dy", dy, shape, h.dtype, dev)
    _dense("dh_in", dh_in, shape, h.dtype, dev)
    code = _dtype(h)
    g = {"dh": torch.empty(shape, dtype=h.dtype, device=dev)}
    if weight is not None:
        g["dw"] = torch.empty_like(weight)
    if gate is not None:
        g["dgate"] = torch.empty(shape, dtype=h.dtype, device=dev)
    ws = _workspace(workspace, load_library().prism_norm_bwd_workspace_bytes(rows, D, code), dev)
    _run("prism_norm_bwd", dev, stream, _ptr(h), hs, _ptr(weight), _ptr(gate), gs, _ptr(dy), _ptr(dh_in), rows, D, eps,
         code, _ptr(g["dh"]), _ptr(g.get("dgate")), _ptr(g.get("dw")), _ptr(ws), ws.numel())
    return g
