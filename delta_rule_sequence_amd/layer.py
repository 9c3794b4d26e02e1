"""The state space layer: causal convolution, selective scan and root-mean-square norm.

Argument marshalling only, as the rest of the binding; the operators are described in
include/prism.h.  Tensors of shape [B, H, T, width] may have any positive strides with a unit
stride in the last axis, so that the heads of a token-major projection output are passed as
views; new outputs take the axis order of the matching input (heads outermost, or tokens).
Calls run on the device of their tensors, on its current stream or on the one given as the
keyword `stream` (a raw stream handle of that device), to which new outputs then belong.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import PRISM_BF16, PRISM_F32, PrismError, load_library, status_string

_DTYPES = {torch.bfloat16: PRISM_BF16, torch.float32: PRISM_F32}
_F32, _I32 = torch.float32, torch.int32


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


def declare(lib) -> None:
    """Argument types of the layer's functions."""
    p, i, ll, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    st = ctypes.POINTER(_Strides)
    scan_in = [p, st, p, st, p, st, p, st, p, p, p]             # x, Bm, Cm, dt with strides; dt_bias, A, D
    sigs = {
        "prism_conv_fwd": [p, st, p, p, p, p] + [i] * 7 + [p, st, p, p],
        "prism_conv_bwd": [p, st, p, p, p, st] + [i] * 7 + [p, st, p, p, p, sz, p],
        "prism_conv_step": [p, st, p, p] + [i] * 6 + [p, p, p],
        "prism_ssm_fwd": scan_in + [p, p] + [i] * 8 + [p, st, p, p, sz, p],
        "prism_ssm_bwd": scan_in + [p, st, p] + [i] * 8 + [p, st, p, st, p, st, p, p, p, p] + [p, sz, p],
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
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise PrismError(f"unsupported dtype {t.dtype}: bfloat16 or float32")
    return code


def _tensor(name, t, shape, dtype, dev):
    """A tensor argument of this shape, dtype and device with a unit stride in the last axis."""
    if not isinstance(t, torch.Tensor):
        raise PrismError(f"{name} is required")
    if t.shape != shape:
        raise PrismError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise PrismError(f"{name} must have dtype {dtype}")
    if t.device != dev:
        raise PrismError(f"{name} must be on {dev}")
    if not t.is_contiguous() and shape[-1] > 1 and t.stride(-1) != 1:
        raise PrismError(f"{name} must have a unit stride in its last axis")
    return t


def _sizes(*n):
    """Sizes as the C interface holds them (ctypes would cut them off)."""
    if max(n) > 0x7fffffff:
        raise PrismError(f"a size of {max(n)} is more than 2^31 - 1")


def _dense(name, t, shape, dtype, dev):
    """A dense tensor argument's pointer (None: not given)."""
    if t is None:
        return None
    if not _tensor(name, t, shape, dtype, dev).is_contiguous():
        raise PrismError(f"{name} must be contiguous")
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _stride_arg(b, h, t):
    return _Strides(b, h, t)


def _strides(t, scalar=False):
    """The strides argument of a [B, H, T, width] tensor (scalar: [B, H, T]; without a token axis: t = 0)."""
    if t.is_contiguous():
        return None
    s = t.stride() if scalar else t.stride()[:-1]
    return _stride_arg(s[0], s[1], s[2] if len(s) > 2 else 0)


def _like(t):
    """A new dense tensor of t's shape and dtype, heads or tokens outermost as in t."""
    if t.dim() == 4 and t.shape[1] > 1 and t.stride(1) < t.stride(2):
        B, H, T, W = t.shape
        return torch.empty((B, T, H, W), dtype=t.dtype, device=t.device).transpose(1, 2)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise PrismError(f"{name} is required")
    if not t.is_cuda:
        raise PrismError("inputs must be on a GPU")
    return t.device


@functools.lru_cache(maxsize=4096)
def _need(name, *shape):
    """Bytes of workspace of a function for a shape (0: refused; the function then says why)."""
    return max(1, getattr(load_library(), name + "_workspace_bytes")(*shape))


def _scratch(workspace, need, dev):
    """The caller's workspace after checking it, or a fresh one of `need` bytes."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise PrismError("workspace must be a uint8 tensor")
    if workspace.device != dev or not workspace.is_contiguous():
        raise PrismError(f"workspace must be a contiguous tensor on {dev}")
    if workspace.numel() < need:
        raise PrismError(f"workspace holds {workspace.numel()} bytes, {need} needed")
    return workspace


def _on_stream(f):
    """Runs f with the stream of its `stream` argument (a raw handle) as torch's current one, so that what it allocates
    belongs to that stream."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        dev = next((t.device for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if dev is None or dev.type != "cuda":
            raise PrismError("inputs must be on a GPU")
        s = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(s):
            return f(*args, **kw)
    return g


@functools.lru_cache(maxsize=None)
def _function(name):
    return getattr(load_library(), name)


def _run(name, dev, *args):
    index = dev.index
    if torch.cuda.current_device() != index:          # kernels launch on the current device
        with torch.cuda.device(dev):
            st = _function(name)(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        st = _function(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise PrismError(f"{name} failed: {status_string(st)}")


# ---- convolution -------------------------------------------------------------------------------
def _conv_shape(x, conv_w, bias, dim):
    dev = _gpu(x, "x")
    if x.dim() != dim:
        raise PrismError(f"x must have {dim} axes")
    if not isinstance(conv_w, torch.Tensor) or conv_w.dim() != 3:
        raise PrismError("conv_w must be a tensor [H, K, D]")
    shape, K = x.shape, conv_w.shape[1]
    B, H, D = shape[0], shape[1], shape[-1]
    _sizes(K, *shape)
    _tensor("x", x, shape, x.dtype, dev)
    return dev, B, H, D, K, _dense("conv_w", conv_w, (H, K, D), _F32, dev), _dense("bias", bias, (H, D), _F32, dev)


@_on_stream
def conv_fwd(x, conv_w, bias=None, silu=True, conv_in=None, lens=None, out=None, want_conv=True):
    """y, conv_out = conv_fwd(x, conv_w, bias): the depthwise causal convolution of x [B,H,T,D] with conv_w
    [H,K,D] and bias [H,D] (float32).  conv_in [B,H,K-1,D]: the rows before the first token.  lens [B] int32:
    tokens of each sequence; y rows past them keep what `out` holds (a new y holds nothing defined there).
    conv_out [B,H,K-1,D]: the rows that continue the sequence (None if want_conv is False).  A token-major
    [B,T,C] tensor is x.unsqueeze(1)."""
    dev, B, H, D, K, pw, pb = _conv_shape(x, conv_w, bias, 4)
    T = x.shape[2]
    p_in, p_lens = _dense("conv_in", conv_in, (B, H, K - 1, D), x.dtype, dev), _dense("lens", lens, (B,), _I32, dev)
    y = _like(x) if out is None else _tensor("out", out, (B, H, T, D), x.dtype, dev)
    conv_out = torch.empty((B, H, max(K - 1, 0), D), dtype=x.dtype, device=dev) if want_conv else None
    _run("prism_conv_fwd", dev, x.data_ptr(), _strides(x), pw, pb, p_in, p_lens, B, H, T, D, K, bool(silu), _dtype(x),
         y.data_ptr(), _strides(y), conv_out.data_ptr() if want_conv else None)
    return y, conv_out


@_on_stream
def conv_bwd(x, conv_w, dy, bias=None, silu=True, out=None, workspace=None):
    """Gradients of <dy, y> for conv_fwd(x, conv_w, bias, silu) from a sequence start: a dict of dx (dtype of x; out:
    a tensor to write it to), dconv_w and dbias (float32; dbias only with a bias)."""
    dev, B, H, D, K, pw, pb = _conv_shape(x, conv_w, bias, 4)
    T = x.shape[2]
    _tensor("dy", dy, (B, H, T, D), x.dtype, dev)
    dx = _like(x) if out is None else _tensor("out", out, (B, H, T, D), x.dtype, dev)
    dw = torch.empty_like(conv_w)
    db = torch.empty_like(bias) if bias is not None else None
    code = _dtype(x)
    ws = _scratch(workspace, _need("prism_conv_bwd", B, H, T, D, K, code), dev)
    _run("prism_conv_bwd", dev, x.data_ptr(), _strides(x), pw, pb, dy.data_ptr(), _strides(dy), B, H, T, D, K, bool(silu),
         code, dx.data_ptr(), _strides(dx), dw.data_ptr(), None if db is None else db.data_ptr(), ws.data_ptr(), ws.numel())
    return {"dx": dx, "dconv_w": dw} if db is None else {"dx": dx, "dconv_w": dw, "dbias": db}


@_on_stream
def conv_step(conv_state, x, conv_w, bias=None, silu=True):
    """y = conv_step(conv_state, x, conv_w, bias): one token x [B,H,D]; conv_state [B,H,K-1,D] is updated in place."""
    dev, B, H, D, K, pw, pb = _conv_shape(x, conv_w, bias, 3)
    if conv_state is None:
        raise PrismError("conv_state is required")
    p_state = _dense("conv_state", conv_state, (B, H, K - 1, D), x.dtype, dev)
    y = torch.empty((B, H, D), dtype=x.dtype, device=dev)
    _run("prism_conv_step", dev, x.data_ptr(), _strides(x), pw, pb, B, H, D, K, bool(silu), _dtype(x), p_state, y.data_ptr())
    return y


# ---- scan --------------------------------------------------------------------------------------
def _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, token):
    dev = _gpu(x, "x")
    if x.dim() != (3 if token else 4):
        raise PrismError(f"x must have {3 if token else 4} axes")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != x.dim():
        raise PrismError("Bm must be a tensor with the axes of x")
    shape, (G, N) = x.shape, (Bm.shape[1], Bm.shape[-1])
    B, H, P = shape[0], shape[1], shape[-1]
    bc = (B, G, N) if token else (B, G, shape[2], N)
    _sizes(G, N, *shape)
    _tensor("x", x, shape, x.dtype, dev)
    _tensor("Bm", Bm, bc, x.dtype, dev)
    _tensor("Cm", Cm, bc, x.dtype, dev)
    if not isinstance(dt, torch.Tensor) or dt.device != dev or dt.dtype is not _F32 or dt.shape != shape[:-1]:
        raise PrismError(f"dt must be a float32 tensor of shape {tuple(shape[:-1])} on {dev}")
    if A is None:
        raise PrismError("A is required")
    vec = (H,)
    args = (x.data_ptr(), _strides(x), Bm.data_ptr(), _strides(Bm), Cm.data_ptr(), _strides(Cm), dt.data_ptr(), _strides(dt, True),
            _dense("dt_bias", dt_bias, vec, _F32, dev), _dense("A", A, vec, _F32, dev), _dense("D", D, vec, _F32, dev))
    return dev, B, H, G, (1 if token else shape[2]), N, P, args


@_on_stream
def ssm_fwd(x, Bm, Cm, dt, A, D=None, dt_bias=None, softplus=True, S0=None, lens=None, out=None, workspace=None):
    """y, S_final = ssm_fwd(x, Bm, Cm, dt, A, D, dt_bias): the selective state space scan of x [B,H,T,P] with Bm, Cm
    [B,G,T,N] (one dtype, bfloat16 or float32) and dt [B,H,T], A, D, dt_bias [H] (float32).  S0 [B,H,N,P] float32:
    the state before the first token.  lens [B] int32: tokens of each sequence; y rows past them keep what `out`
    holds (a new y holds nothing defined there).  S_final [B,H,N,P] float32 is the state after the last token."""
    dev, B, H, G, T, N, P, args = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, False)
    p_s0, p_lens = _dense("S0", S0, (B, H, N, P), _F32, dev), _dense("lens", lens, (B,), _I32, dev)
    y = _like(x) if out is None else _tensor("out", out, (B, H, T, P), x.dtype, dev)
    S = torch.empty((B, H, N, P), dtype=torch.float32, device=dev)
    code = _dtype(x)
    ws = _scratch(workspace, _need("prism_ssm_fwd", B, H, G, T, N, P, code), dev)
    _run("prism_ssm_fwd", dev, *args, p_s0, p_lens, B, H, G, T, N, P, bool(softplus), code, y.data_ptr(), _strides(y),
         S.data_ptr(), ws.data_ptr(), ws.numel())
    return y, S


@_on_stream
def ssm_bwd(x, Bm, Cm, dt, A, dy, D=None, dt_bias=None, softplus=True, dS_final=None, out=None, workspace=None):
    """Gradients of <dy, y> + <dS_final, S_final> for ssm_fwd from a zero state: a dict of dx, dB, dC (dtype of x; out:
    three tensors to write them to), ddt, dA (float32) and, where the argument is given, dD and ddt_bias."""
    dev, B, H, G, T, N, P, args = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, False)
    _tensor("dy", dy, (B, H, T, P), x.dtype, dev)
    p_ds = _dense("dS_final", dS_final, (B, H, N, P), _F32, dev)
    if out is None:
        dx, dB, dC = _like(x), _like(Bm), _like(Cm)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 3:
            raise PrismError("out must be three tensors (dx, dB, dC)")
        dx, dB, dC = (_tensor(n, t, s.shape, x.dtype, dev) for n, t, s in zip(("dx", "dB", "dC"), out, (x, Bm, Cm)))
    g = {"dx": dx, "dB": dB, "dC": dC, "ddt": torch.empty((B, H, T), dtype=torch.float32, device=dev),
         "dA": torch.empty_like(A)}
    if D is not None:
        g["dD"] = torch.empty_like(D)
    if dt_bias is not None:
        g["ddt_bias"] = torch.empty_like(dt_bias)
    code = _dtype(x)
    ws = _scratch(workspace, _need("prism_ssm_bwd", B, H, G, T, N, P, code), dev)
    _run("prism_ssm_bwd", dev, *args, dy.data_ptr(), _strides(dy), p_ds, B, H, G, T, N, P, bool(softplus), code,
         dx.data_ptr(), _strides(dx), dB.data_ptr(), _strides(dB), dC.data_ptr(), _strides(dC), g["ddt"].data_ptr(),
         g["dA"].data_ptr(), None if D is None else g["dD"].data_ptr(), None if dt_bias is None else g["ddt_bias"].data_ptr(),
         ws.data_ptr(), ws.numel())
    return g


@_on_stream
def ssm_step(S, x, Bm, Cm, dt, A, D=None, dt_bias=None, softplus=True):
    """y = ssm_step(S, x, Bm, Cm, dt, A, D, dt_bias): one token x [B,H,P], Bm, Cm [B,G,N], dt [B,H]; S [B,H,N,P] float32
    is updated in place."""
    dev, B, H, G, _, N, P, args = _scan_shape(x, Bm, Cm, dt, A, D, dt_bias, True)
    if S is None:
        raise PrismError("S is required")
    p_s = _dense("S", S, (B, H, N, P), _F32, dev)
    y = torch.empty((B, H, P), dtype=x.dtype, device=dev)
    _run("prism_ssm_step", dev, *args, B, H, G, N, P, bool(softplus), _dtype(x), p_s, y.data_ptr())
    return y


# ---- norm --------------------------------------------------------------------------------------
def _rows(name, t, shape, dtype, dev):
    """Rows of the last axis and their stride; the axes before it must merge into one."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise PrismError(f"{name} must be a tensor")
    if t.device != dev or t.dtype != dtype:
        raise PrismError(f"{name} must have dtype {dtype} on {dev}")
    if t.shape != shape:
        raise PrismError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
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


@_on_stream
def norm_fwd(x, weight=None, residual=None, gate=None, eps=1e-5, bits8=False):
    """Root-mean-square norm over the last axis of x, with h = x + residual before it and y * silu(gate) after: a dict
    of y (the dtype of x, or with bits8 torch.float8_e4m3fn), scales (bits8: float32, one per 128 values of a row,
    y.float() * scale is the value) and h (with residual; the dtype of x).  weight [D] float32; gate like x; both
    x and gate may be views with evenly spaced rows."""
    dev = _gpu(x, "x")
    if x.dim() < 1:
        raise PrismError("x must have at least one axis")
    shape, D = x.shape, x.shape[-1]
    rows = x.numel() // D if D else 0
    _sizes(rows, D)
    xs = _rows("x", x, shape, x.dtype, dev)
    gs = _rows("gate", gate, shape, x.dtype, dev) if gate is not None else 0
    pw, pr = _dense("weight", weight, (D,), _F32, dev), _dense("residual", residual, shape, x.dtype, dev)
    code = _dtype(x)
    y, ps, ph = torch.empty(shape, dtype=torch.float8_e4m3fn if bits8 else x.dtype, device=dev), None, None
    r = {"y": y}
    if bits8:
        r["scales"] = scales = torch.empty((*shape[:-1], -(-D // 128)), dtype=_F32, device=dev)
        ps = scales.data_ptr()
    if pr is not None:
        r["h"] = h = torch.empty(shape, dtype=x.dtype, device=dev)
        ph = h.data_ptr()
    _run("prism_norm_fwd", dev, x.data_ptr(), xs, pr, pw, None if gate is None else gate.data_ptr(), gs, rows, D, eps, code,
         y.data_ptr(), ps, ph)
    return r


@_on_stream
def norm_bwd(h, weight, dy, gate=None, dh_in=None, eps=1e-5, workspace=None):
    """Gradients of <dy, y> + <dh_in, h> for norm_fwd, with h the row that was normalised: a dict of dh (the gradient of x
    and of residual), dw (float32; with a weight) and dgate (with a gate)."""
    dev = _gpu(h, "h")
    if h.dim() < 1:
        raise PrismError("h must have at least one axis")
    shape, D = h.shape, h.shape[-1]
    rows = h.numel() // D if D else 0
    _sizes(rows, D)
    hs = _rows("h", h, shape, h.dtype, dev)
    gs = _rows("gate", gate, shape, h.dtype, dev) if gate is not None else 0
    pw, pi = _dense("weight", weight, (D,), _F32, dev), _dense("dh_in", dh_in, shape, h.dtype, dev)
    if dy is None:
        raise PrismError("dy is required")
    py, code = _dense("dy", dy, shape, h.dtype, dev), _dtype(h)
    dh, dw, dz = torch.empty(shape, dtype=h.dtype, device=dev), None, None
    g = {"dh": dh}
    if weight is not None:
        g["dw"] = dw = torch.empty_like(weight)
    if gate is not None:
        g["dgate"] = dz = torch.empty(shape, dtype=h.dtype, device=dev)
    ws = _scratch(workspace, _need("prism_norm_bwd", rows, D, code), dev)
    _run("prism_norm_bwd", dev, h.data_ptr(), hs, pw, None if gate is None else gate.data_ptr(), gs, py, pi, rows, D, eps, code,
         dh.data_ptr(), None if dz is None else dz.data_ptr(), None if dw is None else dw.data_ptr(), ws.data_ptr(), ws.numel())
    return g
