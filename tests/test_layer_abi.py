"""Argument checks of the state space layer's entry points.  Every call here fails on the host before anything is
enqueued, so no GPU is needed."""
import ctypes
import os

import pytest

import delta_rule_sequence_amd as prism
from delta_rule_sequence_amd.layer import _Strides

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
BIG = 1 << 40
P = 1 << 20          # an aligned stand-in for a device pointer


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(prism.LIB_PATH):
        pytest.fail("libprism.so is not built (run __graft_entry__.build())")
    return prism.load_library()


def st(b, h, t):
    return ctypes.byref(_Strides(b, h, t))


def ssm_fwd(lib, x=P, xs=None, Bm=P, bs=None, Cm=P, cs=None, dt=P, ts=None, A=P, B=1, H=2, G=1, T=8, N=16, Pw=16, ty=1, y=P,
            ys=None, S=P, ws=P, ws_bytes=BIG):
    return lib.prism_ssm_fwd(x, xs, Bm, bs, Cm, cs, dt, ts, None, A, None, None, None, B, H, G, T, N, Pw, 1, ty, y, ys, S,
                             ws, ws_bytes, None)


def ssm_bwd(lib, x=P, Bm=P, Cm=P, dt=P, A=P, dy=P, B=1, H=2, G=1, T=8, N=16, Pw=16, ty=1, dx=P, dxs=None, dB=P, dBs=None,
            dC=P, ddt=P, dA=P, ws=P, ws_bytes=BIG):
    return lib.prism_ssm_bwd(x, None, Bm, None, Cm, None, dt, None, None, A, None, dy, None, None, B, H, G, T, N, Pw, 1, ty,
                             dx, dxs, dB, dBs, dC, None, ddt, dA, None, None, ws, ws_bytes, None)


def ssm_step(lib, x=P, Bm=P, Cm=P, dt=P, A=P, B=1, H=2, G=1, N=16, Pw=16, ty=1, S=P, y=P, xs=None):
    return lib.prism_ssm_step(x, xs, Bm, None, Cm, None, dt, None, None, A, None, B, H, G, N, Pw, 1, ty, S, y, None)


def conv_fwd(lib, x=P, xs=None, w=P, B=1, H=1, T=8, D=16, K=4, dt=1, y=P, ys=None):
    return lib.prism_conv_fwd(x, xs, w, None, None, None, B, H, T, D, K, 1, dt, y, ys, None, None)


def conv_bwd(lib, x=P, w=P, dy=P, B=1, H=1, T=8, D=16, K=4, dt=1, dx=P, dxs=None, dw=P, ws=P, ws_bytes=BIG):
    return lib.prism_conv_bwd(x, None, w, None, dy, None, B, H, T, D, K, 1, dt, dx, dxs, dw, None, ws, ws_bytes, None)


def conv_step(lib, x=P, w=P, B=1, H=1, D=16, K=4, dt=1, state=P, y=P):
    return lib.prism_conv_step(x, None, w, None, B, H, D, K, 1, dt, state, y, None)


def norm_fwd(lib, x=P, xs=16, gate=None, gs=0, rows=4, D=16, eps=1e-5, dt=1, y=P):
    return lib.prism_norm_fwd(x, xs, None, None, gate, gs, rows, D, eps, dt, y, None, None, None)


def norm_bwd(lib, h=P, hs=16, gate=None, gs=16, dy=P, rows=4, D=16, eps=1e-5, dt=1, dh=P, dgate=None, ws=P, ws_bytes=BIG):
    return lib.prism_norm_bwd(h, hs, None, gate, gs, dy, None, rows, D, eps, dt, dh, dgate, None, ws, ws_bytes, None)


@pytest.mark.parametrize("call,names", [(ssm_fwd, ["x", "Bm", "Cm", "dt", "A", "y", "S"]),
                                        (ssm_bwd, ["x", "Bm", "Cm", "dt", "A", "dy", "dx", "dB", "dC", "ddt", "dA"]),
                                        (ssm_step, ["x", "Bm", "Cm", "dt", "A", "S", "y"]), (conv_fwd, ["x", "w", "y"]),
                                        (conv_bwd, ["x", "w", "dy", "dx", "dw"]), (conv_step, ["x", "w", "state", "y"]),
                                        (norm_fwd, ["x", "y"]), (norm_bwd, ["h", "dy", "dh"])])
def test_null_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == INVALID, n


@pytest.mark.parametrize("call", [ssm_fwd, ssm_bwd])
def test_scan_shapes(lib, call):
    for k in ("B", "H", "G", "T", "N", "Pw"):
        assert call(lib, **{k: 0}) == INVALID and call(lib, **{k: -1}) == INVALID, k
    assert call(lib, ty=2) == INVALID and call(lib, ty=-7) == INVALID
    assert call(lib, H=3, G=2) == INVALID
    assert call(lib, N=24) == UNSUPPORTED and call(lib, Pw=48) == UNSUPPORTED and call(lib, N=256) == UNSUPPORTED
    assert call(lib, B=1 << 15, H=4) == UNSUPPORTED
    assert call(lib, B=1 << 14, H=2, Pw=128) == UNSUPPORTED       # two virtual heads each
    assert call(lib, ws=None) == WORKSPACE and call(lib, ws_bytes=255) == WORKSPACE
    assert call(lib, ws=P + 8) == INVALID
    assert call(lib, x=P + 2) == UNSUPPORTED                       # rows start on 16-byte boundaries


def test_scan_workspace_sizes(lib):
    for name in ("prism_ssm_fwd", "prism_ssm_bwd"):
        f = getattr(lib, name + "_workspace_bytes")
        assert f(1, 1, 1, 1, 16, 16, 0) > 0
        assert f(2, 4, 2, 1000, 128, 128, 1) > 0
        assert f(0, 1, 1, 1, 16, 16, 0) == 0 and f(1, 1, 1, 1, 16, 17, 0) == 0 and f(1, 3, 2, 1, 16, 16, 1) == 0
        assert f(1, 1, 1, 1, 16, 16, 9) == 0
    need = lib.prism_ssm_bwd_workspace_bytes(1, 2, 1, 300, 16, 16, 1)
    assert ssm_bwd(lib, T=300, ws_bytes=need - 1) == WORKSPACE
    need = lib.prism_ssm_fwd_workspace_bytes(1, 2, 1, 3000, 16, 16, 1)
    assert need > 256 and ssm_fwd(lib, T=3000, ws_bytes=need - 1) == WORKSPACE


def test_scan_strides(lib):
    assert ssm_fwd(lib, xs=st(0, 128, 16), B=2) == INVALID         # a broadcast input
    assert ssm_fwd(lib, xs=st(256, -16, 16)) == INVALID
    assert ssm_fwd(lib, xs=st(256, 16, 0)) == INVALID
    assert ssm_fwd(lib, xs=st(256, 16, 33)) == UNSUPPORTED         # rows off the 16-byte boundary
    assert ssm_fwd(lib, xs=st(1 << 62, 16, 32), B=4) == INVALID
    assert ssm_fwd(lib, ys=st(256, 16, 16)) == INVALID             # rows of the output overlap
    assert ssm_bwd(lib, dxs=st(256, 16, 24)) == INVALID
    assert ssm_bwd(lib, dBs=st(256, 16, 8)) == INVALID
    assert ssm_step(lib, xs=st(0, 16, 0), B=2) == INVALID


def test_scan_step_shapes(lib):
    for k in ("B", "H", "G", "N", "Pw"):
        assert ssm_step(lib, **{k: 0}) == INVALID, k
    assert ssm_step(lib, N=20) == UNSUPPORTED and ssm_step(lib, Pw=256) == UNSUPPORTED
    assert ssm_step(lib, H=3, G=2) == INVALID and ssm_step(lib, ty=3) == INVALID
    assert ssm_step(lib, S=P + 4) == UNSUPPORTED
    assert ssm_step(lib, B=1 << 23, H=2) == UNSUPPORTED


@pytest.mark.parametrize("call", [conv_fwd, conv_bwd, conv_step])
def test_conv_shapes(lib, call):
    for k in ("B", "H", "D"):
        assert call(lib, **{k: 0}) == INVALID, k
    assert call(lib, K=1) == UNSUPPORTED and call(lib, K=5) == UNSUPPORTED
    assert call(lib, dt=4) == INVALID
    assert call(lib, B=1 << 16) == UNSUPPORTED
    assert call(lib, B=1 << 10, D=1 << 24) == UNSUPPORTED


def test_conv_strides_and_workspace(lib):
    assert conv_fwd(lib, xs=st(0, 0, 16), B=2) == INVALID
    assert conv_fwd(lib, ys=st(0, 0, 8)) == INVALID                # overlapping output rows
    assert conv_fwd(lib, T=0) == INVALID and conv_bwd(lib, T=-3) == INVALID
    need = lib.prism_conv_bwd_workspace_bytes(1, 1, 8, 16, 4, 1)
    assert need > 0 and conv_bwd(lib, ws_bytes=need - 1) == WORKSPACE and conv_bwd(lib, ws=None) == WORKSPACE
    assert conv_bwd(lib, ws=P + 4) == INVALID
    assert lib.prism_conv_bwd_workspace_bytes(1, 1, 8, 16, 5, 1) == 0


def test_norm_arguments(lib):
    for k in ("rows", "D"):
        assert norm_fwd(lib, **{k: 0}) == INVALID and norm_bwd(lib, **{k: -1}) == INVALID, k
    assert norm_fwd(lib, eps=-1.0) == INVALID and norm_fwd(lib, eps=float("nan")) == INVALID
    assert norm_fwd(lib, xs=15) == INVALID and norm_fwd(lib, gate=P, gs=8) == INVALID
    assert norm_fwd(lib, dt=2) == INVALID
    assert norm_bwd(lib, gate=P) == INVALID                        # dgate is required with a gate
    need = lib.prism_norm_bwd_workspace_bytes(4, 16, 1)
    assert need > 0 and norm_bwd(lib, ws_bytes=need - 1) == WORKSPACE and norm_bwd(lib, ws=P + 4) == INVALID
    assert lib.prism_norm_bwd_workspace_bytes(0, 16, 1) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    x, w = torch.zeros(1, 1, 4, 16), torch.zeros(1, 4, 16)
    bc, dt, A = torch.zeros(1, 1, 4, 16), torch.zeros(1, 1, 4), torch.zeros(1)
    for f in (lambda: prism.conv_fwd(x, w), lambda: prism.conv_bwd(x, w, x), lambda: prism.conv_step(x, x[:, :, 0], w),
              lambda: prism.ssm_fwd(x, bc, bc, dt, A), lambda: prism.ssm_bwd(x, bc, bc, dt, A, x),
              lambda: prism.ssm_step(x, x[:, :, 0], bc[:, :, 0], bc[:, :, 0], dt[:, :, 0], A),
              lambda: prism.norm_fwd(x), lambda: prism.norm_bwd(x, None, x), lambda: prism.norm_fwd(None)):
        with pytest.raises(prism.PrismError):
            f()


def test_conv_in_place_rows(lib):
    """A strip reads rows that its neighbour would overwrite."""
    assert conv_fwd(lib, x=P, y=P) == INVALID
    assert conv_bwd(lib, x=P, dy=2 * P, dx=P) == INVALID and conv_bwd(lib, x=P, dy=2 * P, dx=2 * P) == INVALID


@pytest.mark.parametrize("call", [ssm_fwd, ssm_bwd, conv_fwd, conv_bwd])
def test_longest_sequence(lib, call):
    assert call(lib, T=2 ** 31 - 1) == UNSUPPORTED


@pytest.mark.parametrize("call", [norm_fwd, norm_bwd, conv_fwd, conv_bwd])
def test_widest_rows(lib, call):
    wide = {"xs": 1 << 27} if call is norm_fwd else {"hs": 1 << 27} if call is norm_bwd else {}
    assert call(lib, D=(1 << 26) + 1, **wide) == UNSUPPORTED
