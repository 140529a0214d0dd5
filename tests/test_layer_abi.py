"""Refusals of the recurrence, norm and 8-bit calls (CPU only): every call here
fails its argument checks and returns before it touches the CUDA runtime."""
import ctypes

import pytest
import torch

from kalman_filter_linear_b200 import build, kdn

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)
WS = ctypes.c_void_p(0x20000)
INVALID, UNSUPPORTED, WORKSPACE = (kdn.KDN_ERR_INVALID_ARG, kdn.KDN_ERR_UNSUPPORTED,
                                   kdn.KDN_ERR_WORKSPACE)


@pytest.fixture(scope='module')
def L():
    if build.is_stale():
        build.build()
    return kdn.lib()


def _caller(fn, base):
    return lambda **kw: fn(*{**base, **kw}.values())


def test_scan_forward(L):
    x = _caller(L.kdn_linear_scan_forward,
                dict(a=FAKE, b=None, gate=0, x=FAKE, dt=1, h0=None, cu=None, y=FAKE, h=FAKE, B=2,
                     T=300, D=64, ws=WS, wsb=1 << 40, stream=None))
    for name in ('a', 'x', 'y', 'h'):
        assert x(**{name: None}) == INVALID
    for name in ('a', 'b', 'x', 'h0', 'y', 'h', 'cu'):
        assert x(**{name: ctypes.c_void_p(0x10002)}) == INVALID
    assert x(gate=2) == INVALID and x(dt=2) == INVALID and x(dt=-1) == INVALID
    assert x(B=0) == INVALID and x(T=-1) == INVALID and x(D=0) == INVALID
    assert x(T=(1 << 30) + 1) == INVALID
    assert x(B=1 << 20, T=1 << 20, D=1024) == INVALID
    assert x(ws=None) == WORKSPACE and x(wsb=255) == WORKSPACE
    assert x(ws=ctypes.c_void_p(0x20010)) == INVALID
    assert L.kdn_linear_scan_workspace_size(2, 300, 64) >= 256
    assert L.kdn_linear_scan_workspace_size(2, 0, 64) == 256
    assert L.kdn_linear_scan_workspace_size(0, 300, 64) == 0
    # more than 2^31 tiles
    assert x(B=1 << 30, T=64, D=65) == INVALID or x(B=1 << 30, T=64, D=65) == UNSUPPORTED


def test_scan_backward(L):
    x = _caller(L.kdn_linear_scan_backward,
                dict(a=FAKE, b=None, gate=0, x=None, y=FAKE, dy=FAKE, dt=1, h0=None, dhT=None,
                     cu=None, da=FAKE, db=None, dx=FAKE, dh0=FAKE, B=2, T=300, D=64, ws=WS,
                     wsb=1 << 40, stream=None))
    for name in ('a', 'y', 'dy', 'da', 'dx', 'dh0'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: MIS}) == INVALID
    assert x(b=FAKE, db=FAKE) == INVALID            # db needs x
    assert x(b=FAKE, x=FAKE) == INVALID             # and its output
    assert x(dhT=MIS) == INVALID and x(h0=MIS) == INVALID
    assert x(B=0) == INVALID and x(gate=3) == INVALID
    assert x(ws=None) == WORKSPACE and x(wsb=64) == WORKSPACE


def test_scan_step(L):
    x = _caller(L.kdn_linear_scan_step,
                dict(a=FAKE, b=None, gate=0, x=FAKE, dt=1, h=FAKE, y=FAKE, B=2, D=64, stream=None))
    for name in ('a', 'x', 'h', 'y'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: MIS}) == INVALID
    assert x(B=0) == INVALID and x(D=-1) == INVALID and x(dt=2) == INVALID


def test_norm_forward(L):
    x = _caller(L.kdn_rmsnorm_forward,
                dict(x=FAKE, xt=0, res=None, rt=0, w=FAKE, h=None, y=FAKE, yt=1, ldy=0, scale=None,
                     rows=4, D=64, eps=1e-6, stream=None))
    for name in ('x', 'w', 'y'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: MIS}) == INVALID
    assert x(xt=2) == INVALID and x(yt=3) == INVALID
    assert x(res=FAKE) == INVALID                   # h is needed with a residual
    assert x(h=FAKE) == INVALID                     # and only with one
    assert x(res=FAKE, h=FAKE, rt=2) == INVALID
    assert x(rows=-1) == INVALID and x(D=0) == INVALID
    assert x(eps=-1.0) == INVALID and x(eps=float('nan')) == INVALID
    assert x(eps=float('inf')) == INVALID
    assert x(D=16385) == UNSUPPORTED
    assert x(yt=2, ldy=64) == INVALID               # e4m3 needs scales
    assert x(yt=2, scale=FAKE, ldy=63) == INVALID
    assert x(yt=2, scale=FAKE, ldy=72) == INVALID   # not a multiple of 16
    assert x(yt=2, scale=ctypes.c_void_p(0x10002), ldy=64) == INVALID
    assert x(rows=0) == kdn.KDN_OK


def test_norm_backward(L):
    x = _caller(L.kdn_rmsnorm_backward,
                dict(h=FAKE, ht=0, w=FAKE, dy=FAKE, yt=1, dh=None, dx=FAKE, xt=0, dres=None,
                     dw=FAKE, rows=4, D=64, eps=1e-6, ws=WS, wsb=1 << 30, stream=None))
    for name in ('h', 'w', 'dy', 'dx', 'dw'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: MIS}) == INVALID
    assert x(dh=MIS) == INVALID and x(dres=MIS) == INVALID
    assert x(ht=2) == INVALID and x(yt=2) == INVALID and x(xt=2) == INVALID
    assert x(D=20000) == UNSUPPORTED
    assert x(ws=None) == WORKSPACE and x(wsb=16) == WORKSPACE
    assert x(ws=ctypes.c_void_p(0x20010)) == INVALID
    assert L.kdn_rmsnorm_backward_workspace_size(4, 64) >= 4 * 64 * 4
    assert L.kdn_rmsnorm_backward_workspace_size(0, 64) == 0


def test_quantize(L):
    x = _caller(L.kdn_fp8_quantize,
                dict(x=FAKE, xt=0, rows=4, cols=100, tile=0, tr=0, q=FAKE, ldq=112, s=FAKE,
                     stream=None))
    for name in ('x', 'q', 's'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: ctypes.c_void_p(0x10002)}) == INVALID
    assert x(xt=2) == INVALID and x(rows=-1) == INVALID and x(cols=0) == INVALID
    assert x(ldq=100) == INVALID and x(ldq=96) == INVALID
    assert x(tr=1, rows=120, ldq=112) == INVALID    # the output's rows are 120 long
    assert x(rows=0) == kdn.KDN_OK


def test_matmul(L):
    x = _caller(L.kdn_fp8_matmul,
                dict(x=FAKE, ldx=112, sx=FAKE, w=FAKE, ldw=112, sw=FAKE, tile=1, out=FAKE, ot=1,
                     M=4, N=8, K=100, status=None, stream=None))
    for name in ('x', 'sx', 'w', 'sw', 'out'):
        assert x(**{name: None}) == INVALID
        assert x(**{name: ctypes.c_void_p(0x10002)}) == INVALID
    assert x(status=ctypes.c_void_p(0x10002)) == INVALID
    assert x(ot=2) == INVALID and x(M=-1) == INVALID and x(N=0) == INVALID and x(K=0) == INVALID
    assert x(ldx=96) == INVALID and x(ldw=104) == INVALID
    assert x(M=1 << 30, N=1 << 30) == UNSUPPORTED
    assert x(M=0) == kdn.KDN_OK


def test_cpu_tensors_are_refused():
    f = torch.zeros(2, 4, 8)
    e = torch.zeros(4, 16, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    for call in (lambda: kdn.kdn_linear_scan_forward(f, f), lambda: kdn.kdn_linear_scan_step(s, s, s),
                 lambda: kdn.kdn_linear_scan_backward(f, f, f, f),
                 lambda: kdn.kdn_rmsnorm_forward(f, torch.ones(8)),
                 lambda: kdn.kdn_rmsnorm_backward(f, torch.ones(8), f),
                 lambda: kdn.kdn_fp8_quantize(s), lambda: kdn.kdn_fp8_matmul(e, s, e, s)):
        with pytest.raises(TypeError, match='CUDA tensor'):
            call()
