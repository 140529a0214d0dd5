"""Thin ctypes binding of libkdn (include/kdn.h).

Argument marshalling only: every function checks that its tensors are CUDA
(host, for kdn_forward_host), contiguous and of the right dtype, allocates
outputs with PyTorch when the caller gives none, and passes raw pointers and
the current CUDA stream to the C ABI.  All arithmetic happens in the library's kernels.  If
``libkdn.so`` cannot be loaded the first call raises; there is no fallback.  The
calls around a layer (linear recurrence, norm, 8 bits), which are small when
decoding, have a quick form in C++ that does the same (csrc/quick_binding.cpp).
Function names match the C entry points.
"""
from __future__ import annotations

import ctypes
import functools
import os
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, 'libkdn.so')

KDN_OK, KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED, KDN_ERR_WORKSPACE, KDN_ERR_TIMEOUT, \
    KDN_ERR_CUDA = range(6)
KDN_F32, KDN_BF16, KDN_E4M3 = 0, 1, 2
KDN_ISO, KDN_DIAG = 0, 1
KDN_CHUNK_AUTO, KDN_CHUNK_RECURRENT, KDN_CHUNK_64 = 0, 1, 64

_lib = None
_vp, _i64, _i32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                              ctypes.c_size_t)


class KdnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f'{where}: {lib().kdn_status_string(status).decode()}')


def lib():
    """Load libkdn.so (once) and declare the prototypes of include/kdn.h."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f'{LIB_PATH} is missing: build it with '
                           '`python -m kalman_filter_linear_b200.build`')
    L = ctypes.CDLL(LIB_PATH)
    L.kdn_status_string.restype = ctypes.c_char_p
    L.kdn_status_string.argtypes = [_i32]
    L.kdn_version.restype = _i32
    L.kdn_mobius_scan_workspace_size.restype = _sz
    L.kdn_mobius_scan_workspace_size.argtypes = [_i64, _i64]
    L.kdn_mobius_scan.restype = _i32
    L.kdn_mobius_scan.argtypes = [_vp] * 5 + [_f32] + [_vp] * 3 + [_i64, _i64, _vp, _sz, _vp]
    L.kdn_mobius_scan_noalloc.restype = _i32
    L.kdn_mobius_scan_noalloc.argtypes = [_vp] * 5 + [_f32] + [_vp] * 3 + [_i64, _i64, _vp]
    L.kdn_forward_workspace_size.restype = _sz
    L.kdn_forward_workspace_size.argtypes = [_i32] * 7
    L.kdn_iso_forward.restype = _i32
    L.kdn_iso_forward.argtypes = [_vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + \
        [_f32, _i32, _vp, _sz, _vp]
    L.kdn_forward_varlen_workspace_size.restype = _sz
    L.kdn_forward_varlen_workspace_size.argtypes = [_i32] * 6
    L.kdn_forward_varlen.restype = _i32
    L.kdn_forward_varlen.argtypes = [_i32, _vp, _vp, _vp, _i32] + [_vp] * 9 + [_i32] * 5 + \
        [_f32, _i32, _vp, _sz, _vp]
    L.kdn_forward_host_workspace_size.restype = _sz
    L.kdn_forward_host_workspace_size.argtypes = [_i32] * 9
    L.kdn_forward_host.restype = _i32
    L.kdn_forward_host.argtypes = [_i32, _vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + \
        [_f32, _i32, _i32, _vp, _sz, _vp]
    L.kdn_diag_forward.restype = _i32
    L.kdn_diag_forward.argtypes = [_vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + \
        [_i32, _vp, _sz, _vp]
    L.kdn_decode_step.restype = _i32
    L.kdn_decode_step.argtypes = [_i32, _vp, _vp, _vp, _i32] + [_vp] * 6 + [_i32] * 4 + \
        [_f32, _vp]
    L.kdn_exact_forward.restype = _i32
    L.kdn_exact_forward.argtypes = [_i32, _vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + [_vp]
    L.kdn_backward_workspace_size.restype = _sz
    L.kdn_backward_workspace_size.argtypes = [_i32] * 6
    L.kdn_backward.restype = _i32
    L.kdn_backward.argtypes = [_i32, _vp, _vp, _vp, _i32] + [_vp] * 16 + [_i32] * 5 + \
        [_f32, _vp, _sz, _vp]
    L.kdn_kla_forward.restype = _i32
    L.kdn_kla_forward.argtypes = [_vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + [_vp]
    L.kdn_kla_workspace_size.restype = _sz
    L.kdn_kla_workspace_size.argtypes = [_i32] * 5
    L.kdn_kla_forward_ws.restype = _i32
    L.kdn_kla_forward_ws.argtypes = [_vp, _vp, _vp, _i32] + [_vp] * 8 + [_i32] * 5 + \
        [_vp, _sz, _vp]
    L.kdn_linear_scan_workspace_size.restype = _sz
    L.kdn_linear_scan_workspace_size.argtypes = [_i32] * 3
    L.kdn_linear_scan_forward.restype = _i32
    L.kdn_linear_scan_forward.argtypes = [_vp, _vp, _i32, _vp, _i32] + [_vp] * 4 + [_i32] * 3 + \
        [_vp, _sz, _vp]
    L.kdn_linear_scan_backward.restype = _i32
    L.kdn_linear_scan_backward.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _i32] + [_vp] * 7 + \
        [_i32] * 3 + [_vp, _sz, _vp]
    L.kdn_linear_scan_step.restype = _i32
    L.kdn_linear_scan_step.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp]
    L.kdn_rmsnorm_forward.restype = _i32
    L.kdn_rmsnorm_forward.argtypes = [_vp, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _vp, _i64,
                                      _i32, _f32, _vp]
    L.kdn_rmsnorm_backward_workspace_size.restype = _sz
    L.kdn_rmsnorm_backward_workspace_size.argtypes = [_i64, _i32]
    L.kdn_rmsnorm_backward.restype = _i32
    L.kdn_rmsnorm_backward.argtypes = [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _i64,
                                       _i32, _f32, _vp, _sz, _vp]
    L.kdn_fp8_quantize.restype = _i32
    L.kdn_fp8_quantize.argtypes = [_vp, _i32, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp]
    L.kdn_fp8_matmul.restype = _i32
    L.kdn_fp8_matmul.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _i32, _i32, _i32,
                                 _i32, _vp, _vp]
    L.kdn_read_workspace_status.restype = _i32
    L.kdn_read_workspace_status.argtypes = [_vp, _sz, _vp]
    L.kdn_testing_mobius_scan_unpublished_tile.restype = _i32
    L.kdn_testing_kla_skip_v_copy.restype = _i32
    L.kdn_testing_kla_skip_v_copy.argtypes = [_vp] * 9 + [_i32] * 4 + [_vp, _sz, _vp]
    L.kdn_testing_linear_scan_skip_copy.restype = _i32
    L.kdn_testing_linear_scan_skip_copy.argtypes = [_vp] * 4 + [_i32] * 3 + [_i64, _vp, _sz, _vp]
    L.kdn_testing_fp8_matmul_skip_copy.restype = _i32
    L.kdn_testing_fp8_matmul_skip_copy.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _i32, _vp] + \
        [_i32] * 5 + [_vp, _vp]
    L.kdn_testing_forward_skip_v_copy.restype = _i32
    L.kdn_testing_forward_skip_v_copy.argtypes = [_i32] + [_vp] * 9 + [_i32] * 4 + [_vp, _sz, _vp]
    L.kdn_testing_mobius_scan_unpublished_tile.argtypes = [_vp] * 5 + [_f32, _vp, _i64, _i64,
                                                                       _vp, _sz, _i64, _vp]
    _lib = L
    return L


def _check(status, where):
    if status != KDN_OK:
        raise KdnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _req(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f'{name} must be a CUDA tensor')
    if not t.is_contiguous():
        raise ValueError(f'{name} must be contiguous')
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f'{name} must be {dtype}, got {t.dtype}')
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f'{name} must have shape {tuple(shape)}, got {tuple(t.shape)}')
    return t


def _opt(t, name, dtype, shape):
    return None if t is None else _req(t, name, dtype, shape)


def _in_dtype(t):
    if t.dtype == torch.bfloat16:
        return KDN_BF16
    if t.dtype == torch.float32:
        return KDN_F32
    raise TypeError(f'q/k/v must be bfloat16 or float32, got {t.dtype}')


def _workspace(nbytes, device, ws):
    if nbytes == 0:
        return ws
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def kdn_mobius_scan_workspace_size(N, T):
    return int(lib().kdn_mobius_scan_workspace_size(N, T))


def kdn_mobius_scan(a, w, r, n, lambda0=None, info_scale=1.0, lambda_out=None, prior_out=None,
                    gain_out=None, workspace=None, want_prior=False, want_gain=False):
    """Variance (Mobius) scan over [N, T] lanes.  Returns (lambda, prior, gain,
    workspace); prior / gain are None unless requested or given."""
    N, T = a.shape
    f = torch.float32
    for name, t in (('a', a), ('w', w), ('r', r), ('n', n)):
        _req(t, name, f, (N, T))
    _opt(lambda0, 'lambda0', f, (N,))
    lambda_out = _opt(lambda_out, 'lambda_out', f, (N, T)) if lambda_out is not None else \
        torch.empty_like(a)
    if prior_out is None and want_prior:
        prior_out = torch.empty_like(a)
    if gain_out is None and want_gain:
        gain_out = torch.empty_like(a)
    _opt(prior_out, 'prior_out', f, (N, T))
    _opt(gain_out, 'gain_out', f, (N, T))
    need = kdn_mobius_scan_workspace_size(N, T)
    workspace = _workspace(need, a.device, workspace)
    st = lib().kdn_mobius_scan(_ptr(a), _ptr(w), _ptr(r), _ptr(n), _ptr(lambda0),
                               float(info_scale), _ptr(lambda_out), _ptr(prior_out),
                               _ptr(gain_out), N, T, _ptr(workspace),
                               workspace.numel() if workspace is not None else 0, _stream())
    _check(st, 'kdn_mobius_scan')
    return lambda_out, prior_out, gain_out, workspace


KDN_SCAN_NOALLOC_MAX_TILES = 229376


def kdn_mobius_scan_noalloc(a, w, r, n, lambda0=None, info_scale=1.0, lambda_out=None,
                            prior_out=None, gain_out=None, want_prior=False, want_gain=False):
    """kdn_mobius_scan with the library's internal scratch (no workspace):
    for callers that cannot allocate device memory at the call.  Returns
    (lambda, prior, gain); calls that overlap on the GPU race."""
    N, T = a.shape
    f = torch.float32
    for name, t in (('a', a), ('w', w), ('r', r), ('n', n)):
        _req(t, name, f, (N, T))
    _opt(lambda0, 'lambda0', f, (N,))
    lambda_out = _opt(lambda_out, 'lambda_out', f, (N, T)) if lambda_out is not None else \
        torch.empty_like(a)
    if prior_out is None and want_prior:
        prior_out = torch.empty_like(a)
    if gain_out is None and want_gain:
        gain_out = torch.empty_like(a)
    _opt(prior_out, 'prior_out', f, (N, T))
    _opt(gain_out, 'gain_out', f, (N, T))
    st = lib().kdn_mobius_scan_noalloc(_ptr(a), _ptr(w), _ptr(r), _ptr(n), _ptr(lambda0),
                                       float(info_scale), _ptr(lambda_out), _ptr(prior_out),
                                       _ptr(gain_out), N, T, _stream())
    _check(st, 'kdn_mobius_scan_noalloc')
    return lambda_out, prior_out, gain_out


def kdn_forward_workspace_size(variant, B, T, H, dk, dv, chunk=KDN_CHUNK_AUTO):
    return int(lib().kdn_forward_workspace_size(variant, B, T, H, dk, dv, chunk))


def _forward(variant, q, k, v, a, w, r, S0, p0, info_scale, chunk, o, S_out, p_out, workspace):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _in_dtype(q)
    _req(q, 'q', dt)
    _req(k, 'k', dt, (B, T, H, dk))
    _req(v, 'v', dt, (B, T, H, dv))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    pshape = (B, H) if variant == KDN_ISO else (B, H, dk)
    _req(w, 'w', f, (B, T, H) if variant == KDN_ISO else (B, T, H, dk))
    _opt(S0, 'S0', f, (B, H, dv, dk))
    _opt(p0, 'p0', f, pshape)
    dev = q.device
    o = _req(o, 'o', f, (B, T, H, dv)) if o is not None else \
        torch.empty((B, T, H, dv), dtype=f, device=dev)
    S_out = _req(S_out, 'S_out', f, (B, H, dv, dk)) if S_out is not None else \
        torch.empty((B, H, dv, dk), dtype=f, device=dev)
    p_out = _req(p_out, 'p_out', f, pshape) if p_out is not None else \
        torch.empty(pshape, dtype=f, device=dev)
    need = kdn_forward_workspace_size(variant, B, T, H, dk, dv, chunk)
    workspace = _workspace(need, dev, workspace)
    wsb = workspace.numel() if workspace is not None else 0
    L = lib()
    if variant == KDN_ISO:
        st = L.kdn_iso_forward(_ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w), _ptr(r),
                               _ptr(S0), _ptr(p0), _ptr(o), _ptr(S_out), _ptr(p_out), B, T, H, dk,
                               dv, float(info_scale), int(chunk), _ptr(workspace), wsb, _stream())
        _check(st, 'kdn_iso_forward')
    else:
        st = L.kdn_diag_forward(_ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                                _ptr(r), _ptr(S0), _ptr(p0), _ptr(o), _ptr(S_out), _ptr(p_out), B,
                                T, H, dk, dv, int(chunk), _ptr(workspace), wsb, _stream())
        _check(st, 'kdn_diag_forward')
    return o, S_out, p_out


def kdn_iso_forward(q, k, v, a, w, r, S0=None, p0=None, info_scale=0.0, chunk=KDN_CHUNK_AUTO,
                    o=None, S_out=None, p_out=None, workspace=None):
    """Isotropic KDN forward.  Returns (o fp32 [B,T,H,dv], S_T, p_T)."""
    return _forward(KDN_ISO, q, k, v, a, w, r, S0, p0, info_scale, chunk, o, S_out, p_out,
                    workspace)


def kdn_diag_forward(q, k, v, a, w, r, S0=None, p0=None, chunk=KDN_CHUNK_AUTO, o=None,
                     S_out=None, p_out=None, workspace=None):
    """Diagonal KDN forward.  Returns (o fp32 [B,T,H,dv], S_T, p_T [B,H,dk])."""
    return _forward(KDN_DIAG, q, k, v, a, w, r, S0, p0, 1.0, chunk, o, S_out, p_out, workspace)


def kdn_forward_varlen_workspace_size(variant, N, H, dk, dv, chunk=KDN_CHUNK_AUTO):
    return int(lib().kdn_forward_varlen_workspace_size(variant, N, H, dk, dv, chunk))


def kdn_forward_varlen(variant, q, k, v, a, w, r, cu_seqlens, S0=None, p0=None, info_scale=0.0,
                       chunk=KDN_CHUNK_AUTO, o=None, S_out=None, p_out=None, workspace=None):
    """The forward over packed sequences: q, k [total, H, dk], v [total, H, dv],
    a, r [total, H], w [total, H] (iso) or [total, H, dk] (diag), cu_seqlens
    [N + 1] int32.  Returns (o [total, H, dv], S_T [N, H, dv, dk], p_T)."""
    total, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dt = q.dtype
    _in_dtype(q)
    _req(q, 'q', dt)
    _req(k, 'k', dt, (total, H, dk))
    _req(v, 'v', dt, (total, H, dv))
    f = torch.float32
    _req(a, 'a', f, (total, H))
    _req(r, 'r', f, (total, H))
    pshape = (N, H) if variant == KDN_ISO else (N, H, dk)
    _req(w, 'w', f, (total, H) if variant == KDN_ISO else (total, H, dk))
    _req(cu_seqlens, 'cu_seqlens', torch.int32, (N + 1,))
    _opt(S0, 'S0', f, (N, H, dv, dk))
    _opt(p0, 'p0', f, pshape)
    dev = q.device
    o = _req(o, 'o', f, (total, H, dv)) if o is not None else \
        torch.empty((total, H, dv), dtype=f, device=dev)
    S_out = _req(S_out, 'S_out', f, (N, H, dv, dk)) if S_out is not None else \
        torch.empty((N, H, dv, dk), dtype=f, device=dev)
    p_out = _req(p_out, 'p_out', f, pshape) if p_out is not None else \
        torch.empty(pshape, dtype=f, device=dev)
    need = kdn_forward_varlen_workspace_size(variant, N, H, dk, dv, chunk)
    workspace = _workspace(need, dev, workspace)
    st = lib().kdn_forward_varlen(variant, _ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a),
                                  _ptr(w), _ptr(r), _ptr(cu_seqlens), _ptr(S0), _ptr(p0), _ptr(o),
                                  _ptr(S_out), _ptr(p_out), N, total, H, dk, dv,
                                  float(info_scale), int(chunk), _ptr(workspace),
                                  workspace.numel(), _stream())
    _check(st, 'kdn_forward_varlen')
    return o, S_out, p_out


def _req_host(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f'{name} must be a host (CPU) tensor')
    if not t.is_contiguous():
        raise ValueError(f'{name} must be contiguous')
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f'{name} must be {dtype}, got {t.dtype}')
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f'{name} must have shape {tuple(shape)}, got {tuple(t.shape)}')
    return t


def kdn_forward_host_workspace_size(variant, B, T, H, dk, dv, in_dtype=KDN_BF16,
                                    chunk=KDN_CHUNK_AUTO, slice_b=0):
    return int(lib().kdn_forward_host_workspace_size(variant, B, T, H, dk, dv, in_dtype, chunk,
                                                     slice_b))


def kdn_forward_host(variant, q, k, v, a, w, r, S0=None, p0=None, info_scale=0.0,
                     chunk=KDN_CHUNK_AUTO, slice_b=0, o=None, S_out=None, p_out=None,
                     workspace=None, device=None):
    """The forward with host tensors (pinned for overlap); outputs are host
    tensors, valid once the current stream has been synchronised.  Returns
    (o, S_T, p_T)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _in_dtype(q)
    _req_host(q, 'q', dt)
    _req_host(k, 'k', dt, (B, T, H, dk))
    _req_host(v, 'v', dt, (B, T, H, dv))
    f = torch.float32
    _req_host(a, 'a', f, (B, T, H))
    _req_host(r, 'r', f, (B, T, H))
    pshape = (B, H) if variant == KDN_ISO else (B, H, dk)
    _req_host(w, 'w', f, (B, T, H) if variant == KDN_ISO else (B, T, H, dk))
    if S0 is not None:
        _req_host(S0, 'S0', f, (B, H, dv, dk))
    if p0 is not None:
        _req_host(p0, 'p0', f, pshape)
    o = _req_host(o, 'o', f, (B, T, H, dv)) if o is not None else \
        torch.empty((B, T, H, dv), dtype=f).pin_memory()
    S_out = _req_host(S_out, 'S_out', f, (B, H, dv, dk)) if S_out is not None else \
        torch.empty((B, H, dv, dk), dtype=f).pin_memory()
    p_out = _req_host(p_out, 'p_out', f, pshape) if p_out is not None else \
        torch.empty(pshape, dtype=f).pin_memory()
    need = kdn_forward_host_workspace_size(variant, B, T, H, dk, dv, _in_dtype(q), chunk, slice_b)
    dev = device if device is not None else torch.device('cuda', torch.cuda.current_device())
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _req(workspace, 'workspace', torch.uint8)
    st = lib().kdn_forward_host(variant, _ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a),
                                _ptr(w), _ptr(r), _ptr(S0), _ptr(p0), _ptr(o), _ptr(S_out),
                                _ptr(p_out), B, T, H, dk, dv, float(info_scale), int(chunk),
                                int(slice_b), _ptr(workspace), workspace.numel(), _stream())
    _check(st, 'kdn_forward_host')
    return o, S_out, p_out


def kdn_decode_step(variant, q, k, v, a, w, r, S, p, o=None, info_scale=0.0):
    """One decode step; S and p are updated in place.  Returns o [B,H,dv]."""
    var = KDN_DIAG if variant in ('diag', KDN_DIAG) else KDN_ISO
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _req(q, 'q', dt)
    _req(k, 'k', dt, (B, H, dk))
    _req(v, 'v', dt, (B, H, dv))
    f = torch.float32
    _req(a, 'a', f, (B, H))
    _req(r, 'r', f, (B, H))
    _req(w, 'w', f, (B, H) if var == KDN_ISO else (B, H, dk))
    _req(S, 'S', f, (B, H, dv, dk))
    _req(p, 'p', f, (B, H) if var == KDN_ISO else (B, H, dk))
    o = _req(o, 'o', f, (B, H, dv)) if o is not None else \
        torch.empty((B, H, dv), dtype=f, device=q.device)
    st = lib().kdn_decode_step(var, _ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                               _ptr(r), _ptr(S), _ptr(p), _ptr(o), B, H, dk, dv,
                               float(info_scale), _stream())
    _check(st, 'kdn_decode_step')
    return o


def kdn_exact_forward(variant, q, k, v, a, w, r, S0=None, P0=None, o=None, S_out=None,
                      P_out=None):
    """The dense (full-covariance) Kalman filter: q, k [B,T,H,dk], v [B,T,H,dv],
    a, r [B,T,H], w [B,T,H] (iso: W = w I) or [B,T,H,dk] (diag: W = diag(w)).
    Returns (o [B,T,H,dv], S_T [B,H,dv,dk], P_T [B,H,dk,dk])."""
    var = KDN_DIAG if variant in ('diag', KDN_DIAG) else KDN_ISO
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _in_dtype(q)
    _req(q, 'q', dt)
    _req(k, 'k', dt, (B, T, H, dk))
    _req(v, 'v', dt, (B, T, H, dv))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    _req(w, 'w', f, (B, T, H) if var == KDN_ISO else (B, T, H, dk))
    _opt(S0, 'S0', f, (B, H, dv, dk))
    _opt(P0, 'P0', f, (B, H, dk, dk))
    dev = q.device
    o = _req(o, 'o', f, (B, T, H, dv)) if o is not None else \
        torch.empty((B, T, H, dv), dtype=f, device=dev)
    S_out = _req(S_out, 'S_out', f, (B, H, dv, dk)) if S_out is not None else \
        torch.empty((B, H, dv, dk), dtype=f, device=dev)
    P_out = _req(P_out, 'P_out', f, (B, H, dk, dk)) if P_out is not None else \
        torch.empty((B, H, dk, dk), dtype=f, device=dev)
    st = lib().kdn_exact_forward(var, _ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                                 _ptr(r), _ptr(S0), _ptr(P0), _ptr(o), _ptr(S_out), _ptr(P_out),
                                 B, T, H, dk, dv, _stream())
    _check(st, 'kdn_exact_forward')
    return o, S_out, P_out


def kdn_backward_workspace_size(variant, B, T, H, dk, dv):
    return int(lib().kdn_backward_workspace_size(variant, B, T, H, dk, dv))


def kdn_backward(variant, q, k, v, a, w, r, dO, S0=None, p0=None, dS_T=None, dp_T=None,
                 info_scale=0.0, workspace=None):
    """Backward of the layer forward: returns a dict of the gradients
    q, k, v, a, w, r, S0, p0 (fp32, shaped like the inputs) of the loss whose
    gradients with respect to o, S_T and p_T are dO, dS_T, dp_T."""
    var = KDN_DIAG if variant in ('diag', KDN_DIAG) else KDN_ISO
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _in_dtype(q)
    _req(q, 'q', dt)
    _req(k, 'k', dt, (B, T, H, dk))
    _req(v, 'v', dt, (B, T, H, dv))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    wshape = (B, T, H) if var == KDN_ISO else (B, T, H, dk)
    pshape = (B, H) if var == KDN_ISO else (B, H, dk)
    _req(w, 'w', f, wshape)
    _req(dO, 'dO', f, (B, T, H, dv))
    _opt(S0, 'S0', f, (B, H, dv, dk))
    _opt(p0, 'p0', f, pshape)
    _opt(dS_T, 'dS_T', f, (B, H, dv, dk))
    _opt(dp_T, 'dp_T', f, pshape)
    dev = q.device
    g = dict(q=torch.empty((B, T, H, dk), dtype=f, device=dev),
             k=torch.empty((B, T, H, dk), dtype=f, device=dev),
             v=torch.empty((B, T, H, dv), dtype=f, device=dev),
             a=torch.empty((B, T, H), dtype=f, device=dev),
             w=torch.empty(wshape, dtype=f, device=dev),
             r=torch.empty((B, T, H), dtype=f, device=dev),
             S0=torch.empty((B, H, dv, dk), dtype=f, device=dev),
             p0=torch.empty(pshape, dtype=f, device=dev))
    need = kdn_backward_workspace_size(var, B, T, H, dk, dv)
    workspace = _workspace(need, dev, workspace)
    st = lib().kdn_backward(var, _ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                            _ptr(r), _ptr(S0), _ptr(p0), _ptr(dO), _ptr(dS_T), _ptr(dp_T),
                            _ptr(g['q']), _ptr(g['k']), _ptr(g['v']), _ptr(g['a']), _ptr(g['w']),
                            _ptr(g['r']), _ptr(g['S0']), _ptr(g['p0']), B, T, H, dk, dv,
                            float(info_scale), _ptr(workspace), workspace.numel(), _stream())
    _check(st, 'kdn_backward')
    return g


def kdn_kla_workspace_size(B, T, H, dk, dv):
    return int(lib().kdn_kla_workspace_size(B, T, H, dk, dv))


def kdn_kla_forward(q, k, v, a, w, r, S0=None, lam0=None, o=None, S_out=None, lam_out=None,
                    workspace=None, recurrent=False):
    """The information-form diagonal filter (KLA): q, k [B,T,H,dk], v [B,T,H,dv],
    a, r [B,T,H], w [B,T,H,dk].  Returns (o [B,T,H,dv], S_T [B,H,dv,dk],
    lam_T [B,H,dk]) -- lam is the precision.  By default this is
    kdn_kla_forward_ws (the chunked tensor-core engine at dk = dv = 128 with
    bf16 inputs, the token-recurrent kernel otherwise); recurrent=True calls
    kdn_kla_forward, the token-recurrent kernel for every shape."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _in_dtype(q)
    _req(q, 'q', dt)
    _req(k, 'k', dt, (B, T, H, dk))
    _req(v, 'v', dt, (B, T, H, dv))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    _req(w, 'w', f, (B, T, H, dk))
    _opt(S0, 'S0', f, (B, H, dv, dk))
    _opt(lam0, 'lam0', f, (B, H, dk))
    dev = q.device
    o = _req(o, 'o', f, (B, T, H, dv)) if o is not None else \
        torch.empty((B, T, H, dv), dtype=f, device=dev)
    S_out = _req(S_out, 'S_out', f, (B, H, dv, dk)) if S_out is not None else \
        torch.empty((B, H, dv, dk), dtype=f, device=dev)
    lam_out = _req(lam_out, 'lam_out', f, (B, H, dk)) if lam_out is not None else \
        torch.empty((B, H, dk), dtype=f, device=dev)
    if recurrent:
        st = lib().kdn_kla_forward(_ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                                   _ptr(r), _ptr(S0), _ptr(lam0), _ptr(o), _ptr(S_out),
                                   _ptr(lam_out), B, T, H, dk, dv, _stream())
        _check(st, 'kdn_kla_forward')
        return o, S_out, lam_out
    need = kdn_kla_workspace_size(B, T, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = lib().kdn_kla_forward_ws(_ptr(q), _ptr(k), _ptr(v), _in_dtype(q), _ptr(a), _ptr(w),
                                  _ptr(r), _ptr(S0), _ptr(lam0), _ptr(o), _ptr(S_out),
                                  _ptr(lam_out), B, T, H, dk, dv, _ptr(workspace),
                                  workspace.numel(), _stream())
    _check(st, 'kdn_kla_forward_ws')
    return o, S_out, lam_out


# ------------------------------------------ linear recurrence, norm, 8 bits
# These calls run on the device of their tensors (which may differ from the
# current one) and on that device's current stream.

_CODE = {torch.float32: KDN_F32, torch.bfloat16: KDN_BF16, torch.float8_e4m3fn: KDN_E4M3}


class _NoQuick:
    """Stands in for a _kdn_quick.so that was not built."""
    scan_step = scan_forward = scan_backward = norm_forward = norm_backward = quantize = matmul = \
        staticmethod(lambda *args: None)


_quick = None


def _load_quick():
    """The calls below in one C++ function each (csrc/quick_binding.cpp), which
    gives None where anything is out of the ordinary; then the code here runs."""
    global _quick
    lib()
    try:
        from . import _kdn_quick
        built = getattr(_kdn_quick, 'torch_version', 'of another build')
        why = None if built == torch.__version__.partition('+')[0] else \
            f'it was built against torch {built}'
    except ImportError as e:
        why = e
    if why is None:
        _quick = _kdn_quick
    else:
        warnings.warn(f'_kdn_quick.so is not used ({why}): small calls take about twice as long. '
                      '`python -m kalman_filter_linear_b200.build` builds it', RuntimeWarning,
                      stacklevel=3)
        _quick = _NoQuick
    return _quick


def _float_code(t, name):
    if t.dtype != torch.float32 and t.dtype != torch.bfloat16:
        raise TypeError(f'{name} must be bfloat16 or float32, got {t.dtype}')
    return _CODE[t.dtype]


def _arg(t, name, dtype, shape, dev):
    """The data pointer of a checked tensor (None for a missing one)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.device == dev and t.dtype is dtype and \
            t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f'{name} must be a CUDA tensor')
    if t.dtype != dtype:
        raise TypeError(f'{name} must be {dtype}, got {t.dtype}')
    if t.shape != shape:
        raise ValueError(f'{name} must have shape {tuple(shape)}, got {tuple(t.shape)}')
    if t.device != dev:
        raise ValueError(f'{name} must be on {dev}, got {t.device}')
    raise ValueError(f'{name} must be contiguous')


def _cuda_tensor(t, name, ndim):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f'{name} must be a CUDA tensor')
    if t.dim() not in ndim:
        raise ValueError(f'{name} must have {" or ".join(map(str, ndim))} dimensions, '
                         f'got {t.dim()}')
    return t.device


def _call(fn, dev, *args):
    """Call an entry point with `dev` current, on its current stream.  (The two
    torch._C calls are what torch.cuda.current_device and current_stream end in;
    those cost 3 us a call, as much as the launch.)"""
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(dev):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _ws_arg(workspace, need, dev):
    """(tensor, pointer, bytes) of a workspace of at least `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or \
            not workspace.is_contiguous():
        raise TypeError(f'workspace must be a contiguous CUDA tensor on {dev}')
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=1024)
def kdn_linear_scan_workspace_size(B, T, D):
    return int(lib().kdn_linear_scan_workspace_size(B, T, D))


_status_words = {}


def _scan_ws_arg(workspace, need, dev):
    """_ws_arg; a call that needs no more than a status word, and whose caller
    gave no place for one, shares the device's word that nobody reads."""
    if workspace is None and 0 < need <= 256:
        workspace = _status_words.get(dev)
        if workspace is None:
            workspace = _status_words[dev] = torch.empty(256, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), 256
    return _ws_arg(workspace, need, dev)


def _f32_empty(like, shape, near):
    """A new fp32 tensor, like the checked tensor `like` if there is one (which is
    quicker), else on `near`'s device."""
    return near.new_empty(shape, dtype=torch.float32) if like is None else torch.empty_like(like)


def _scan_dims(a, cu_seqlens):
    dev = _cuda_tensor(a, 'a', (3,) if cu_seqlens is None else (2,))
    if cu_seqlens is None:
        B, T, D = a.shape
        return dev, B, T, D, kdn_linear_scan_workspace_size(B, T, D)
    T, D = a.shape
    if not isinstance(cu_seqlens, torch.Tensor) or not cu_seqlens.is_cuda:
        raise TypeError('cu_seqlens must be a CUDA tensor')
    return dev, cu_seqlens.numel() - 1, T, D, kdn_linear_scan_workspace_size(1, T, D)


def kdn_linear_scan_forward(a, x, b=None, h0=None, cu_seqlens=None, y=None, h_out=None,
                            workspace=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + b_t x_t: a, b, x
    [B, T, D], or [T, D] with cu_seqlens [B + 1] int32 (packed sequences);
    a and b share a dtype (fp32 or bf16), h0 [B, D] fp32.  Returns (y like x,
    h_T [B, D] fp32).  With cu_seqlens, the rows of y behind the last sequence
    are left as they were.  Offsets out of order and a wait that gave up are told
    by kdn_read_workspace_status(workspace), so only where a workspace is given;
    without one such a call returns unspecified values."""
    if workspace is None:
        r = (_quick or _load_quick()).scan_forward(a, x, b, h0, cu_seqlens, y, h_out)
        if r is not None:
            return r
    dev, B, T, D, need = _scan_dims(a, cu_seqlens)
    f, shape, ends = torch.float32, a.shape, (B, D)
    gate = _float_code(a, 'a')
    xt = _float_code(x, 'x')
    pa, pb, px = a.data_ptr(), _arg(b, 'b', a.dtype, shape, dev), _arg(x, 'x', x.dtype, shape, dev)
    if not a.is_contiguous():
        raise ValueError('a must be contiguous')
    p0 = _arg(h0, 'h0', f, ends, dev)
    pc = _arg(cu_seqlens, 'cu_seqlens', torch.int32, (B + 1,), dev)
    if y is None:
        y = torch.empty_like(x)
    if h_out is None:
        h_out = _f32_empty(h0, ends, a)
    workspace, pw, nw = _scan_ws_arg(workspace, need, dev)
    st = _call(lib().kdn_linear_scan_forward, dev, pa, pb, gate, px, xt, p0, pc,
               _arg(y, 'y', x.dtype, shape, dev), _arg(h_out, 'h_out', f, ends, dev), B, T, D, pw,
               nw)
    _check(st, 'kdn_linear_scan_forward')
    return y, h_out


def kdn_linear_scan_backward(a, x, y, dy, b=None, h0=None, dh_T=None, cu_seqlens=None, da=None,
                             dx=None, db=None, dh0=None, workspace=None):
    """The gradients of kdn_linear_scan_forward, given its output y, dy like y
    and dh_T [B, D] fp32 (or None): a dict of a, x, h0 (fp32) and, when b is
    given, b.  x is read only with b, and may be None without.  The status is in a
    given workspace, as the forward's."""
    if workspace is None:
        r = (_quick or _load_quick()).scan_backward(a, x, y, dy, b, h0, dh_T, cu_seqlens, da, dx, db,
                                                    dh0)
        if r is not None:
            return r
    dev, B, T, D, need = _scan_dims(a, cu_seqlens)
    f, shape, ends = torch.float32, a.shape, (B, D)
    gate = _float_code(a, 'a')
    yt = _float_code(y, 'y')
    if b is not None and x is None:
        raise ValueError('x is needed for the gradient of b')
    if not a.is_contiguous():
        raise ValueError('a must be contiguous')
    pa, pb = a.data_ptr(), _arg(b, 'b', a.dtype, shape, dev)
    px, py = _arg(x, 'x', y.dtype, shape, dev), _arg(y, 'y', y.dtype, shape, dev)
    pdy = _arg(dy, 'dy', y.dtype, shape, dev)
    p0, pT = _arg(h0, 'h0', f, ends, dev), _arg(dh_T, 'dh_T', f, ends, dev)
    pc = _arg(cu_seqlens, 'cu_seqlens', torch.int32, (B + 1,), dev)
    da = torch.empty_like(a) if da is None else da
    dx = torch.empty_like(y) if dx is None else dx
    if b is not None and db is None:
        db = torch.empty_like(b)
    dh0 = _f32_empty(h0, ends, a) if dh0 is None else dh0
    workspace, pw, nw = _scan_ws_arg(workspace, need, dev)
    st = _call(lib().kdn_linear_scan_backward, dev, pa, pb, gate, px, py, pdy, yt, p0, pT, pc,
               _arg(da, 'da', a.dtype, shape, dev),
               _arg(db, 'db', a.dtype, shape, dev) if b is not None else None,
               _arg(dx, 'dx', y.dtype, shape, dev), _arg(dh0, 'dh0', f, ends, dev), B, T, D, pw,
               nw)
    _check(st, 'kdn_linear_scan_backward')
    g = dict(a=da, x=dx, h0=dh0)
    if b is not None:
        g['b'] = db
    return g


def kdn_linear_scan_step(a, x, h, b=None, y=None):
    """One step of the recurrence: a, b, x [B, D], h [B, D] fp32 updated in
    place.  Returns y like x."""
    r = (_quick or _load_quick()).scan_step(a, x, h, b, y)
    if r is not None:
        return r
    dev = _cuda_tensor(a, 'a', (2,))
    shape = a.shape
    gate, xt = _float_code(a, 'a'), _float_code(x, 'x')
    if y is None:
        y = torch.empty_like(x)
    st = _call(lib().kdn_linear_scan_step, dev, _arg(a, 'a', a.dtype, shape, dev),
               _arg(b, 'b', a.dtype, shape, dev), gate, _arg(x, 'x', x.dtype, shape, dev), xt,
               _arg(h, 'h', torch.float32, shape, dev), _arg(y, 'y', x.dtype, shape, dev),
               shape[0], shape[1])
    _check(st, 'kdn_linear_scan_step')
    return y


def _fp8_empty(rows, cols, near):
    """An e4m3 matrix on `near`'s device whose rows start on 16-byte boundaries."""
    ld = (cols + 15) // 16 * 16
    q = near.new_empty((rows, ld), dtype=torch.float8_e4m3fn)
    return q if ld == cols else q[:, :cols]


def _fp8_arg(q, name, rows, cols, dev):
    """(pointer, row distance in bytes) of an e4m3 matrix."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError(f'{name} must be a CUDA tensor')
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f'{name} must be torch.float8_e4m3fn, got {q.dtype}')
    if q.shape != (rows, cols):
        raise ValueError(f'{name} must have shape {(rows, cols)}, got {tuple(q.shape)}')
    if q.device != dev:
        raise ValueError(f'{name} must be on {dev}, got {q.device}')
    if rows == 0 or cols == 0:  # (nothing is read or written)
        return None, 0
    ld = q.stride(0) if rows > 1 else (cols + 15) // 16 * 16
    if (cols > 1 and q.stride(1) != 1) or ld % 16 or ld < cols:
        raise ValueError(f'the rows of {name} must be contiguous and a multiple of 16 bytes apart '
                         f'(kdn_fp8_quantize lays them out so), got strides {q.stride()}')
    return q.data_ptr(), ld


def kdn_rmsnorm_forward(x, weight, residual=None, eps=1e-6, out_dtype=torch.bfloat16, y=None,
                        scale=None, h=None):
    """Residual addition and RMS norm over the last dimension: x [rows, D] or
    [..., D], residual like x (its own dtype), weight [D] fp32.  Returns
    (y, scale, h): y in out_dtype (bfloat16, float32 or float8_e4m3fn), scale
    [rows, ceil(D / 128)] for e4m3 else None, and h = x + residual in the
    residual's dtype (None without a residual).  An e4m3 y is two-dimensional,
    its rows on 16-byte boundaries."""
    r = (_quick or _load_quick()).norm_forward(x, weight, residual, eps, _CODE.get(out_dtype, -1), y,
                                               scale, h)
    if r is not None:
        return r
    dev = _cuda_tensor(x, 'x', range(1, 9))
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    xt = _float_code(x, 'x')
    if out_dtype not in _CODE:
        raise TypeError(f'out_dtype must be bfloat16, float32 or float8_e4m3fn, got {out_dtype}')
    px, pw = _arg(x, 'x', x.dtype, x.shape, dev), _arg(weight, 'weight', torch.float32, (D,), dev)
    if pw is None:
        raise TypeError('weight must be a CUDA tensor')
    rt, pr, ph = KDN_F32, None, None
    if residual is not None:
        rt, pr = _float_code(residual, 'residual'), _arg(residual, 'residual', residual.dtype,
                                                         x.shape, dev)
        h = torch.empty_like(residual) if h is None else h
        ph = _arg(h, 'h', residual.dtype, x.shape, dev)
    elif h is not None:
        raise ValueError('h is an output only with a residual')
    ld, ps = 0, None
    if out_dtype == torch.float8_e4m3fn:
        y = _fp8_empty(rows, D, x) if y is None else y
        py, ld = _fp8_arg(y, 'y', rows, D, dev)
        blocks = (rows, (D + 127) // 128)
        scale = x.new_empty(blocks, dtype=torch.float32) if scale is None else scale
        ps = _arg(scale, 'scale', torch.float32, blocks, dev)
    else:
        if scale is not None:
            raise ValueError('scale is an output only for float8_e4m3fn')
        if y is None:
            y = torch.empty_like(x) if out_dtype is x.dtype else x.new_empty(x.shape, dtype=out_dtype)
        py = _arg(y, 'y', out_dtype, x.shape, dev)
    if rows:
        st = _call(lib().kdn_rmsnorm_forward, dev, px, xt, pr, rt, pw, ph, py, _CODE[out_dtype],
                   ld, ps, rows, D, eps)
        _check(st, 'kdn_rmsnorm_forward')
    return y, scale, h


@functools.lru_cache(maxsize=1024)
def kdn_rmsnorm_backward_workspace_size(rows, D):
    return int(lib().kdn_rmsnorm_backward_workspace_size(rows, D))


def kdn_rmsnorm_backward(h, weight, dy, dh=None, eps=1e-6, x_dtype=None, want_residual=None,
                         dx=None, dresidual=None, dweight=None, workspace=None):
    """The gradients of kdn_rmsnorm_forward: h its h (x without a residual),
    dy like h in bfloat16 or float32, dh the gradient that reaches h from its
    other use (h's dtype, or None).  Returns a dict of x (in x_dtype, h's by
    default), weight (fp32) and residual (h's dtype; by default when dh is
    given, else None)."""
    if workspace is None:
        want = dresidual is not None or (dh is not None if want_residual is None
                                         else bool(want_residual))
        r = (_quick or _load_quick()).norm_backward(
            h, weight, dy, dh, eps, -1 if x_dtype is None else _CODE.get(x_dtype, 9), want, dx,
            dresidual, dweight)
        if r is not None:
            return r
    dev = _cuda_tensor(h, 'h', range(1, 9))
    D = h.shape[-1]
    rows = h.numel() // D if D else 0
    x_dtype = h.dtype if x_dtype is None else x_dtype
    ht, yt = _float_code(h, 'h'), _float_code(dy, 'dy')
    if x_dtype != torch.float32 and x_dtype != torch.bfloat16:
        raise TypeError(f'x_dtype must be bfloat16 or float32, got {x_dtype}')
    if want_residual is None:
        want_residual = dh is not None or dresidual is not None
    f, shape = torch.float32, h.shape
    ph, pw = _arg(h, 'h', h.dtype, shape, dev), _arg(weight, 'weight', f, (D,), dev)
    pdy, pdh = _arg(dy, 'dy', dy.dtype, shape, dev), _arg(dh, 'dh', h.dtype, shape, dev)
    if dx is None:
        dx = torch.empty_like(h) if x_dtype is h.dtype else h.new_empty(shape, dtype=x_dtype)
    if want_residual and dresidual is None:
        dresidual = torch.empty_like(h)
    dweight = torch.empty_like(weight) if dweight is None else dweight
    px, pr = _arg(dx, 'dx', x_dtype, shape, dev), _arg(dresidual, 'dresidual', h.dtype, shape, dev)
    pdw = _arg(dweight, 'dweight', f, (D,), dev)
    if rows == 0:
        dweight.zero_()
    else:
        workspace, pws, nws = _ws_arg(workspace, kdn_rmsnorm_backward_workspace_size(rows, D), dev)
        st = _call(lib().kdn_rmsnorm_backward, dev, ph, ht, pw, pdy, yt, pdh, px, _CODE[x_dtype],
                   pr, pdw, rows, D, eps, pws, nws)
        _check(st, 'kdn_rmsnorm_backward')
    return dict(x=dx, weight=dweight, residual=dresidual)


def kdn_fp8_quantize(x, tile=False, transpose=False, q=None, scale=None):
    """x [rows, cols] (bfloat16 or float32) in e4m3 with fp32 scales: one for
    each 128 of an output row, or with tile=True for each 128 x 128 tile;
    transpose=True quantises x's transpose.  Returns (q [R, C], its rows on
    16-byte boundaries; scale [R or ceil(R / 128), ceil(C / 128)]).  In a given q
    the bytes between a row's end and the next multiple of 16 are overwritten,
    but nothing behind the last row."""
    r = (_quick or _load_quick()).quantize(x, tile, transpose, q, scale)
    if r is not None:
        return r
    dev = _cuda_tensor(x, 'x', (2,))
    rows, cols = x.shape
    xt = _float_code(x, 'x')
    px = _arg(x, 'x', x.dtype, x.shape, dev)
    R, C = (cols, rows) if transpose else (rows, cols)
    blocks = ((R + 127) // 128 if tile else R, (C + 127) // 128)
    q = _fp8_empty(R, C, x) if q is None else q
    scale = x.new_empty(blocks, dtype=torch.float32) if scale is None else scale
    pq, ld = _fp8_arg(q, 'q', R, C, dev)
    ps = _arg(scale, 'scale', torch.float32, blocks, dev)
    if rows and cols:
        st = _call(lib().kdn_fp8_quantize, dev, px, xt, rows, cols, int(tile), int(transpose), pq,
                   ld, ps)
        _check(st, 'kdn_fp8_quantize')
    return q, scale


def kdn_fp8_matmul(x, x_scale, w, w_scale, out_dtype=torch.bfloat16, out=None, status=None):
    """The 8-bit projection x w^T: x [M, K] and w [N, K] in e4m3 (rows on
    16-byte boundaries, as kdn_fp8_quantize lays them out), x_scale
    [M, ceil(K / 128)], w_scale [ceil(N / 128), ceil(K / 128)] (128 x 128
    tiles) or [N, ceil(K / 128)], fp32.  Returns [M, N] in out_dtype (bfloat16
    or float32): zeros for K = 0.  status: one zeroed int32 word that a timed-out
    wait sets (kdn_read_workspace_status); without one it is not told."""
    r = (_quick or _load_quick()).matmul(x, x_scale, w, w_scale, _CODE.get(out_dtype, -1), out, status)
    if r is not None:
        return r
    dev = _cuda_tensor(x, 'x', (2,))
    _cuda_tensor(w, 'w', (2,))
    M, K = x.shape
    N = w.shape[0]
    px, ldx = _fp8_arg(x, 'x', M, K, dev)
    pw, ldw = _fp8_arg(w, 'w', N, K, dev)
    kb = (K + 127) // 128
    psx = _arg(x_scale, 'x_scale', torch.float32, (M, kb), dev)
    _cuda_tensor(w_scale, 'w_scale', (2,))
    tile = w_scale.shape[0] != N  # (the two forms agree for N = 1)
    psw = _arg(w_scale, 'w_scale', torch.float32, ((N + 127) // 128 if tile else N, kb), dev)
    if psx is None:
        raise TypeError('x_scale must be a CUDA tensor')
    if out_dtype != torch.float32 and out_dtype != torch.bfloat16:
        raise TypeError(f'out_dtype must be bfloat16 or float32, got {out_dtype}')
    out = x.new_empty((M, N), dtype=out_dtype) if out is None else out
    po = _arg(out, 'out', out_dtype, (M, N), dev)
    pst = _arg(status, 'status', torch.int32, (1,), dev)
    if K == 0:  # a sum over nothing
        out.zero_()
    elif M and N:
        st = _call(lib().kdn_fp8_matmul, dev, px, ldx, psx, pw, ldw, psw, int(tile), po,
                   _CODE[out_dtype], M, N, K, pst)
        _check(st, 'kdn_fp8_matmul')
    return out


def kdn_read_workspace_status(workspace):
    """Synchronise the current stream and return the workspace's status code."""
    return int(lib().kdn_read_workspace_status(_ptr(workspace), workspace.numel(), _stream()))


def kdn_testing_mobius_scan_unpublished_tile(a, w, r, n, silent_tile, info_scale=1.0):
    """Fault-injection hook: the scan with one tile that never publishes."""
    N, T = a.shape
    out = torch.empty_like(a)
    need = kdn_mobius_scan_workspace_size(N, T)
    ws = torch.empty(need, dtype=torch.uint8, device=a.device)
    st = lib().kdn_testing_mobius_scan_unpublished_tile(
        _ptr(a), _ptr(w), _ptr(r), _ptr(n), None, float(info_scale), _ptr(out), N, T, _ptr(ws),
        need, int(silent_tile), _stream())
    _check(st, 'kdn_testing_mobius_scan_unpublished_tile')
    return out, ws


def kdn_testing_forward_skip_v_copy(variant, q, k, v, a, w, r, skip_chunk, workspace):
    """Fault-injection hook: the chunked forward (d = 128, bf16) with one V
    copy left out, so a bounded wait gives up.  Returns (o, S_T, p_T); the
    status is in the workspace."""
    B, T, H, d = q.shape
    for t, n in ((q, 'q'), (k, 'k'), (v, 'v')):
        _req(t, n, torch.bfloat16, (B, T, H, d))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    _req(w, 'w', f, (B, T, H) if variant == KDN_ISO else (B, T, H, d))
    _req(workspace, 'workspace', torch.uint8)
    o = torch.empty((B, T, H, d), dtype=f, device=q.device)
    S = torch.empty((B, H, d, d), dtype=f, device=q.device)
    p = torch.empty((B, H) if variant == KDN_ISO else (B, H, d), dtype=f, device=q.device)
    st = lib().kdn_testing_forward_skip_v_copy(variant, _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                               _ptr(w), _ptr(r), _ptr(o), _ptr(S), _ptr(p), B, T,
                                               H, int(skip_chunk), _ptr(workspace),
                                               workspace.numel(), _stream())
    _check(st, 'kdn_testing_forward_skip_v_copy')
    return o, S, p


def kdn_testing_kla_skip_v_copy(q, k, v, a, w, r, skip_chunk, workspace):
    """Fault-injection hook: the KLA engine (d = 128, bf16) with one V copy
    left out, so a bounded wait gives up.  Returns (o, S_T, lam_T); the status
    is in the workspace."""
    B, T, H, d = q.shape
    for t, n in ((q, 'q'), (k, 'k'), (v, 'v')):
        _req(t, n, torch.bfloat16, (B, T, H, d))
    f = torch.float32
    _req(a, 'a', f, (B, T, H))
    _req(r, 'r', f, (B, T, H))
    _req(w, 'w', f, (B, T, H, d))
    _req(workspace, 'workspace', torch.uint8)
    o = torch.empty((B, T, H, d), dtype=f, device=q.device)
    S = torch.empty((B, H, d, d), dtype=f, device=q.device)
    lam = torch.empty((B, H, d), dtype=f, device=q.device)
    st = lib().kdn_testing_kla_skip_v_copy(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(w), _ptr(r),
                                           _ptr(o), _ptr(S), _ptr(lam), B, T, H, int(skip_chunk),
                                           _ptr(workspace), workspace.numel(), _stream())
    _check(st, 'kdn_testing_kla_skip_v_copy')
    return o, S, lam


def kdn_testing_linear_scan_skip_copy(a, x, skip_tile, workspace):
    """Fault-injection hook: the streamed recurrence (fp32) with one copy of the
    first block left out.  Returns (y, h_T); the status is in the workspace."""
    B, T, D = a.shape
    for t, n in ((a, 'a'), (x, 'x')):
        _req(t, n, torch.float32, (B, T, D))
    _req(workspace, 'workspace', torch.uint8)
    y, h = torch.empty_like(x), torch.empty((B, D), dtype=torch.float32, device=x.device)
    st = lib().kdn_testing_linear_scan_skip_copy(_ptr(a), _ptr(x), _ptr(y), _ptr(h), B, T, D,
                                                 int(skip_tile), _ptr(workspace),
                                                 workspace.numel(), _stream())
    _check(st, 'kdn_testing_linear_scan_skip_copy')
    return y, h


def kdn_testing_fp8_matmul_skip_copy(x, x_scale, w, w_scale, skip_block, status):
    """Fault-injection hook: kdn_fp8_matmul with the first block's copies of one
    block along K left out.  Returns the product (fp32); `status` is one zeroed
    int32 word."""
    (M, K), N = x.shape, w.shape[0]
    px, ldx = _fp8_arg(x, 'x', M, K, x.device)
    pw, ldw = _fp8_arg(w, 'w', N, K, x.device)
    _req(status, 'status', torch.int32, (1,))
    out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    st = lib().kdn_testing_fp8_matmul_skip_copy(
        px, ldx, _ptr(x_scale), pw, ldw, _ptr(w_scale), int(w_scale.shape[0] != N), _ptr(out),
        KDN_F32, M, N, K, int(skip_block), _ptr(status), _stream())
    _check(st, 'kdn_testing_fp8_matmul_skip_copy')
    return out
