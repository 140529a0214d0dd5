"""The residual RMS norm (kdn_rmsnorm_*) against the fp64 oracle (needs a
B200).

Tolerances.  All of the norm is fp32.  A sum of squares goes through at most 64
additions in a thread and 13 between threads, and its terms are positive, so it
is within 78 roundings of 2^-24; half of that reaches the inverse root, which
adds 4 of its own (division, eps, root), and two products follow: 64 in all is
an upper bound for y before its own rounding.  The backward's second sum adds
as many, so 160 on the sum of absolute values; a column sum adds one rounding
for each row of a block and each block, rows / 592 + 592 / 8 + 16.
e4m3: a code may be that of either end of the interval that value / scale lies
in.  Half steps of the output types: bf16 2^-8, fp32 2^-24.
"""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import fp8_ref, rmsnorm_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {F32: U, BF16: 2.0 ** -8}


def _inputs(rows, D, xt, rt, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, D, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(xt)
    res = None if rt is None else torch.randn(rows, D, generator=g).to(rt).cuda()
    w = torch.rand(D, generator=g) + 0.5
    return x.cuda(), res, w.cuda()


def _check_codes(q, s, want, rel):
    """Codes and scales of values known to `rel` relative error."""
    s, q = f64(s), f64(q.float())
    ref_s = fp8_ref.scales(want)
    assert (np.abs(s - ref_s) <= (rel + 2 * U) * ref_s).all()
    # value / scale: the value's and the scale's error, and three roundings
    v = want / fp8_ref.spread(ref_s, *want.shape)
    d = 2 * rel + 8 * U
    lo, hi = fp8_ref.e4m3(v - np.abs(v) * d), fp8_ref.e4m3(v + np.abs(v) * d)
    assert ((q >= lo) & (q <= hi)).all(), np.argwhere(~((q >= lo) & (q <= hi)))[:3]


SIZES = [(1, 1), (3, 7), (5, 128), (300, 129), (2, 256), (33, 264), (9, 1000), (4, 2048),
         (7, 2056), (2, 4100), (3, 8192), (2, 16384), (700, 65)]


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("xt,rt,out", [(F32, BF16, E4M3), (BF16, None, BF16), (F32, F32, F32),
                                       (BF16, BF16, E4M3), (F32, None, E4M3), (BF16, F32, BF16)])
def test_forward(rows, D, xt, rt, out):
    x, res, w = _inputs(rows, D, xt, rt, seed=rows + D)
    y, scale, h = kdn.kdn_rmsnorm_forward(x, w, residual=res, eps=1e-5, out_dtype=out)
    if res is None:
        assert h is None
        hs = x
    else:
        # one rounding of the fp32 sum, and (bf16) one to the stream's type
        assert torch.equal(h, (x.float() + res.float()).to(rt))
        hs = h
    want = rmsnorm_ref.forward(f64(hs), f64(w), 1e-5)
    if out == E4M3:
        assert y.shape == (rows, D) and y.stride(0) % 16 == 0
        _check_codes(y, scale, want, 64 * U)
    else:
        assert scale is None and y.dtype == out
        assert (np.abs(f64(y) - want) <= (64 * U + HALF[out] * (1 + 64 * U)) * np.abs(want)).all()


@pytest.mark.parametrize("rows,D", SIZES + [(2500, 96), (1500, 2048)])
@pytest.mark.parametrize("ht,yt,xt,through", [(BF16, BF16, F32, True), (F32, F32, F32, False),
                                              (BF16, F32, BF16, True), (F32, BF16, BF16, False)])
def test_backward(rows, D, ht, yt, xt, through):
    h, _, w = _inputs(rows, D, ht, None, seed=rows * 3 + D)
    dy, dh, _ = _inputs(rows, D, yt, ht, seed=rows * 5 + D)
    dh = dh if through else None
    g = kdn.kdn_rmsnorm_backward(h, w, dy, dh=dh, eps=1e-5, x_dtype=xt)
    args = f64(h), f64(w), f64(dy), 1e-5, None if dh is None else f64(dh)
    d, dw = rmsnorm_ref.backward(*args)
    md, mw = rmsnorm_ref.backward_magnitude(*args)
    tol = 160 * U * md
    assert (np.abs(f64(g['x']) - d) <= tol + HALF[xt] * (np.abs(d) + tol)).all()
    if through:
        assert (np.abs(f64(g['residual']) - d) <= tol + HALF[ht] * (np.abs(d) + tol)).all()
    else:
        assert g['residual'] is None
    assert (np.abs(f64(g['weight']) - dw) <= (64 + rows / 592 + 74 + 16) * U * mw).all()


@pytest.mark.parametrize("rows,D", [(700, 2048), (700, 1001), (150, 8200)])
def test_codes_are_the_exact_quotients(rows, D):
    """The factor of a row's norm is in all its elements alike, so a code is that
    of 448 h w / max |h w| over its block, also where fp32 roundings would
    decide between two."""
    g = torch.Generator().manual_seed(rows + D)
    x = torch.randn(rows, D, generator=g).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    y, _, _ = kdn.kdn_rmsnorm_forward(x, w, out_dtype=torch.float8_e4m3fn)
    u = f64(x) * f64(w)
    top = fp8_ref.spread(fp8_ref.scales(u) * 448.0, rows, D)
    assert (f64(y.float()) == fp8_ref.e4m3(448.0 * u / top)).all()


def test_rows_of_zeros_and_tiny_or_huge_values():
    D = 256
    x = torch.zeros(5, D, device='cuda')
    x[1] = 1e-30
    x[2] = 1e15 * torch.randn(D, device='cuda')
    x[3, 5] = 1e-20
    x[4] = torch.randn(D, device='cuda')
    w = torch.ones(D, device='cuda')
    y, scale, _ = kdn.kdn_rmsnorm_forward(x, w, eps=1e-6, out_dtype=E4M3)
    want = rmsnorm_ref.forward(f64(x), f64(w), 1e-6)
    _check_codes(y, scale, want, 64 * U)
    assert bool((y[0].float() == 0).all())
    g = kdn.kdn_rmsnorm_backward(x, w, x, eps=1e-6)
    assert all(torch.isfinite(g[k]).all() for k in ('x', 'weight'))


def test_what_is_not_finite_stays_in_its_row():
    D = 384
    x = torch.randn(4, D, device='cuda')
    x[1, 3], x[2, 200] = float('nan'), float('inf')
    w = torch.ones(D, device='cuda')
    for out in (F32, BF16, E4M3):
        y, scale, _ = kdn.kdn_rmsnorm_forward(x, w, out_dtype=out)
        y = y.float()
        assert torch.isfinite(y[[0, 3]]).all()
        assert torch.isnan(y[1, 3]) and torch.isnan(y[2, 200])
        if out == E4M3:
            assert torch.isfinite(scale[[0, 3]]).all()
            assert torch.isnan(scale[1, 0]) and torch.isnan(scale[2, 1])


def test_in_place_stream_padding_and_shapes():
    """h may be the residual itself, dresidual dh; any leading shape; the
    padding of an 8-bit row ends at the next 8 bytes."""
    x, res, w = _inputs(6, 100, F32, BF16, seed=1)
    y, s, h = kdn.kdn_rmsnorm_forward(x, w, residual=res, out_dtype=E4M3)
    stream = res.clone()
    buf = torch.zeros(6, 128, dtype=torch.uint8, device='cuda').fill_(7).view(E4M3)
    y2, s2, h2 = kdn.kdn_rmsnorm_forward(x, w, residual=stream, out_dtype=E4M3, h=stream,
                                         y=buf[:, :100])
    assert h2.data_ptr() == stream.data_ptr() and torch.equal(h2, h) and torch.equal(s, s2)
    assert torch.equal(y.float(), y2.float())
    assert bool((buf.view(torch.uint8)[:, 104:] == 7).all())
    x3 = x.view(2, 3, 100)
    y3, _, h3 = kdn.kdn_rmsnorm_forward(x3, w, residual=res.view(2, 3, 100))
    assert y3.shape == x3.shape and torch.equal(h3.view(6, 100), h)
    dh = torch.randn(6, 100, device='cuda').bfloat16()
    g = kdn.kdn_rmsnorm_backward(h, w, x, dh=dh)
    g2 = kdn.kdn_rmsnorm_backward(h, w, x, dh=dh, dresidual=dh)
    assert torch.equal(g['residual'], g2['residual']) and g2['residual'].data_ptr() == dh.data_ptr()


def test_no_rows():
    w = torch.ones(64, device='cuda')
    x = torch.empty(0, 64, device='cuda')
    for out in (F32, E4M3):
        y, s, h = kdn.kdn_rmsnorm_forward(x, w, residual=x, out_dtype=out)
        assert y.shape == (0, 64) and h.shape == (0, 64)
    g = kdn.kdn_rmsnorm_backward(x, w, x)
    assert bool((g['weight'] == 0).all())


def test_repeatable_and_graph():
    h, _, w = _inputs(3000, 512, BF16, None, seed=3)
    dy = torch.randn(3000, 512, device='cuda')
    g = kdn.kdn_rmsnorm_backward(h, w, dy, dh=h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hh, dd = torch.zeros_like(h), torch.zeros_like(dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gg = kdn.kdn_rmsnorm_backward(hh, w, dd, dh=hh)
        yy = kdn.kdn_rmsnorm_forward(hh, w, residual=hh, out_dtype=E4M3)
    for _ in range(2):
        hh.copy_(h), dd.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g[k], gg[k]) for k in g)
    y = kdn.kdn_rmsnorm_forward(h, w, residual=h, out_dtype=E4M3)
    assert torch.equal(y[0].float(), yy[0].float()) and torch.equal(y[1], yy[1])


def test_refusals():
    x, res, w = _inputs(4, 64, F32, BF16, seed=2)
    with pytest.raises(TypeError):
        kdn.kdn_rmsnorm_forward(x.half(), w)
    with pytest.raises(TypeError):
        kdn.kdn_rmsnorm_forward(x, w.bfloat16())
    with pytest.raises(ValueError):
        kdn.kdn_rmsnorm_forward(x, w[:32])
    with pytest.raises(ValueError):
        kdn.kdn_rmsnorm_forward(x, w, residual=res[:2])
    with pytest.raises(ValueError):
        kdn.kdn_rmsnorm_forward(x.t(), torch.ones(4, device='cuda'))
    with pytest.raises(TypeError):
        kdn.kdn_rmsnorm_forward(x, w, out_dtype=torch.float16)
    with pytest.raises(kdn.KdnError):
        kdn.kdn_rmsnorm_forward(x, w, eps=-1.0)
    with pytest.raises(kdn.KdnError) as e:
        kdn.kdn_rmsnorm_forward(torch.ones(1, 16400, device='cuda'),
                                torch.ones(16400, device='cuda'))
    assert e.value.status == kdn.KDN_ERR_UNSUPPORTED
