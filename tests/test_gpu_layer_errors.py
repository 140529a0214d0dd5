"""What the calls around a layer report when the CUDA runtime reports an error
(needs a B200).  The errors here are answers of ordinary runtime calls; nothing
on the GPU goes wrong."""
import ctypes

import pytest
import torch

from kalman_filter_linear_b200 import kdn

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(params=['quick', 'python'])
def form(request, monkeypatch):
    """Both forms of the binding."""
    if request.param == 'python':
        monkeypatch.setattr(kdn, '_quick', kdn._NoQuick)


@pytest.fixture
def runtime():
    rt = ctypes.CDLL('libcudart.so.12')
    yield rt
    rt.cudaGetLastError()


def _leave_an_error(rt):
    """An invalid argument to the runtime, whose error stays to be read."""
    assert rt.cudaSetDevice(1 << 20) != 0


def _calls():
    g = torch.Generator().manual_seed(2)
    t = lambda *s: torch.randn(s, generator=g).cuda()
    a, x = torch.sigmoid(t(2, 40, 72)), t(2, 40, 72)
    one, long = torch.sigmoid(t(1, 20000, 64)), t(1, 20000, 64)   # (one column: another kernel)
    rows, w = t(30, 200), t(200)
    q, s = kdn.kdn_fp8_quantize(t(30, 200))
    big, sb = kdn.kdn_fp8_quantize(t(600, 200))
    w8, sw = kdn.kdn_fp8_quantize(t(1024, 200), tile=True)
    yield 'scan', lambda: kdn.kdn_linear_scan_forward(a, x)
    yield 'scan, long', lambda: kdn.kdn_linear_scan_forward(one, long)
    yield 'scan backward', lambda: kdn.kdn_linear_scan_backward(a, None, x, x).values()
    yield 'scan backward, long', lambda: kdn.kdn_linear_scan_backward(one, None, long, long).values()
    yield 'norm', lambda: kdn.kdn_rmsnorm_forward(rows, w, residual=rows)
    yield 'norm backward', lambda: kdn.kdn_rmsnorm_backward(rows, w, rows, dh=rows).values()
    for tile in (False, True):
        for tr in (False, True):
            yield f'quantize {tile} {tr}', lambda tile=tile, tr=tr: kdn.kdn_fp8_quantize(
                rows, tile=tile, transpose=tr)
    yield 'product', lambda: [kdn.kdn_fp8_matmul(q, s, w8, sw)]
    yield 'product of many rows', lambda: [kdn.kdn_fp8_matmul(big, sb, w8, sw)]


def test_an_error_left_behind_is_not_the_calls(form, runtime):
    for name, call in _calls():
        want = [t for t in call() if t is not None]
        _leave_an_error(runtime)
        got = [t for t in call() if t is not None]
        assert runtime.cudaGetLastError() != 0, 'the error was somebody else\'s to read'
        torch.cuda.synchronize()
        assert all(torch.equal(p.float(), r.float()) for p, r in zip(got, want)), name


def test_a_step_in_place_is_one_step(form, runtime):
    """The state and the gradient that are updated in place."""
    a, x = torch.full((2, 8), 0.5, device='cuda'), torch.ones(2, 8, device='cuda')
    h = torch.zeros(2, 8, device='cuda')
    _leave_an_error(runtime)
    kdn.kdn_linear_scan_step(a, x, h)
    runtime.cudaGetLastError()
    assert bool((h == 1).all())
    dy = torch.randn(2, 8, device='cuda')
    want = kdn.kdn_rmsnorm_backward(x, x[0], dy, dh=a)['residual']
    dh = a.clone()
    _leave_an_error(runtime)
    kdn.kdn_rmsnorm_backward(x, x[0], dy, dh=dh, dresidual=dh)
    runtime.cudaGetLastError()
    assert torch.equal(dh, want)


def test_a_call_that_fails_is_not_made_again(monkeypatch, runtime):
    """On a stream whose capture has been invalidated (a synchronisation is not
    allowed in one) a launch is an error; the Python form is not tried then."""
    a, x = torch.full((2, 8), 0.5, device='cuda'), torch.ones(2, 8, device='cuda')
    h, y = torch.zeros(2, 8, device='cuda'), torch.empty(2, 8, device='cuda')
    kdn.kdn_linear_scan_step(a, x, h, y=y)
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    torch.cuda.synchronize()

    def again(*args):
        raise AssertionError('the call was made a second time')

    monkeypatch.setattr(kdn, '_call', again)
    assert kdn._load_quick() is not kdn._NoQuick
    assert runtime.cudaStreamBeginCapture(handle, 2) == 0       # 2: relaxed
    try:
        assert runtime.cudaStreamSynchronize(handle) != 0
        with torch.cuda.stream(side), pytest.raises(kdn.KdnError) as e:
            kdn.kdn_linear_scan_step(a, x, h, y=y)
    finally:
        runtime.cudaStreamEndCapture(handle, ctypes.byref(graph))
    assert e.value.status == kdn.KDN_ERR_CUDA
    assert 'kdn_linear_scan_step' in str(e.value)
    runtime.cudaGetLastError()
    torch.cuda.synchronize()
    assert bool((h == 1).all())
    kdn._quick.scan_step(a, x, h, None, y)
    assert bool((h == 1.5).all())
