"""The quick C++ form of the calls around a layer against the Python form: the
same bits, the same outputs in place, the same refusals (needs a B200)."""
import pytest
import torch

from kalman_filter_linear_b200 import kdn

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _flat(r):
    if isinstance(r, dict):
        return {k: v for k, v in r.items() if v is not None}
    return dict(enumerate(t for t in (r if isinstance(r, tuple) else (r,)) if t is not None))


def _calls():
    g = torch.Generator().manual_seed(1)
    t = lambda *s, d=F32: torch.randn(s, generator=g).to(d).cuda()
    a, x, b, h0 = torch.rand(2, 40, 72, device='cuda'), t(2, 40, 72, d=BF16), t(2, 40, 72), t(2, 72)
    cu = torch.tensor([0, 15, 40], dtype=torch.int32, device='cuda')
    y = t(2, 40, 72, d=BF16)
    rows, w = t(30, 200), t(200)
    q, s = kdn.kdn_fp8_quantize(t(30, 200))
    w8, sw = kdn.kdn_fp8_quantize(t(50, 200), tile=True)
    w1, s1 = kdn.kdn_fp8_quantize(t(50, 200))
    yield lambda: kdn.kdn_linear_scan_step(a[:, 0].contiguous(), x[:, 0].contiguous(), h0.clone())
    yield lambda: kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    yield lambda: kdn.kdn_linear_scan_forward(a[0], x[0], h0=h0, cu_seqlens=cu)
    yield lambda: kdn.kdn_linear_scan_forward(a, x, y=torch.empty_like(x), h_out=torch.empty_like(h0))
    yield lambda: kdn.kdn_linear_scan_forward(a[:, :0], x[:, :0], h0=h0)
    yield lambda: kdn.kdn_linear_scan_backward(a, x, y, x, b=b, h0=h0, dh_T=h0)
    yield lambda: kdn.kdn_linear_scan_backward(a[0], None, y[0], x[0], cu_seqlens=cu)
    for out in (F32, BF16, E4M3):
        yield lambda out=out: kdn.kdn_rmsnorm_forward(rows, w, out_dtype=out)
        yield lambda out=out: kdn.kdn_rmsnorm_forward(rows.bfloat16(), w, residual=rows, eps=0.1,
                                                      out_dtype=out)
    yield lambda: kdn.kdn_rmsnorm_backward(rows, w, rows.bfloat16())
    yield lambda: kdn.kdn_rmsnorm_backward(rows, w, rows, dh=rows, x_dtype=BF16)
    yield lambda: kdn.kdn_rmsnorm_backward(rows, w, rows, want_residual=True)
    yield lambda: kdn.kdn_rmsnorm_backward(rows[:0], w, rows[:0])
    for tile in (False, True):
        for tr in (False, True):
            yield lambda tile=tile, tr=tr: kdn.kdn_fp8_quantize(rows, tile=tile, transpose=tr)
    yield lambda: kdn.kdn_fp8_matmul(q, s, w8, sw)
    yield lambda: kdn.kdn_fp8_matmul(q, s, w1, s1, out_dtype=F32)
    yield lambda: kdn.kdn_fp8_matmul(q[:1], s[:1], w8, sw, out_dtype=F32)
    yield lambda: kdn.kdn_fp8_matmul(q[:0], s[:0], w8, sw)


def test_both_forms_give_the_same(monkeypatch):
    quick = kdn._load_quick()
    assert quick is not kdn._NoQuick, 'the quick form is not built'
    for call in _calls():
        monkeypatch.setattr(kdn, '_quick', quick)
        one = _flat(call())
        monkeypatch.setattr(kdn, '_quick', kdn._NoQuick)
        two = _flat(call())
        assert one.keys() == two.keys()
        for k in one:
            assert one[k].dtype == two[k].dtype and one[k].shape == two[k].shape
            assert one[k].numel() == 0 or one[k].stride() == two[k].stride()
            assert torch.equal(one[k].float(), two[k].float())


def test_given_outputs_are_the_ones_returned():
    a, x = torch.rand(2, 8, 16, device='cuda'), torch.randn(2, 8, 16, device='cuda')
    y, h = torch.empty_like(x), torch.empty(2, 16, device='cuda')
    y2, h2 = kdn.kdn_linear_scan_forward(a, x, y=y, h_out=h)
    assert y2 is y and h2 is h
    q = torch.empty(4, 16, dtype=E4M3, device='cuda')
    assert kdn.kdn_fp8_quantize(torch.randn(4, 16, device='cuda'), q=q)[0] is q


def test_what_is_out_of_the_ordinary_goes_to_the_python_form():
    """None, and nothing done: other types, shapes, strides, devices, counts."""
    m = kdn._load_quick()
    a, x = torch.rand(2, 8, 16, device='cuda'), torch.randn(2, 8, 16, device='cuda')
    h = torch.zeros(2, 16, device='cuda')
    n = (None,) * 5
    assert m.scan_forward(a, x, *n) is not None
    for bad in ((a, x.half()), (a, x[:, :4]), (a.transpose(0, 1), x), (a.cpu(), x.cpu()), (a, None),
                (1, x), (a.double(), x)):
        assert m.scan_forward(*bad, *n) is None
    assert m.scan_forward(a, x) is None and m.matmul() is None
    assert m.scan_step(a[:, 0].contiguous(), x[:, 0].contiguous(), h.bfloat16(), None, None) is None
    assert m.norm_forward(h, h[0], None, float('nan'), 0, None, None, None) is None
    assert m.norm_forward(h, h[0], None, 1e-6, -1, None, None, None) is None
    assert m.norm_forward(h, h[0], None, 'x', 0, None, None, None) is None
    assert m.quantize(h[:, ::2], False, False, None, None) is None
    assert bool((h == 0).all())
    with pytest.raises(TypeError):
        kdn.kdn_linear_scan_forward(a, x.half())
    with pytest.raises(kdn.KdnError):
        kdn.kdn_rmsnorm_forward(h, h[0].clone(), eps=-1.0)
