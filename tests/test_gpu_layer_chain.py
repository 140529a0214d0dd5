"""The pieces around a mixing layer, run together as a model would: norm to 8
bits, projections to q, k, v and gates, the mixers, the residual norm, and back
(needs a B200)."""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import fp8_ref, kdn_ref, linear_scan_ref, rmsnorm_ref
from gpu_util import f64, rel_maxabs, OUT_TOL

pytestmark = pytest.mark.gpu

B, T, H, d = 1, 70, 2, 128
D = H * d


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda n: kdn.kdn_fp8_quantize((torch.randn(n, D, generator=g) * D ** -0.5).cuda(),
                                          tile=True)


def test_norm_projections_and_kdn_layer_forward_and_back():
    weight = _weights(1)
    g = torch.Generator().manual_seed(2)
    stream = torch.randn(B * T, D, generator=g).bfloat16().cuda()
    mixed = torch.randn(B * T, D, generator=g).cuda()   # the layer before
    w_norm = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    wq, wk, wv, wg = weight(D), weight(D), weight(D), weight(3 * H)

    x8, sx, h = kdn.kdn_rmsnorm_forward(mixed, w_norm, residual=stream,
                                        out_dtype=torch.float8_e4m3fn)
    q, k, v = (kdn.kdn_fp8_matmul(x8, sx, *w).view(B, T, H, d) for w in (wq, wk, wv))
    gates = kdn.kdn_fp8_matmul(x8, sx, *wg, out_dtype=torch.float32).view(B, T, H, 3)
    k = (k.float() / k.float().norm(dim=-1, keepdim=True)).bfloat16()
    a = torch.sigmoid(2 + gates[..., 0]).contiguous()
    w = torch.nn.functional.softplus(gates[..., 1] - 2).contiguous()
    r = torch.nn.functional.softplus(gates[..., 2]).contiguous()
    o, S, p = kdn.kdn_iso_forward(q, k, v, a, w, r)

    # the projections from what was quantised, the layer from what was projected
    x64 = f64(x8.float()) * fp8_ref.spread(f64(sx), B * T, D)
    for got, wt in ((q, wq), (v, wv)):
        w64 = f64(wt[0].float()) * fp8_ref.spread(f64(wt[1]), D, D, True)
        assert rel_maxabs(got.reshape(B * T, D), x64 @ w64.T) <= OUT_TOL
    y64 = rmsnorm_ref.forward(f64(h), f64(w_norm), 1e-6)
    # (e4m3: half a step of 2^-3 relative, or of 2^-9 of the scale)
    assert (np.abs(x64 - y64) <= 1.01 * np.maximum(2.0 ** -4 * np.abs(y64), 2.0 ** -10 *
                                                   fp8_ref.spread(f64(sx), B * T, D))).all()
    ref = kdn_ref.iso_forward(*(f64(t) for t in (q, k, v, a, w, r)))
    assert rel_maxabs(o, ref[0]) <= OUT_TOL

    # the next norm takes o (fp32) as it is; its gradient is the layer's dO
    y, _, h2 = kdn.kdn_rmsnorm_forward(o.view(B * T, D), w_norm, residual=h)
    dy = torch.randn(B * T, D, generator=g).bfloat16().cuda()
    dh = torch.randn(B * T, D, generator=g).bfloat16().cuda()
    gn = kdn.kdn_rmsnorm_backward(h2, w_norm, dy, dh=dh, x_dtype=torch.float32)
    gl = kdn.kdn_backward('iso', q, k, v, a, w, r, gn['x'].view(B, T, H, d))
    d64, _ = rmsnorm_ref.backward(f64(h2), f64(w_norm), f64(dy), 1e-6, f64(dh))
    from oracle import kdn_grad
    want = kdn_grad.kdn_backward('iso', *(f64(t) for t in (q, k, v, a, w, r)),
                                 d64.reshape(B, T, H, d))
    for name in 'qkvawr':
        assert rel_maxabs(gl[name], want[name]) <= 1e-3, name


def test_norm_projections_and_linear_recurrence():
    """A recurrent layer: input and gates by 8-bit projections, the scan, its
    output normalised; then a token at a time from the scan's state."""
    weight = _weights(3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, T + 5, D, generator=g).bfloat16().cuda()
    w_norm = torch.ones(D, device='cuda')
    wx, wa = weight(D), weight(D)

    def parts(t):
        rows = t.reshape(-1, D)
        x8, sx, _ = kdn.kdn_rmsnorm_forward(rows, w_norm, out_dtype=torch.float8_e4m3fn)
        u = kdn.kdn_fp8_matmul(x8, sx, *wx)
        a = torch.sigmoid(2 + kdn.kdn_fp8_matmul(x8, sx, *wa, out_dtype=torch.float32))
        return a, torch.sqrt(1 - a * a), u

    a, b, u = (t.view(B, T + 5, D) for t in parts(x))
    y, h = kdn.kdn_linear_scan_forward(a, u, b=b)
    y64, h64 = linear_scan_ref.forward(f64(a[0]), f64(u[0]), f64(b[0]))
    assert rel_maxabs(y[0], y64) <= OUT_TOL and rel_maxabs(h[0], h64) <= 1e-5
    out, _, stream = kdn.kdn_rmsnorm_forward(y.view(-1, D), w_norm, residual=x.view(-1, D))
    assert out.shape == (T + 5, D) and torch.isfinite(out).all()

    # prefill, then single tokens
    _, state = kdn.kdn_linear_scan_forward(a[:, :T].contiguous(), u[:, :T].contiguous(),
                                           b=b[:, :T].contiguous())
    for t in range(T, T + 5):
        at, bt, ut = parts(x[:, t])
        yt = kdn.kdn_linear_scan_step(at, ut, state, b=bt)
        assert rel_maxabs(yt, f64(y[:, t])) <= OUT_TOL
    assert rel_maxabs(state, h64) <= 1e-4

    # gradients through norm and scan
    dout = torch.randn(T + 5, D, generator=g).cuda()
    gn = kdn.kdn_rmsnorm_backward(stream, w_norm, dout, x_dtype=torch.bfloat16)
    gs = kdn.kdn_linear_scan_backward(a, u, y, gn['x'].view(B, T + 5, D), b=b)
    want = linear_scan_ref.backward(f64(a[0]), f64(u[0]), f64(y[0]), f64(gn['x']), f64(b[0]))
    for name, ref in zip(('a', 'x', 'b', 'h0'), want):
        assert rel_maxabs(gs[name][0], ref) <= (OUT_TOL if name == 'x' else 1e-4), name


def test_different_calls_on_many_streams_at_once():
    """Products on pairs and on clusters, scans, norms and a mixing layer share
    the SMs, their tensor memory and one status word, and give the bits that
    each gives alone."""
    from kalman_filter_linear_b200 import synth
    g = torch.Generator().manual_seed(9)
    t = lambda *s: torch.randn(*s, generator=g).cuda()
    x8, sx = kdn.kdn_fp8_quantize(t(2048, 1024))
    w8, sw = kdn.kdn_fp8_quantize(t(2048, 1024), tile=True)
    v8, sv = kdn.kdn_fp8_quantize(t(1003, 1024))
    a, u, h0 = torch.rand(2, 3000, 512, device='cuda'), t(2, 3000, 512), t(2, 512)
    rows, w_norm = t(3000, 2048), t(2048)
    q = {k: v.cuda() for k, v in synth.layer_inputs(2, 512, 4, 128, 128, 'iso', seed=0,
                                                    dtype='bf16').items()}
    calls = [lambda: kdn.kdn_fp8_matmul(x8, sx, w8, sw),
             lambda: kdn.kdn_fp8_matmul(x8[:700], sx[:700], v8, sv, out_dtype=torch.float32),
             lambda: kdn.kdn_fp8_matmul(x8[:40], sx[:40], w8, sw),
             lambda: kdn.kdn_fp8_matmul(x8[:8], sx[:8], w8, sw),
             lambda: kdn.kdn_linear_scan_forward(a, u, h0=h0)[0],
             lambda: kdn.kdn_linear_scan_backward(a, None, u, u, h0=h0)['a'],
             lambda: kdn.kdn_linear_scan_forward(a[:1, :, :64].contiguous(),
                                                 u[:1, :, :64].contiguous())[1],
             lambda: kdn.kdn_rmsnorm_forward(rows, w_norm, out_dtype=torch.float8_e4m3fn)[0].float(),
             lambda: kdn.kdn_iso_forward(*(q[n] for n in 'qkvawr'))[0]]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for turn in range(12):
        got = []
        for i, call in enumerate(calls):
            with torch.cuda.stream(streams[(i + turn) % len(calls)]):
                got.append(call())
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (turn, i)
