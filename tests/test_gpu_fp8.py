"""8-bit blocks and their product (kdn_fp8_quantize, kdn_fp8_matmul) against
the fp64 oracle (needs a B200).

Tolerances.  Quantising rounds the scale once (the maximum itself is exact) and
a quotient three times, so a code is that of either end of an interval of 4 of
2^-24 around value / scale.  A product of e4m3 numbers is exact in fp32; a
block's sum of 128 adds at most 128 roundings, truncating ones (2^-23) at the
worst, and each block's scaled addition three: (128 + 3 blocks + 8) * 2^-23 of
the sum of absolute values, and half a step of the output type.
"""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import fp8_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {F32: U, BF16: 2.0 ** -8}


def _matrix(rows, cols, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
            ).to(dt).cuda()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (128, 128), (5, 130), (129, 127), (200, 300),
                                       (1000, 16), (64, 1024), (257, 520)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(rows, cols, dt, tile, transpose):
    x = _matrix(rows, cols, dt, seed=rows + cols)
    q, s = kdn.kdn_fp8_quantize(x, tile=tile, transpose=transpose)
    v = f64(x).T if transpose else f64(x)
    want = fp8_ref.scales(v, tile)
    assert q.shape == v.shape and tuple(s.shape) == want.shape
    assert (np.abs(f64(s) - want) <= U * want).all()
    z = v / fp8_ref.spread(want, *v.shape, tile)
    lo, hi = fp8_ref.e4m3(z - 4 * U * np.abs(z)), fp8_ref.e4m3(z + 4 * U * np.abs(z))
    got = f64(q.float())
    assert ((got >= lo) & (got <= hi)).all()


def test_quantize_extreme_blocks():
    """Zeros, numbers below the floor, the largest ones, and what is not
    finite: only its own block is marked."""
    x = torch.zeros(6, 384, device='cuda')
    x[1, :128] = 1e-35
    x[2] = 3e38
    x[3] = torch.randn(384, device='cuda')
    x[3, 5], x[4, 300], x[4, 0] = float('nan'), float('inf'), 1.0
    for tr in (False, True):
        q, s = kdn.kdn_fp8_quantize(x.t().contiguous() if tr else x, transpose=tr)
        qf = q.float()
        assert bool((qf[0] == 0).all()) and bool((s[0] > 0).all())
        # 1e-35 over the floor's scale, 2^-100 / 448, is 0.00568: 2.9 of the
        # smallest steps, 2^-9, so 3
        assert bool((qf[1, :128] == 3 * 2.0 ** -9).all()) and bool((qf[1, 128:] == 0).all())
        assert bool((qf[2] == 448).all())
        assert torch.isnan(s[3, 0]) and torch.isfinite(s[3, 1:]).all()
        assert torch.isnan(qf[3, 5])
        assert not torch.isfinite(s[4, 2]) and torch.isfinite(s[4, :2]).all()
        assert torch.isnan(qf[4, 300]) and qf[4, 0] == 448


def _codes(rows, cols, tile, seed):
    return kdn.kdn_fp8_quantize(_matrix(rows, cols, F32, seed), tile=tile)


SHAPES = [(1, 1, 1), (1, 16, 16), (3, 100, 128), (8, 2048, 2048), (16, 130, 1000), (17, 64, 129),
          (33, 257, 640), (64, 128, 4096), (65, 512, 256), (128, 300, 2000), (200, 2048, 512),
          (300, 1111, 384), (500, 2000, 260), (1000, 1500, 300), (1024, 2048, 128),
          (129, 4100, 1300), (2100, 2300, 200)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("tile,out", [(True, BF16), (True, F32), (False, BF16), (False, F32)])
def test_matmul(M, N, K, tile, out):
    x, sx = _codes(M, K, False, M + K)
    w, sw = _codes(N, K, tile, N + 2 * K)
    status = torch.zeros(1, dtype=torch.int32, device='cuda')
    y = kdn.kdn_fp8_matmul(x, sx, w, sw, out_dtype=out, status=status)
    assert kdn.kdn_read_workspace_status(status.view(torch.uint8)) == kdn.KDN_OK
    want, mag = fp8_ref.matmul(f64(x.float()), f64(sx), f64(w.float()), f64(sw),
                               tile and tuple(sw.shape) != (N, sx.shape[1]))
    tol = (128 + 3 * sx.shape[1] + 8) * 2 * U * mag
    err = np.abs(f64(y) - want)
    assert (err <= tol + HALF[out] * (np.abs(want) + tol)).all(), (err - tol).max()


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(257, 1032, 130), (700, 1000, 1200), (2100, 2312, 260),
                                   (513, 8, 384), (3000, 1544, 2050), (40, 4104, 640),
                                   (64, 2056, 1100), (300, 120, 4300)])
def test_matmul_tiles_that_end_early(M, N, K, out, tile):
    """Pairs of blocks whose rows or columns end inside a tile, with outputs
    that bulk copies store, sums over more blocks than scales come for at once,
    and clusters that share a sum."""
    x, sx = _codes(M, K, False, M)
    w, sw = _codes(N, K, tile, N + 1)
    got = kdn.kdn_fp8_matmul(x, sx, w, sw, out_dtype=out)
    want, mag = fp8_ref.matmul(f64(x.float()), f64(sx), f64(w.float()), f64(sw), tile)
    tol = (128 + 3 * -(-K // 128) + 8) * 2 * U * mag
    tol = tol + HALF[out] * (np.abs(want) + tol)
    assert (np.abs(f64(got) - want) <= tol).all()


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,cols", [(1500, 1024), (900, 1003)])
def test_codes_of_fp32_are_the_exact_quotients(rows, cols, tile, transpose):
    """Of a million numbers a few quotients lie so near the middle of two codes
    that the roundings of fp32 would decide: the code is the exact quotient's.
    (An fp64 quotient is within 2^-52, which no element here comes near to.)"""
    x = _matrix(rows, cols, F32, seed=rows + 1)
    q, _ = kdn.kdn_fp8_quantize(x, tile=tile, transpose=transpose)
    v = f64(x).T if transpose else f64(x)
    top = fp8_ref.spread(fp8_ref.scales(v, tile) * 448.0, *v.shape, tile)
    assert (f64(q.float()) == fp8_ref.e4m3(448.0 * v / top)).all()


def test_matmul_small_integers_are_exact():
    """Codes that are small integers with scales of one: every sum is an
    integer below 2^24, so the product has to be exact."""
    for M, N, K in [(4, 128, 1024), (40, 300, 640), (300, 600, 1000), (1500, 2100, 512)]:
        g = torch.Generator().manual_seed(M)
        ints = lambda r: torch.randint(-8, 9, (r, K), generator=g).float().cuda()
        xi, wi = ints(M), ints(N)
        pad = lambda t: torch.nn.functional.pad(t, (0, -K % 16)).to(E4M3)[:, :K]
        kb = -(-K // 128)
        one = lambda r: torch.ones(r, kb, device='cuda')
        for sw in (one(N), one(-(-N // 128))):
            y = kdn.kdn_fp8_matmul(pad(xi), one(M), pad(wi), sw, out_dtype=F32)
            assert torch.equal(y.double(), xi.double() @ wi.double().t())


def test_matmul_does_not_read_padding_nor_write_outside():
    """Garbage behind K (NaN codes), behind the last row, and around the
    output."""
    for M, N, K in [(5, 100, 200), (300, 333, 200), (1300, 1400, 200)]:
        x, sx = _codes(M, K, False, 1)
        w, sw = _codes(N, K, True, 2)
        want = kdn.kdn_fp8_matmul(x, sx, w, sw)
        big = lambda q, r: (torch.full((r + 200, 256), 0x7f, dtype=torch.uint8, device='cuda'))
        xb, wb = big(x, M), big(w, N)
        xb[:M, :K], wb[:N, :K] = x.view(torch.uint8), w.view(torch.uint8)
        room = torch.full((M + 16, N), 3.0, dtype=BF16, device='cuda')
        y = kdn.kdn_fp8_matmul(xb.view(E4M3)[:M, :K], sx, wb.view(E4M3)[:N, :K], sw,
                               out=room[8:8 + M] if N % 8 == 0 else None)
        assert torch.equal(y, want)
        assert bool((room[:8] == 3).all()) and bool((room[8 + M:] == 3).all())


def test_matmul_what_is_not_finite_stays_in_its_row():
    for M, N, K in [(6, 256, 512), (700, 1500, 512)]:
        xf, wf = _matrix(M, K, F32, 3), _matrix(N, K, F32, 4)
        xf[2, 7] = float('nan')
        wf[130, 300] = float('inf')
        x, sx = kdn.kdn_fp8_quantize(xf)
        w, sw = kdn.kdn_fp8_quantize(wf)
        y = kdn.kdn_fp8_matmul(x, sx, w, sw)
        bad = torch.zeros(M, N, dtype=torch.bool, device='cuda')
        bad[2], bad[:, 130] = True, True
        assert torch.equal(torch.isfinite(y), ~bad)


def test_gradients_of_a_projection():
    """dx = dy w and dw = dy^T x with the quantised transposes, against the
    product of the dequantised factors, for a ragged number of tokens."""
    M, N, K = 333, 260, 400
    x, w, dy = _matrix(M, K, BF16, 5), _matrix(N, K, F32, 6), _matrix(M, N, F32, 7)
    for a, b, tile, shape in [(kdn.kdn_fp8_quantize(dy),
                               kdn.kdn_fp8_quantize(w, tile=True, transpose=True), True, (M, K)),
                              (kdn.kdn_fp8_quantize(dy, transpose=True),
                               kdn.kdn_fp8_quantize(x, transpose=True), False, (N, K))]:
        got = kdn.kdn_fp8_matmul(*a, *b, out_dtype=F32)
        assert got.shape == shape
        want, mag = fp8_ref.matmul(f64(a[0].float()), f64(a[1]), f64(b[0].float()), f64(b[1]), tile)
        assert (np.abs(f64(got) - want) <= (128 + 3 * a[1].shape[1] + 8) * 2 * U * mag).all()
    # and near the true gradients: each factor within half an e4m3 step (2^-4)
    # of its value, or 2^-10 of its block's scale times 448
    true = f64(dy).T @ f64(x)
    assert np.linalg.norm(f64(got) - true) <= 2 * 2.0 ** -4 * np.linalg.norm(
        np.abs(f64(dy)).T @ np.abs(f64(x)))


def test_streams_graph_and_repeatability():
    cases = [(8, 2048, 2048), (300, 1000, 512), (2000, 2048, 256)]
    sets = [(_codes(m, k, False, 1), _codes(n, k, True, 2)) for m, n, k in cases]
    want = [kdn.kdn_fp8_matmul(*x, *w) for x, w in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, (x, w) in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(kdn.kdn_fp8_matmul(*x, *w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    side = torch.cuda.Stream()
    xin = _matrix(300, 512, BF16, 9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = kdn.kdn_fp8_matmul(*kdn.kdn_fp8_quantize(xin), *sets[1][1])
    for seed in (9, 10):
        xin.copy_(_matrix(300, 512, BF16, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, kdn.kdn_fp8_matmul(*kdn.kdn_fp8_quantize(xin), *sets[1][1]))


def test_refusals_and_empty():
    x, sx = _codes(4, 64, False, 1)
    w, sw = _codes(300, 64, True, 2)
    assert kdn.kdn_fp8_matmul(x[:0], sx[:0], w, sw).shape == (0, 300)
    q, s = kdn.kdn_fp8_quantize(torch.empty(0, 64, device='cuda'))
    assert q.shape == (0, 64) and s.shape == (0, 1)
    with pytest.raises(TypeError):
        kdn.kdn_fp8_matmul(x.float(), sx, w, sw)
    with pytest.raises(ValueError):
        kdn.kdn_fp8_matmul(x, sx[:2], w, sw)
    with pytest.raises(ValueError):
        kdn.kdn_fp8_matmul(x, sx, w, sw[:2])
    with pytest.raises(ValueError):
        kdn.kdn_fp8_matmul(x[:, :32], sx, w, sw)
    odd = torch.zeros(4, 68, dtype=torch.uint8, device='cuda').view(E4M3)[:, :64]
    with pytest.raises(ValueError):
        kdn.kdn_fp8_matmul(odd, sx, w, sw)
    with pytest.raises(TypeError):
        kdn.kdn_fp8_matmul(x, sx, w, sw, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        kdn.kdn_fp8_quantize(torch.ones(4, 4, device='cuda', dtype=torch.float16))
