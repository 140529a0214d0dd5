"""Where the 8-bit calls end: outputs that the caller lays out to the last byte,
empty batches, quotients next to the middle of two codes (needs a B200)."""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import fp8_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
GUARD = 0x55


@pytest.fixture(params=['quick', 'python'])
def form(request, monkeypatch):
    """Both forms of the binding."""
    if request.param == 'python':
        monkeypatch.setattr(kdn, '_quick', kdn._NoQuick)


def _guarded(R, C, more=0):
    """An e4m3 matrix [R, C] whose last row ends at C, in a room of guard bytes;
    which of the room's bytes lie between a row's end and the next multiple of
    16, and which others are not the matrix's.  (One row is contiguous, whatever
    its length.)"""
    up = -(-C // 16) * 16
    ld = up + more
    room = torch.full((R * ld + 64,), GUARD, dtype=torch.uint8, device='cuda')
    gaps, outside = torch.zeros_like(room, dtype=torch.bool), torch.ones_like(room, dtype=torch.bool)
    for r in range(R):
        outside[r * ld:r * ld + (up if r + 1 < R else C)] = False
        gaps[r * ld + C:r * ld + up] = r + 1 < R
    return room.view(E4M3).as_strided((R, C), (ld if R > 1 else C, 1)), room, gaps, outside


@pytest.mark.parametrize("R,C", [(1, 1), (1, 7), (1, 8), (1, 100), (1, 104), (1, 112), (1, 131),
                                 (3, 100), (130, 104), (20, 131), (20, 136), (129, 255)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_writes_nothing_behind_a_given_matrix(R, C, dt, tile, transpose, form):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(*((C, R) if transpose else (R, C)), generator=g).to(dt).cuda()
    want, s_want = kdn.kdn_fp8_quantize(x, tile=tile, transpose=transpose)
    for more in (0, 32):
        q, room, _, outside = _guarded(R, C, more)
        got, s = kdn.kdn_fp8_quantize(x, tile=tile, transpose=transpose, q=q)
        assert got is q and torch.equal(s, s_want)
        assert torch.equal(q.float(), want.float())
        assert bool((room[outside] == GUARD).all())


@pytest.mark.parametrize("R,C", [(1, 1), (1, 100), (1, 104), (3, 100), (40, 2056), (40, 1003)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_norm_writes_nothing_behind_a_row(R, C, dt, form):
    g = torch.Generator().manual_seed(R + C)
    x, w = torch.randn(R, C, generator=g).to(dt).cuda(), torch.rand(C, generator=g).cuda()
    want, s_want, _ = kdn.kdn_rmsnorm_forward(x, w, out_dtype=E4M3)
    y, room, gaps, outside = _guarded(R, C)
    got, s, _ = kdn.kdn_rmsnorm_forward(x, w, out_dtype=E4M3, y=y)
    assert got is y and torch.equal(s, s_want) and torch.equal(y.float(), want.float())
    assert bool((room[outside | gaps] == GUARD).all())


def _exact_codes(v, tile):
    """The codes of the exact quotients 448 v / magnitude, ties to the even one.
    (448 v is exact in fp64, the magnitude is one of the values, and a tie's
    quotient has five bits, so it is seen as one; another quotient of bf16 numbers
    is 2^-13 of itself away from a tie.)"""
    rows, cols = v.shape
    p = np.pad(np.abs(v), ((0, -rows % 128 if tile else 0), (0, -cols % 128)))
    top = p.reshape(-1, 128 if tile else 1, p.shape[1] // 128, 128).max((1, 3))
    top = fp8_ref.spread(np.maximum(top, fp8_ref.FLOOR), rows, cols, tile)
    return fp8_ref.e4m3(448.0 * v / top)


@pytest.mark.parametrize("transpose", [False, True])
def test_codes_of_bf16_round_ties_to_even_in_rows(transpose):
    """Every significand of a value against every one of its block's largest, over
    the exponents that give codes: blocks of one largest and 127 others."""
    m = torch.arange(128, 256, dtype=torch.float64)
    v = (m[:, None] * 2.0 ** -torch.arange(8, 29)).flatten()          # below every m, to codes of 0
    v = torch.cat([v, v.new_zeros(-len(v) % 127)]).reshape(-1, 127)
    x = torch.cat([m[:, None, None].expand(-1, len(v), 1), v.expand(128, -1, -1)], 2).reshape(128, -1)
    x = (x * torch.where(torch.arange(x.shape[1]) % 3 == 1, -1.0, 1.0)).bfloat16().cuda()
    for part in (x, x[:, :x.shape[1] - 3].contiguous()):                # whole pieces, and not
        q, _ = kdn.kdn_fp8_quantize(part.t().contiguous() if transpose else part, transpose=transpose)
        np.testing.assert_array_equal(f64(q.float()), _exact_codes(f64(part), False))


@pytest.mark.parametrize("transpose", [False, True])
def test_codes_of_bf16_round_ties_to_even_in_tiles(transpose):
    """A tile for every significand of the largest value."""
    g = torch.Generator().manual_seed(3)
    v = torch.randint(128, 256, (1024, 2048), generator=g) * 2.0 ** -torch.randint(8, 24, (1024, 2048),
                                                                                  generator=g)
    v = v.double()
    for i, m in enumerate(range(128, 256)):
        v[i // 16 * 128 + i % 100, i % 16 * 128 + i % 77] = -m
    x = v.bfloat16().cuda()
    q, _ = kdn.kdn_fp8_quantize(x, tile=True, transpose=transpose)
    want = _exact_codes(f64(x).T if transpose else f64(x), True)
    np.testing.assert_array_equal(f64(q.float()), want)


def _next_to_middles(rows, blocks, seed):
    """fp32 blocks of 128: their largest value, then for each middle of two codes
    below 2^-6 and some above it the five numbers whose quotients are nearest."""
    rng = np.random.default_rng(seed)
    top = rng.uniform(1, 2, (rows, blocks, 1)).astype(np.float32)
    mid = np.concatenate([(2 * np.arange(8) + 1) * 2.0 ** -10,
                          (2 * rng.integers(8, 16, 17) + 1) * 2.0 ** rng.integers(-10, 3, 17)])
    v = (mid * top.astype(np.float64) / 448.0).astype(np.float32)
    v = (v.view(np.int32)[..., None] + np.arange(-2, 3, dtype=np.int32)).view(np.float32)
    v = np.concatenate([top, v.reshape(rows, blocks, 125), np.zeros((rows, blocks, 2))], 2)
    return (v * rng.choice([-1.0, 1.0], v.shape)).astype(np.float32)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("cols", [1024, 1016, 1003])
def test_codes_of_fp32_next_to_middles_in_rows(cols, transpose):
    x = torch.from_numpy(_next_to_middles(512, 8, cols).reshape(512, 1024)[:, :cols].copy()).cuda()
    q, _ = kdn.kdn_fp8_quantize(x.t().contiguous() if transpose else x, transpose=transpose)
    np.testing.assert_array_equal(f64(q.float()), _exact_codes(f64(x), False))


@pytest.mark.parametrize("transpose", [False, True])
def test_codes_of_fp32_next_to_middles_in_tiles(transpose):
    v = _next_to_middles(1, 64, 5).reshape(8, 8, 1, 128)
    x = np.repeat(v, 128, 2)
    x[:, :, 1:, 0] = 0
    x = torch.from_numpy(x.transpose(0, 2, 1, 3).reshape(1024, 1024).copy()).cuda()
    q, _ = kdn.kdn_fp8_quantize(x.t().contiguous() if transpose else x, tile=True, transpose=transpose)
    np.testing.assert_array_equal(f64(q.float()), _exact_codes(f64(x), True))


@pytest.mark.parametrize("cols", [128, 1024, 1003, 4096])
@pytest.mark.parametrize("weighted", [False, True])
def test_codes_of_the_norm_next_to_middles(cols, weighted):
    """The factor 1 / rms is the same in a whole row, so a code is that of 448 h w
    over the block's largest |h w|."""
    rng = np.random.default_rng(cols)
    v = _next_to_middles(256, 32, cols).reshape(256, 4096)[:, :cols]
    w = rng.uniform(0.5, 2, cols).astype(np.float32) if weighted else np.ones(cols, np.float32)
    w[::128] = 2.0                                       # (the largest stays so)
    h = (v.astype(np.float64) / w).astype(np.float32)
    y, _, _ = kdn.kdn_rmsnorm_forward(torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda(),
                                      out_dtype=E4M3)
    np.testing.assert_array_equal(f64(y.float()), _exact_codes(h.astype(np.float64) * w, False))


@pytest.mark.parametrize("tile", [False, True])
def test_empty_matrices(tile, form):
    """No rows or no columns, either way round; an empty batch's weight gradient
    is zeros."""
    blocks = lambda n: -(-n // 128)
    for shape in ((0, 300), (300, 0), (0, 0), (1, 0), (0, 1)):
        x = torch.empty(shape, device='cuda')
        for tr in (False, True):
            R, C = shape[::-1] if tr else shape
            q, s = kdn.kdn_fp8_quantize(x, tile=tile, transpose=tr)
            assert q.shape == (R, C) and q.dtype == E4M3
            assert s.shape == (blocks(R) if tile else R, blocks(C))
            q2, _ = kdn.kdn_fp8_quantize(x, tile=tile, transpose=tr, q=q)
            assert q2 is q


def test_products_over_nothing(form):
    dy, x = torch.empty(0, 300, device='cuda'), torch.empty(0, 40, device='cuda')
    a, b = (kdn.kdn_fp8_quantize(t, transpose=True) for t in (dy, x))
    for out in (F32, BF16):
        room = torch.full((300, 40), 7.0, dtype=out, device='cuda')
        got = kdn.kdn_fp8_matmul(*a, *b, out_dtype=out, out=room)
        assert got is room and bool((got == 0).all())
        assert bool((kdn.kdn_fp8_matmul(*a, *b, out_dtype=out) == 0).all())
    w = kdn.kdn_fp8_quantize(torch.randn(300, 40, device='cuda'), tile=True)
    rows = kdn.kdn_fp8_quantize(torch.randn(5, 40, device='cuda'))
    assert kdn.kdn_fp8_matmul(rows[0][:0], rows[1][:0], *w).shape == (0, 300)
    assert kdn.kdn_fp8_matmul(*rows, w[0][:0], w[1][:0]).shape == (5, 0)
    one = (torch.empty(1, 0, device='cuda').to(E4M3), torch.empty(1, 0, device='cuda'))
    assert bool((kdn.kdn_fp8_matmul(*one, *one) == 0).all())
    with pytest.raises(ValueError):
        kdn.kdn_fp8_matmul(*a, b[0], b[1][:3])


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("M,N,K", [(5, 100, 200), (17, 129, 384), (40, 333, 200), (300, 333, 200),
                                   (700, 1000, 260), (1300, 1403, 200), (2100, 2312, 130),
                                   (4000, 2047, 260)])
def test_matmul_writes_nothing_around_its_output(M, N, K, tile, out):
    """Few rows and tiles of both widths, rows that bulk copies store and rows that
    they cannot; several tiles a pair."""
    g = torch.Generator().manual_seed(M + N)
    x = kdn.kdn_fp8_quantize(torch.randn(M, K, generator=g).cuda())
    w = kdn.kdn_fp8_quantize(torch.randn(N, K, generator=g).cuda(), tile=tile)
    want = kdn.kdn_fp8_matmul(*x, *w, out_dtype=out)
    room = torch.full((M + 16, N), 3.0, dtype=out, device='cuda')
    got = kdn.kdn_fp8_matmul(*x, *w, out_dtype=out, out=room[8:8 + M])
    assert torch.equal(got, want)
    assert bool((room[:8] == 3).all()) and bool((room[8 + M:] == 3).all())
    v = [f64(q.float()) * fp8_ref.spread(f64(s), *q.shape, t) for q, s, t in ((*x, False), (*w, tile))]
    exact, size = v[0] @ v[1].T, np.abs(v[0]) @ np.abs(v[1]).T
    # (a block's 128 additions at 2^-23, three for each block, and the output's own)
    tol = (128 + 3 * -(-K // 128) + 8) * 2.0 ** -23 * size
    tol = tol + (2.0 ** -24 if out is F32 else 2.0 ** -8) * (np.abs(exact) + tol)
    assert (np.abs(f64(got) - exact) <= tol).all()
