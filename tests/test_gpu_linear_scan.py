"""The gated linear recurrence (kdn_linear_scan_*) against the fp64 oracle
(needs a B200).

Tolerances: the oracle's bound counts, per element, the roundings that an fp32
evaluation of the recurrence can add in any order of composition (in units of
2^-24); an output in bf16 adds half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import linear_scan_ref as ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def _half_step(dt):
    return torch.finfo(dt).eps / 2 if dt != F32 else 0.0


def _inputs(shape, ends, gate, dt, with_b, seed, device='cuda'):
    g = torch.Generator().manual_seed(seed)
    a = torch.sigmoid(2 + torch.randn(shape, generator=g))
    b = torch.randn(shape, generator=g) if with_b else None
    x = torch.randn(shape, generator=g)
    h0 = torch.randn(ends, generator=g)
    to = lambda t, d: None if t is None else t.to(d).to(device)
    return to(a, gate), to(x, dt), to(b, gate), h0.to(device)


def _np(t):
    return None if t is None else f64(t)


def _close(got, want, bound, dt, what):
    """got within bound * 2^-24 and the output's own rounding of want."""
    got = f64(got)
    tol = U * bound
    tol = tol + _half_step(dt) * (np.abs(want) + tol)
    # (the smallest bf16 / fp32 numbers: flushing is not allowed, rounding is)
    bad = ~(np.abs(got - want) <= tol + 1e-38)
    assert not bad.any(), (what, np.argwhere(bad)[:3], np.abs(got - want)[bad][:3], tol[bad][:3])


def _check_forward(a, x, b, h0, y, h, ranges):
    """ranges: (index of arrays, row of h0) per sequence."""
    for rows, s in ranges:
        args = [_np(t[rows]) if t is not None else None for t in (a, x, b)] + [_np(h0[s])]
        yr, hr = ref.forward(*args)
        by, bh = ref.forward_bound(*args)
        _close(y[rows], yr, by, x.dtype, 'y')
        _close(h[s], hr, bh, F32, 'h')


def _check_backward(a, x, b, h0, y, dy, dh, g, ranges):
    for rows, s in ranges:
        sl = lambda t: _np(t[rows]) if t is not None else None
        dar, dxr, dbr, d0r = ref.backward(sl(a), sl(x), sl(y), sl(dy), sl(b), _np(h0[s]), _np(dh[s]))
        bg, bc = ref.backward_bound(sl(a), sl(dy), _np(dh[s]))
        before = np.concatenate([_np(h0[s])[None], sl(y)[:-1]])[:bg.shape[0]]
        _close(g['a'][rows], dar, 2 * bg * np.abs(before), a.dtype, 'da')
        one = np.ones_like(bg) if b is None else np.abs(sl(b))
        _close(g['x'][rows], dxr, 2 * bg * one, x.dtype, 'dx')
        if b is not None:
            _close(g['b'][rows], dbr, 2 * bg * np.abs(sl(x)), b.dtype, 'db')
        _close(g['h0'][s], d0r, 2 * bc, F32, 'dh0')


@pytest.mark.parametrize("gate,dt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("with_b", [False, True])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 0, 5), (3, 2, 64), (2, 63, 65), (1, 128, 130),
                                   (2, 129, 62), (1, 1025, 33)])
def test_forward_and_backward(gate, dt, with_b, B, T, D):
    a, x, b, h0 = _inputs((B, T, D), (B, D), gate, dt, with_b, seed=B * 100 + T + D)
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    ranges = [(s, s) for s in range(B)]
    _check_forward(a, x, b, h0, y, h, ranges)
    gen = torch.Generator().manual_seed(7)
    dy = torch.randn((B, T, D), generator=gen).to(dt).cuda()
    dh = torch.randn((B, D), generator=gen).cuda()
    g = kdn.kdn_linear_scan_backward(a, x if with_b else None, y, dy, b=b, h0=h0, dh_T=dh)
    _check_backward(a, x, b, h0, y, dy, dh, g, ranges)


def _packed(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device='cuda')


LENGTHS = [[5], [1, 1, 1], [0, 3, 0, 0, 200, 1, 0], [64, 64, 128, 127, 1, 129],
           [700, 0, 1, 2, 900, 16, 15, 17], list(range(40)), [1] * 300]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("gate,dt,with_b,D", [(F32, F32, True, 66), (F32, BF16, False, 63),
                                              (BF16, BF16, True, 128)])
def test_packed_forward_and_backward(lengths, gate, dt, with_b, D):
    N, T = len(lengths), sum(lengths)
    pad = 37  # rows behind the last sequence
    a, x, b, h0 = _inputs((T + pad, D), (N, D), gate, dt, with_b, seed=N + T)
    cu = _packed(lengths)
    ends = np.cumsum(lengths)
    ranges = [(slice(int(e - n), int(e)), s) for s, (n, e) in enumerate(zip(lengths, ends))]
    ws = torch.empty(kdn.kdn_linear_scan_workspace_size(1, T + pad, D), dtype=torch.uint8,
                     device='cuda')
    y = torch.full((T + pad, D), 3.0, dtype=dt, device='cuda')
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0, cu_seqlens=cu, y=y, workspace=ws)
    assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_OK
    _check_forward(a, x, b, h0, y, h, ranges)
    assert bool((y[T:] == 3).all())
    gen = torch.Generator().manual_seed(8)
    dy = torch.randn((T + pad, D), generator=gen).to(dt).cuda()
    dh = torch.randn((N, D), generator=gen).cuda()
    outs = {k: torch.full((T + pad, D), 3.0, dtype=d, device='cuda')
            for k, d in (('da', gate), ('dx', dt), ('db', gate))}
    if not with_b:
        outs.pop('db')
    g = kdn.kdn_linear_scan_backward(a, x, y, dy, b=b, h0=h0, dh_T=dh, cu_seqlens=cu,
                                     workspace=ws, **outs)
    assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_OK
    _check_backward(a, x, b, h0, y, dy, dh, g, ranges)
    for t in outs.values():
        assert bool((t[T:] == 3).all())


def test_packed_equals_separate_calls_without_optional_inputs():
    lengths, D = [150, 0, 33], 64
    a, x, _, _ = _inputs((183, D), (3, D), F32, F32, False, seed=4)
    y, h = kdn.kdn_linear_scan_forward(a, x, cu_seqlens=_packed(lengths))
    y1, h1 = kdn.kdn_linear_scan_forward(a[None, :150], x[None, :150])
    torch.testing.assert_close(y[:150], y1[0], rtol=1e-5, atol=1e-6)
    torch.testing.assert_close(h[0], h1[0], rtol=1e-5, atol=1e-6)
    assert bool((h[1] == 0).all())
    g = kdn.kdn_linear_scan_backward(a, None, y, x, cu_seqlens=_packed(lengths))
    assert bool((g['h0'][1] == 0).all())


def test_an_infinity_stays_in_its_sequence():
    """An infinity or NaN in one packed sequence, batch entry or channel does
    not reach another."""
    D, lengths = 70, [300, 200, 0, 400]
    a, x, _, h0 = _inputs((900, D), (4, D), F32, F32, False, seed=5)
    x[10, 3], x[20, 4], a[30, 5] = float('inf'), float('nan'), float('inf')
    cu = _packed(lengths)
    y, h = kdn.kdn_linear_scan_forward(a, x, h0=h0, cu_seqlens=cu)
    assert not torch.isfinite(y[299, 3:5]).any()
    assert torch.isfinite(y[300:]).all() and torch.isfinite(h[1:]).all()
    keep = [c for c in range(D) if c not in (3, 4, 5)]
    assert torch.isfinite(y[:, keep]).all()
    dy = torch.randn(900, D, device='cuda')
    dy[600, 7], dy[599, 8] = float('nan'), float('inf')   # (in the last sequence)
    g = kdn.kdn_linear_scan_backward(a, None, torch.nan_to_num(y, 0., 0., 0.), dy, h0=h0,
                                     cu_seqlens=cu)
    assert torch.isfinite(g['x'][300:500]).all() and torch.isfinite(g['h0'][1]).all()
    xb = torch.randn(2, 700, D, device='cuda')
    ab = torch.rand(2, 700, D, device='cuda')
    xb[0, 5] = float('inf')
    yb, hb = kdn.kdn_linear_scan_forward(ab, xb)
    assert torch.isfinite(yb[1]).all() and torch.isfinite(hb[1]).all()


def test_gates_of_zero_one_and_minus_one():
    """a = 0 forgets, a = 1 sums, negative gates alternate; also packed, where a
    gate of -0.0 is an ordinary zero."""
    T, D = 500, 64
    x = torch.randn(T, D, device='cuda')
    for v in (0.0, -0.0, 1.0, -1.0):
        a = torch.full((T, D), v, device='cuda')
        h0 = torch.randn(2, D, device='cuda')
        for cu in (None, _packed([200, 300])):
            if cu is None:
                y, h = kdn.kdn_linear_scan_forward(a[None], x[None], h0=h0[:1])
                _check_forward(a[None], x[None], None, h0, y, h, [(0, 0)])
            else:
                y, h = kdn.kdn_linear_scan_forward(a, x, h0=h0, cu_seqlens=cu)
                _check_forward(a, x, None, h0, y, h, [(slice(0, 200), 0), (slice(200, 500), 1)])


def test_long_sequence_and_repeatability():
    """70001 steps; the same call gives the same bits however its tiles met."""
    T, D = 70001, 192
    a, x, b, h0 = _inputs((1, T, D), (1, D), F32, F32, True, seed=6)
    a = a ** 0.01  # long memories
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    cols = [0, 63, 64, 190]
    _check_forward(a[..., cols], x[..., cols], b[..., cols], h0[:, cols], y[..., cols], h[:, cols],
                   [(0, 0)])
    dy = torch.randn_like(y)
    g = kdn.kdn_linear_scan_backward(a, x, y, dy, b=b, h0=h0)
    for _ in range(5):
        y2, h2 = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        g2 = kdn.kdn_linear_scan_backward(a, x, y, dy, b=b, h0=h0)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_state_in_place_and_handoff_to_steps():
    """h_out may alias h0 (dh0 dh_T); a prefill, then steps, is one scan."""
    B, T, D = 3, 400, 100
    a, x, b, h0 = _inputs((B, T, D), (B, D), F32, BF16, True, seed=9)
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    state = h0.clone()
    y1, _ = kdn.kdn_linear_scan_forward(a[:, :397].contiguous(), x[:, :397].contiguous(),
                                        b=b[:, :397].contiguous(), h0=state, h_out=state)
    assert torch.equal(y1, y[:, :397])
    for t in range(397, T):
        yt = kdn.kdn_linear_scan_step(a[:, t].contiguous(), x[:, t].contiguous(), state,
                                      b=b[:, t].contiguous())
        _close(yt, f64(y[:, t]), 64 * np.abs(f64(y[:, t])) + 64, BF16, 'step')
    torch.testing.assert_close(state, h, rtol=1e-5, atol=1e-6)
    dh = torch.randn(B, D, device='cuda')
    dy = torch.randn_like(y)
    g = kdn.kdn_linear_scan_backward(a, x, y, dy, b=b, h0=h0, dh_T=dh)
    g2 = kdn.kdn_linear_scan_backward(a, x, y, dy, b=b, h0=h0, dh_T=dh, dh0=dh)
    assert torch.equal(g['h0'], g2['h0']) and g2['h0'].data_ptr() == dh.data_ptr()


@pytest.mark.parametrize("gate,dt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 3), (2, 64), (3, 37), (300, 1025)])
def test_step(gate, dt, B, D):
    for with_b in (False, True):
        a, x, b, h0 = _inputs((B, D), (B, D), gate, dt, with_b, seed=B + D)
        h = h0.clone()
        y = kdn.kdn_linear_scan_step(a, x, h, b=b)
        u = f64(x) if b is None else f64(x) * f64(b)
        want = f64(a) * f64(h0) + u
        mag = np.abs(f64(a) * f64(h0)) + 2 * np.abs(u) + np.abs(want)
        _close(h, want, mag, F32, 'h')
        _close(y, want, mag, dt, 'y')


def test_bad_offsets_are_reported_and_harmless():
    T, D = 300, 64
    a, x, _, _ = _inputs((T, D), (3, D), F32, F32, False, seed=10)
    for offsets in ([0, 200, 100, 300], [5, 10, 20, 300], [0, 100, 200, 400], [0, -7, 3, 300],
                    [0, 2 ** 31 - 1, 5, -2 ** 31], [400, 500, 600, 700]):
        for rows in (T, 40):  # several tiles and one
            cu = torch.tensor(offsets, dtype=torch.int32, device='cuda')
            ws = torch.empty(kdn.kdn_linear_scan_workspace_size(1, rows, D), dtype=torch.uint8,
                             device='cuda')
            room = torch.full((rows + 64, D), 3.0, device='cuda')  # rows on both sides
            y = room[32:32 + rows]
            kdn.kdn_linear_scan_forward(a[:rows], x[:rows], cu_seqlens=cu, y=y, workspace=ws)
            assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_ERR_INVALID_ARG
            assert bool((room[:32] == 3).all()) and bool((room[32 + rows:] == 3).all())
            kdn.kdn_linear_scan_backward(a[:rows], None, a[:rows], x[:rows], cu_seqlens=cu, dx=y,
                                         workspace=ws)
            assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_ERR_INVALID_ARG
            assert bool((room[:32] == 3).all()) and bool((room[32 + rows:] == 3).all())


def test_streams_and_a_replayed_graph():
    """Calls on two streams at once, and a captured forward and backward
    replayed on new inputs, give what eager calls give."""
    B, T, D = 2, 1500, 192
    sets = [_inputs((B, T, D), (B, D), F32, BF16, True, seed=20 + i) for i in range(4)]
    want = [kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0) for a, x, b, h0 in sets]
    grads = [kdn.kdn_linear_scan_backward(a, x, y, x, b=b, h0=h0, dh_T=h0)
             for (a, x, b, h0), (y, _) in zip(sets, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for s, (a, x, b, h0) in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append(kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0))
    torch.cuda.synchronize()
    for (y, h), (y2, h2) in zip(want, got):
        assert torch.equal(y, y2) and torch.equal(h, h2)
    a, x, b, h0 = (t.clone() for t in sets[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
        g = kdn.kdn_linear_scan_backward(a, x, y, x, b=b, h0=h0, dh_T=h0)
    for i in (1, 2, 1):
        for dst, src in zip((a, x, b, h0), sets[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(h, want[i][1])
        assert all(torch.equal(g[k], grads[i][k]) for k in g)


@pytest.mark.parametrize("gate,dt,with_b", [(F32, F32, True), (F32, BF16, False), (BF16, BF16, True),
                                            (BF16, F32, False)])
@pytest.mark.parametrize("D", [8, 9, 24, 57, 64, 71, 136, 201])
@pytest.mark.parametrize("B,T", [(1, 7), (1, 8), (3, 9), (2, 64), (3, 65), (1, 127), (2, 515)])
def test_rows_of_whole_pieces_and_others(gate, dt, with_b, D, B, T):
    """Rows on 16-byte boundaries and not, a last line of fewer than eight rows,
    tiles that end a sequence early."""
    a, x, b, h0 = _inputs((B, T, D), (B, D), gate, dt, with_b, seed=B * 1000 + T + D)
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    _check_forward(a, x, b, h0, y, h, [(s, s) for s in range(B)])
    gen = torch.Generator().manual_seed(11)
    dy = torch.randn((B, T, D), generator=gen).to(dt).cuda()
    dh = torch.randn((B, D), generator=gen).cuda()
    g = kdn.kdn_linear_scan_backward(a, x if with_b else None, y, dy, b=b, h0=h0, dh_T=dh)
    _check_backward(a, x, b, h0, y, dy, dh, g, [(s, s) for s in range(B)])


@pytest.mark.parametrize("B,T,D", [(700, 70, 64), (90, 150, 515), (1, 3000, 200), (2, 1200, 640)])
def test_many_columns_and_few(B, T, D):
    """More columns of 64 channels than run at once, and so few that several
    blocks share one."""
    a, x, b, h0 = _inputs((B, T, D), (B, D), F32, F32, True, seed=B)
    y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0)
    some = sorted({0, B // 2, B - 1})
    _check_forward(a, x, b, h0, y, h, [(s, s) for s in some])
    dh = torch.randn((B, D), device='cuda')
    g = kdn.kdn_linear_scan_backward(a, x, y, x, b=b, h0=h0, dh_T=dh)
    _check_backward(a, x, b, h0, y, x, dh, g, [(s, s) for s in some])
    # every entry by itself gives the same bits
    for s in some:
        a1, x1, b1, y0, s1, d1 = (t[s:s + 1].clone() for t in (a, x, b, y, h0, dh))
        y1, h1 = kdn.kdn_linear_scan_forward(a1, x1, b=b1, h0=s1)
        assert torch.equal(y1, y0) and torch.equal(h1, h[s:s + 1])
        g1 = kdn.kdn_linear_scan_backward(a1, x1, y0, x1, b=b1, h0=s1, dh_T=d1)
        assert all(torch.equal(g1[k], g[k][s:s + 1]) for k in g)


@pytest.mark.parametrize("D", [64, 67, 320, 2048])
@pytest.mark.parametrize("T", [50, 300, 1000, 2500])
def test_states_in_place(D, T):
    """h_out on h0 and dh0 on dh_T, dense and packed, give the bits of separate
    memory."""
    a, x, b, h0 = _inputs((2, T, D), (2, D), F32, BF16, True, seed=T + D)
    cu = _packed([T // 3, 0, T - T // 3 - 5, 5])
    states = torch.randn(4, D, device='cuda')
    for args, s0, kw in (((a, x), h0, {}), ((a[0], x[0]), states, dict(cu_seqlens=cu))):
        bb = b if not kw else b[0]
        y, h = kdn.kdn_linear_scan_forward(*args, b=bb, h0=s0, **kw)
        g = kdn.kdn_linear_scan_backward(*args, y, args[1], b=bb, h0=s0, dh_T=s0, **kw)
        for _ in range(3):
            st = s0.clone()
            y2, h2 = kdn.kdn_linear_scan_forward(*args, b=bb, h0=st, h_out=st, **kw)
            d2 = s0.clone()
            g2 = kdn.kdn_linear_scan_backward(*args, y, args[1], b=bb, h0=s0, dh_T=d2, dh0=d2, **kw)
            if kw:  # (the two may run in different tiles)
                torch.testing.assert_close(h2, h, rtol=1e-5, atol=1e-5)
                torch.testing.assert_close(y2.float(), y.float(), rtol=2 ** -7, atol=1e-5)
                torch.testing.assert_close(g2['h0'], g['h0'], rtol=1e-5, atol=1e-5)
            else:
                assert torch.equal(y2, y) and torch.equal(h2, h)
                assert all(torch.equal(g2[k], g[k]) for k in g)


def test_packed_boundaries_at_every_place():
    """Sequences of 1 to 40 steps, and pairs of boundaries at every distance
    within a warp's steps."""
    D = 64
    for lengths in ([n for n in range(1, 41)], [n for n in range(40, 0, -1)] + [0, 0, 64, 0],
                    [16] * 20, [8, 24, 1, 31, 2, 30, 15, 17] * 6):
        N, T = len(lengths), sum(lengths)
        for gate, dt, width in ((F32, F32, D), (BF16, BF16, D), (F32, BF16, 37)):
            a, x, b, h0 = _inputs((T, width), (N, width), gate, dt, True, seed=N)
            ends = np.cumsum(lengths)
            ranges = [(slice(int(e - n), int(e)), s) for s, (n, e) in enumerate(zip(lengths, ends))]
            y, h = kdn.kdn_linear_scan_forward(a, x, b=b, h0=h0, cu_seqlens=_packed(lengths))
            _check_forward(a, x, b, h0, y, h, ranges)
            dh = torch.randn_like(h)
            g = kdn.kdn_linear_scan_backward(a, x, y, x, b=b, h0=h0, dh_T=dh,
                                             cu_seqlens=_packed(lengths))
            _check_backward(a, x, b, h0, y, x, dh, g, ranges)


def test_refusals():
    a, x, b, h0 = _inputs((2, 30, 64), (2, 64), F32, BF16, True, seed=1)
    with pytest.raises(TypeError):
        kdn.kdn_linear_scan_forward(a, x.half())
    with pytest.raises(TypeError):
        kdn.kdn_linear_scan_forward(a, x, b=b.bfloat16())
    with pytest.raises(ValueError):
        kdn.kdn_linear_scan_forward(a, x[:, :20])
    with pytest.raises(ValueError):
        kdn.kdn_linear_scan_forward(a.transpose(0, 1), x.transpose(0, 1))
    with pytest.raises(ValueError):
        kdn.kdn_linear_scan_forward(a, x, h0=h0[:1])
    with pytest.raises(ValueError):
        kdn.kdn_linear_scan_forward(a, x, cu_seqlens=torch.zeros(2, dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        kdn.kdn_linear_scan_backward(a, None, x, x, b=b)
    with pytest.raises(kdn.KdnError) as e:
        kdn.kdn_linear_scan_forward(a, x, workspace=torch.empty(64, dtype=torch.uint8).cuda())
    assert e.value.status == kdn.KDN_ERR_WORKSPACE
