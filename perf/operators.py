"""The gated linear recurrence, the residual RMS norm and the 8-bit projection: their cases, their plain forms in torch,
and the framework's calls.

Shapes follow the library's workloads: a model width of 2048 (16 heads of 128), 32768 tokens (8 x 4096, or packed sequences),
one sequence of 65536, and decoding.  Matrices in e4m3 have a scale for each block of 128 along their rows (`1x128`) or, for
weights, for each 128 x 128 tile; their rows start on 16-byte boundaries.
"""
import math

import torch

own = False  # False: the plain forms; True: the framework's calls

BLOCK = 128                # length of a scaled block
E4M3_MAX = 448.0           # largest e4m3 value
AMAX_FLOOR = 2.0 ** -100   # a block's largest magnitude is taken as at least this
EPS = 1e-6

TYPES = {'f32': torch.float32, 'bf16': torch.bfloat16, 'e4m3': torch.float8_e4m3fn}
SIZE = {'f32': 4, 'bf16': 2, 'e4m3': 1}


def listed():
    return [
        # one token of a small serving batch
        dict(name='scan step', op='scan_step', B=16, D=2048, gate='f32', dtype='bf16', write_gate=True),
        # a training batch's forward: 8 sequences of 4096, decays in fp32
        dict(name='scan forward', op='scan_forward', B=8, T=4096, D=2048, gate='f32', dtype='bf16',
             write_gate=False, packed=False),
        # one long document, both gates in bf16
        dict(name='scan forward long', op='scan_forward', B=1, T=65536, D=2048, gate='bf16', dtype='bf16',
             write_gate=True, packed=False),
        # a training step over 41 packed sequences
        dict(name='scan backward packed', op='scan_backward', B=41, T=32768, D=2048, gate='f32', dtype='bf16',
             write_gate=True, packed=True),
        # decoding: the norm between two layers
        dict(name='norm decode', op='norm_forward', rows=256, D=2048, x='bf16', stream='bf16', out='bf16'),
        # a mixer's fp32 output into the residual stream, and 8 bits for the next projection
        dict(name='norm to 8 bits', op='norm_forward', rows=32768, D=2048, x='f32', stream='bf16', out='e4m3'),
        # its backward: the mixer's output gradient is fp32
        dict(name='norm backward', op='norm_backward', rows=32768, D=2048, x='f32', stream='bf16', out='bf16'),
        # a mixer's output before the output projection
        dict(name='quantize rows', op='quantize', rows=32768, D=2048, x='f32', tile=False, transpose=False),
        # the activations of a ragged batch, transposed for the weight gradient
        dict(name='quantize transposed', op='quantize', rows=32749, D=1000, x='bf16', tile=False, transpose=True),
        # decoding: a projection of 8 rows
        dict(name='project decode', op='matmul', M=8, N=2048, K=2048, tile=True, out='bf16'),
        # training: a projection of a whole batch
        dict(name='project', op='matmul', M=32768, N=2048, K=2048, tile=True, out='bf16'),
        # a weight gradient: the sum runs over a ragged batch's tokens
        dict(name='weight gradient', op='matmul', M=2048, N=2048, K=32749, tile=False, out='f32'),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(['scan_step', 'scan_forward', 'scan_forward', 'scan_backward', 'norm_forward', 'norm_forward',
                     'norm_backward', 'quantize', 'matmul', 'matmul', 'matmul'])
    coin = lambda: rng.random() < 0.5
    if op == 'scan_step':
        return dict(op=op, B=_log_int(rng, 1, 512), D=_log_int(rng, 16, 8192), gate=rng.choice(['f32', 'bf16']),
                    dtype=rng.choice(['f32', 'bf16']), write_gate=coin())
    if op in ('scan_forward', 'scan_backward'):
        D = _log_int(rng, 16, 4096)
        B = _log_int(rng, 1, 64)
        packed = coin()
        most = (1 << 26) // D
        T = _log_int(rng, 1, min(65536, max(1, most if packed else most // B)))
        return dict(op=op, B=B, T=T, D=D, gate=rng.choice(['f32', 'bf16']), dtype=rng.choice(['f32', 'bf16']),
                    write_gate=coin(), packed=packed)
    if op in ('norm_forward', 'norm_backward'):
        D = _log_int(rng, 64, 16384)
        D = D if rng.random() < 0.25 else max(64, D // 8 * 8)
        return dict(op=op, rows=_log_int(rng, 1, (1 << 26) // D), D=D, x=rng.choice(['f32', 'bf16']),
                    stream=rng.choice(['none', 'f32', 'bf16']),
                    out=rng.choice(['bf16', 'f32', 'e4m3'] if op == 'norm_forward' else ['bf16', 'f32']))
    if op == 'quantize':
        D = _log_int(rng, 64, 8192)
        return dict(op=op, rows=_log_int(rng, 1, (1 << 26) // D), D=D, x=rng.choice(['f32', 'bf16']), tile=coin(),
                    transpose=coin())
    N, K = _log_int(rng, 16, 8192), _log_int(rng, 64, 8192)
    return dict(op=op, M=_log_int(rng, 1, min(32768, (1 << 36) // (N * K))), N=N, K=K, tile=rng.random() < 0.7,
                out=rng.choice(['bf16', 'f32']))


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device='cuda', dtype=torch.float32)


def _offsets(B, T, seed):
    """B lengths that are log-uniform over a factor of 64, and sum to T (a few may be empty when T is small)."""
    g = torch.Generator().manual_seed(int(seed) + 1)
    w = torch.exp(torch.rand(B, generator=g, dtype=torch.float64) * math.log(64.0))
    ends = (torch.cumsum(w, 0) / w.sum() * T).round().to(torch.int32)
    ends[-1] = T
    return torch.cat([torch.zeros(1, dtype=torch.int32), ends]).cuda()


def _codes(g, rows, cols, tile):
    """A random matrix in e4m3 and its scales, its rows padded to 16 bytes."""
    x = _normal(g, rows, cols)
    if tile:
        x *= cols ** -0.5
    q, s = _quantize(x, tile)
    pad = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.float8_e4m3fn, device='cuda')
    pad.view(torch.uint8)[:, :cols] = q.view(torch.uint8)
    return pad[:, :cols], s


def prepare(case, seed):
    g = torch.Generator(device='cuda').manual_seed(int(seed))
    c, op, st = case, case['op'], dict(case=case)
    if op.startswith('scan'):
        B, D = c['B'], c['D']
        gd, xd = TYPES[c['gate']], TYPES[c['dtype']]
        shape = (B, D) if op == 'scan_step' else (c['T'], D) if c['packed'] else (B, c['T'], D)
        a = torch.sigmoid(2 + 0.5 * _normal(g, *shape))
        b = torch.sqrt(1 - a * a) if c['write_gate'] else None
        st.update(a=a.to(gd), b=None if b is None else b.to(gd), x=_normal(g, *shape).to(xd), h0=_normal(g, B, D), cu=None)
        if op != 'scan_step' and c['packed']:
            st['cu'] = _offsets(B, c['T'], seed)
        if op == 'scan_step':
            st['h'] = st['h0'].clone()
        if op == 'scan_backward':
            st['y'] = _scan_forward(st['a'], st['b'], st['x'], st['h0'], st['cu'])[0]
            st['dy'] = _normal(g, *shape).to(xd)
            st['dh'] = _normal(g, B, D)
    elif op.startswith('norm'):
        n, D = c['rows'], c['D']
        w = 1 + 0.1 * _normal(g, D)
        if op == 'norm_forward':
            st.update(w=w, x=_normal(g, n, D).to(TYPES[c['x']]),
                      res=None if c['stream'] == 'none' else (2 * _normal(g, n, D)).to(TYPES[c['stream']]))
        else:
            stream = TYPES[c['x'] if c['stream'] == 'none' else c['stream']]
            st.update(w=w, h=(2 * _normal(g, n, D)).to(stream), dy=_normal(g, n, D).to(TYPES[c['out']]),
                      dh=None if c['stream'] == 'none' else _normal(g, n, D).to(stream))
    elif op == 'quantize':
        # rows of different sizes, as activations are
        st['x'] = (_normal(g, c['rows'], c['D']) * torch.exp(_normal(g, c['rows'], 1))).to(TYPES[c['x']])
    else:
        st['x'], st['sx'] = _codes(g, c['M'], c['K'], False)
        st['w'], st['sw'] = _codes(g, c['N'], c['K'], c['tile'])
    return st


# ------------------------------------------------------------- plain forms

def _previous(h, h0, cu):
    """h_{t-1} for each t: h moved on by one step, the initial states at the sequences' first steps."""
    if cu is None:
        return torch.cat([h0[:, None], h[:, :-1]], 1) if h.shape[1] else h
    p = torch.cat([h0[:1], h[:-1]], 0)
    start, full = cu[:-1].long(), cu[:-1] < cu[1:]
    p[start[full]] = h0[full]
    return p


def _affine_scan(a, u, dim):
    """All h_t = a_t h_{t-1} + u_t with h before the first step zero: maps composed over distances that double."""
    n, step = a.shape[dim], 1
    a, u = a.clone(), u.clone()
    while step < n:
        late_a, late_u = a.narrow(dim, step, n - step), u.narrow(dim, step, n - step)
        early_a, early_u = a.narrow(dim, 0, n - step), u.narrow(dim, 0, n - step)
        new_u = late_u + late_a * early_u
        new_a = late_a * early_a
        late_u.copy_(new_u)
        late_a.copy_(new_a)
        step *= 2
    return u


def _scan_forward(a, b, x, h0, cu):
    af, u = a.float(), x.float()
    if b is not None:
        u = u * b.float()
    dim = 1 if cu is None else 0
    if a.shape[dim] == 0:
        return x.clone(), h0.clone()
    af, u = af.clone(), u.clone()
    if cu is None:
        u[:, 0] += af[:, 0] * h0
        h = _affine_scan(af, u, 1)
        last = h[:, -1].clone()
    else:  # a sequence's first step takes its own initial state, and nothing of the sequence before
        full = cu[:-1] < cu[1:]
        start = cu[:-1].long()[full]
        u[start] += af[start] * h0[full]
        af[start] = 0
        h = _affine_scan(af, u, 0)
        last = h0.clone()
        last[full] = h[cu[1:].long()[full] - 1]
    return h.to(x.dtype), last


def _scan_backward(a, b, x, h0, cu, y, dy, dh):
    """With c the gradient of the state after a step: g = dy + c, and a g is handed to the step before."""
    af, gy = a.float(), dy.float()
    dim = 1 if cu is None else 0
    gy = gy.clone()
    if cu is None:
        gy[:, -1] += dh
        keep = torch.cat([af[:, 1:], torch.zeros_like(af[:, :1])], 1)
    else:
        full = cu[:-1] < cu[1:]
        end = cu[1:].long()[full] - 1
        gy[end] += dh[full]
        keep = torch.cat([af[1:], torch.zeros_like(af[:1])], 0)
        keep[end] = 0
    g = _affine_scan(keep.flip(dim), gy.flip(dim), dim).flip(dim)
    da = g * _previous(y.float(), h0, cu)
    c0 = af * g
    if cu is None:
        dh0 = c0[:, 0].clone()
    else:
        dh0 = dh.clone()
        dh0[full] = c0[cu[:-1].long()[full]]
    dx = g if b is None else g * b.float()
    out = dict(a=da.to(a.dtype), x=dx.to(x.dtype), h0=dh0)
    if b is not None:
        out['b'] = (g * x.float()).to(b.dtype)
    return out


def _blocks(v, dim):
    """v with its dimension `dim` cut into blocks of 128, zeros behind the end."""
    n = v.shape[dim]
    shape = list(v.shape)
    shape[dim] = -n % BLOCK
    v = torch.cat([v, v.new_zeros(shape)], dim) if shape[dim] else v
    return v.unflatten(dim, (-1, BLOCK))


def _quantize(v, tile):
    """e4m3 codes of an fp32 matrix and their scales: one for each 128 of a row, or for each 128 x 128 tile."""
    rows, cols = v.shape
    cut = _blocks(v, 1)                                     # [rows, kb, 128]
    top = cut.abs().amax(2)                                 # [rows, kb]
    if tile:
        top = _blocks(top, 0).amax(1)                       # [rb, kb]
    s = top.clamp_min(AMAX_FLOOR) / E4M3_MAX
    each = s.repeat_interleave(BLOCK, 0)[:rows] if tile else s
    q = (cut / each[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :cols]
    return q.to(torch.float8_e4m3fn), s


def _norm_forward(x, w, res, out):
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * w
    got = dict(zip(('y', 'scale'), _quantize(y, False))) if out == 'e4m3' else dict(y=y.to(TYPES[out]))
    if res is not None:
        got['h'] = h
    return got


def _norm_backward(h, w, dy, dh, x_type):
    f, g = h.float(), dy.float()
    rs = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    gw = g * w
    d = rs * (gw - f * (rs * rs * (gw * f).mean(1, keepdim=True)))
    if dh is not None:
        d = d + dh.float()
    got = dict(x=d.to(x_type), weight=(g * f * rs).double().sum(0).float())
    if dh is not None:
        got['residual'] = d.to(h.dtype)
    return got


def _matmul(x, sx, w, sw, tile, out):
    xf = (_blocks(x.float(), 1) * sx[:, :, None]).flatten(1)
    each = sw.repeat_interleave(BLOCK, 0)[:w.shape[0]] if tile else sw
    wf = (_blocks(w.float(), 1) * each[:, :, None]).flatten(1)
    return (xf @ wf.t()).to(TYPES[out])


def _plain(st):
    c = st['case']
    op = c['op']
    if op == 'scan_step':
        u = st['x'].float() if st['b'] is None else st['x'].float() * st['b'].float()
        h = st['a'].float() * st['h'] + u
        st['h'].copy_(h)
        return dict(y=h.to(st['x'].dtype), h=st['h'])
    if op == 'scan_forward':
        return dict(zip(('y', 'h'), _scan_forward(st['a'], st['b'], st['x'], st['h0'], st['cu'])))
    if op == 'scan_backward':
        return _scan_backward(st['a'], st['b'], st['x'], st['h0'], st['cu'], st['y'], st['dy'], st['dh'])
    if op == 'norm_forward':
        return _norm_forward(st['x'], st['w'], st['res'], c['out'])
    if op == 'norm_backward':
        return _norm_backward(st['h'], st['w'], st['dy'], st['dh'], TYPES[c['x']])
    if op == 'quantize':
        x = st['x'].float()
        return dict(zip(('q', 'scale'), _quantize(x.t().contiguous() if c['transpose'] else x, c['tile'])))
    return dict(out=_matmul(st['x'], st['sx'], st['w'], st['sw'], c['tile'], c['out']))


def _framework(st):
    from kalman_filter_linear_b200 import kdn
    c = st['case']
    op = c['op']
    if op == 'scan_step':
        return dict(y=kdn.kdn_linear_scan_step(st['a'], st['x'], st['h'], b=st['b']), h=st['h'])
    if op == 'scan_forward':
        return dict(zip(('y', 'h'), kdn.kdn_linear_scan_forward(st['a'], st['x'], b=st['b'], h0=st['h0'],
                                                                cu_seqlens=st['cu'])))
    if op == 'scan_backward':
        return kdn.kdn_linear_scan_backward(st['a'], st['x'], st['y'], st['dy'], b=st['b'], h0=st['h0'], dh_T=st['dh'],
                                            cu_seqlens=st['cu'])
    if op == 'norm_forward':
        y, scale, h = kdn.kdn_rmsnorm_forward(st['x'], st['w'], residual=st['res'], eps=EPS, out_dtype=TYPES[c['out']])
        got = dict(y=y) if scale is None else dict(y=y, scale=scale)
        return got if st['res'] is None else dict(got, h=h)
    if op == 'norm_backward':
        g = kdn.kdn_rmsnorm_backward(st['h'], st['w'], st['dy'], dh=st['dh'], eps=EPS, x_dtype=TYPES[c['x']])
        return g if st['dh'] is not None else dict(x=g['x'], weight=g['weight'])
    if op == 'quantize':
        q, s = kdn.kdn_fp8_quantize(st['x'], tile=c['tile'], transpose=c['transpose'])
        return dict(q=q, scale=s)
    return dict(out=kdn.kdn_fp8_matmul(st['x'], st['sx'], st['w'], st['sw'], out_dtype=TYPES[c['out']]))


def run(state):
    return _framework(state) if own else _plain(state)


# -------------------------------------------------------------------- work

def work(case):
    c, op = case, case['op']
    if op.startswith('scan'):
        g, x, b = SIZE[c['gate']], SIZE[c['dtype']], 1 if c['write_gate'] else 0
        if op == 'scan_step':  # the state is read and written
            n = c['B'] * c['D']
            return dict(bytes=n * (g * (1 + b) + 2 * x + 8), flops=n * (2 + b))
        n = (c['T'] if c['packed'] else c['B'] * c['T']) * c['D']
        ends = c['B'] * c['D'] * 4
        if op == 'scan_forward':
            return dict(bytes=n * (g * (1 + b) + 2 * x) + 2 * ends, flops=n * (2 + b))
        # a, dy, y (b, x) in; da, dx (db) out; h0, dh_T in, dh0 out
        return dict(bytes=n * (2 * g * (1 + b) + x * (3 + b)) + 3 * ends, flops=n * (3 + 2 * b))
    if op == 'norm_forward':
        n, stream = c['rows'] * c['D'], 0 if c['stream'] == 'none' else SIZE[c['stream']]
        scales = 4 * c['rows'] * -(-c['D'] // BLOCK) if c['out'] == 'e4m3' else 0
        return dict(bytes=n * (SIZE[c['x']] + 2 * stream + SIZE[c['out']]) + scales + 4 * c['D'], flops=5 * n)
    if op == 'norm_backward':
        n, stream = c['rows'] * c['D'], c['x'] if c['stream'] == 'none' else c['stream']
        through = 0 if c['stream'] == 'none' else 2 * SIZE[stream]
        return dict(bytes=n * (SIZE[stream] + through + SIZE[c['out']] + SIZE[c['x']]) + 8 * c['D'], flops=10 * n)
    if op == 'quantize':
        rows, cols = (c['D'], c['rows']) if c['transpose'] else (c['rows'], c['D'])
        scales = 4 * -(-cols // BLOCK) * (-(-rows // BLOCK) if c['tile'] else rows)
        return dict(bytes=rows * cols * (SIZE[c['x']] + 1) + scales, flops=3 * rows * cols)
    M, N, K = c['M'], c['N'], c['K']
    kb = -(-K // BLOCK)
    return dict(bytes=M * K + N * K + 4 * kb * (M + (-(-N // BLOCK) if c['tile'] else N)) + M * N * SIZE[c['out']],
                flops=2 * M * N * K)


# ------------------------------------------------------- 64-bit definitions

def _e4m3_64(v):
    """The nearest e4m3 value (ties to the even one) of each double, as a double."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    _, e = torch.frexp(v)                                   # |v| in [2^(e-1), 2^e)
    unit = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / unit) * unit


def _quantize_64(v, tile):
    """Codes and scales of a matrix of doubles, block by block."""
    rows, cols = v.shape
    kb = -(-cols // BLOCK)
    m = torch.zeros((rows, kb * BLOCK), dtype=torch.float64, device=v.device)
    m[:, :cols] = v
    top = m.reshape(rows, kb, BLOCK).abs().max(2).values
    if tile:
        for r in range(0, rows, BLOCK):
            top[r:r + BLOCK] = top[r:r + BLOCK].max(0).values
    s = torch.maximum(top, torch.tensor(AMAX_FLOOR, dtype=torch.float64, device=v.device)) / E4M3_MAX
    q = torch.empty_like(v)
    for k in range(kb):
        part = slice(k * BLOCK, min(cols, (k + 1) * BLOCK))
        q[:, part] = _e4m3_64(v[:, part] / s[:, k:k + 1])
    return q, s[::BLOCK] if tile else s


def _sequences(st):
    c = st['case']
    if st['cu'] is None:
        return None
    cu = st['cu'].tolist()
    return [(cu[i], cu[i + 1]) for i in range(c['B'])]


def exact(case, seed):
    st = prepare(case, seed)
    op = case['op']
    d = lambda t: None if t is None else t.double()
    if op.startswith('scan'):
        a, x, h0 = d(st['a']), d(st['x']), d(st['h0'])
        b = torch.ones_like(a) if st['b'] is None else d(st['b'])
        if op == 'scan_step':
            h = a * h0 + b * x
            return dict(y=h, h=h)
        seqs = _sequences(st)
        if seqs is None:  # steps first: [T, B, D]
            a, x, b = (v.transpose(0, 1) for v in (a, x, b))
            parts = [(0, case['T'], slice(None))]
        else:
            parts = [(lo, hi, i) for i, (lo, hi) in enumerate(seqs)]
        back = (lambda v: v) if seqs is not None else (lambda v: v.transpose(0, 1))
        if op == 'scan_forward':
            y, last = torch.empty_like(x), torch.empty_like(h0)
            for lo, hi, i in parts:
                h = h0[i]
                for t in range(lo, hi):
                    h = torch.addcmul(b[t] * x[t], a[t], h)
                    y[t] = h
                last[i] = h
            return dict(y=back(y), h=last)
        y, dy = (d(st[k]) if seqs is not None else d(st[k]).transpose(0, 1) for k in ('y', 'dy'))
        dh = d(st['dh'])
        gs, before, dh0 = torch.empty_like(a), torch.empty_like(a), torch.empty_like(h0)
        for lo, hi, i in parts:
            carry = dh[i]
            for t in range(hi - 1, lo - 1, -1):
                gs[t] = dy[t] + carry
                carry = a[t] * gs[t]
            if hi > lo:
                before[lo] = h0[i]
                before[lo + 1:hi] = y[lo:hi - 1]
            dh0[i] = carry
        out = dict(a=back(gs * before), x=back(gs * b), h0=dh0)
        if st['b'] is not None:
            out['b'] = back(gs * x)
        return out
    if op == 'norm_forward':
        x, w, res = d(st['x']), d(st['w']), d(st['res'])
        h = x if res is None else (x + res).to(st['res'].dtype).double()
        y = w * h / torch.sqrt((h ** 2).sum(1, keepdim=True) / case['D'] + EPS)
        got = dict(zip(('y', 'scale'), _quantize_64(y, False))) if case['out'] == 'e4m3' else dict(y=y)
        return got if res is None else dict(got, h=h)
    if op == 'norm_backward':
        h, w, dy, dh = d(st['h']), d(st['w']), d(st['dy']), d(st['dh'])
        r = torch.sqrt((h ** 2).sum(1, keepdim=True) / case['D'] + EPS)
        n = h / r
        inner = (dy * w * n).sum(1, keepdim=True) / case['D']
        dx = (dy * w - n * inner) / r
        if dh is None:
            return dict(x=dx, weight=(dy * n).sum(0))
        return dict(x=dx + dh, weight=(dy * n).sum(0), residual=dx + dh)
    if op == 'quantize':
        x = d(st['x'])
        return dict(zip(('q', 'scale'), _quantize_64(x.t().contiguous() if case['transpose'] else x, case['tile'])))
    x, w, sx, sw = d(st['x'].float()), d(st['w'].float()), d(st['sx']), d(st['sw'])
    out = torch.zeros((case['M'], case['N']), dtype=torch.float64, device=x.device)
    for k in range(sx.shape[1]):
        part = slice(k * BLOCK, min(case['K'], (k + 1) * BLOCK))
        col = sw[:, k]
        if case['tile']:
            col = col[torch.arange(case['N'], device=x.device) // BLOCK]
        out += (sx[:, k:k + 1] * x[:, part]) @ (col[:, None] * w[:, part]).t()
    return dict(out=out)
