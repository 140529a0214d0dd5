"""Pins of the recurrence, norm and 8-bit oracles against facts that do not
reuse their formulas: closed forms, finite differences of the forward, the
information-form filter's mean recursion, torch's e4m3 conversion."""
import numpy as np
import torch

from oracle import fp8_ref, kla_ref, linear_scan_ref, rmsnorm_ref


def test_recurrence_is_a_weighted_sum():
    """h_T = sum_s (prod of the later gates) b_s x_s + (prod of all) h0."""
    rng = np.random.default_rng(0)
    T, D = 9, 4
    a, b, x = rng.uniform(0.2, 1, (T, D)), rng.standard_normal((T, D)), rng.standard_normal((T, D))
    h0 = rng.standard_normal(D)
    y, h = linear_scan_ref.forward(a, x, b, h0)
    want = np.prod(a, 0) * h0 + sum(np.prod(a[s + 1:], 0) * b[s] * x[s] for s in range(T))
    np.testing.assert_allclose(h, want, rtol=1e-12)
    np.testing.assert_allclose(y[-1], h)


def test_recurrence_is_the_filter_mean_given_its_gates():
    """One row of the information-form filter's memory: forget gate f and
    write gate u per key dimension, value v."""
    rng = np.random.default_rng(1)
    T, D = 12, 6
    k = rng.standard_normal((T, D))
    a, r = rng.uniform(0.5, 1, T), rng.uniform(0.3, 2, T)
    w, v = rng.uniform(0.05, 0.6, (T, D)), rng.standard_normal(T)
    f, u, lam = np.empty((T, D)), np.empty((T, D)), np.ones(D)
    for t in range(T):
        prior, post = kla_ref.precision_step(lam, a[t], w[t], r[t], k[t])
        f[t], u[t], lam = a[t] * prior / post, k[t] / r[t] / post, post
    _, S, _ = kla_ref.kla_forward(k[None, :, None], k[None, :, None], v[None, :, None, None],
                                  a[None, :, None], w[None, :, None], r[None, :, None])
    _, h = linear_scan_ref.forward(f, np.repeat(v[:, None], D, 1), u)
    np.testing.assert_allclose(h, S[0, 0, 0], rtol=1e-10)


def _central(f, v, eps=1e-6):
    g = np.empty_like(v)
    for i in np.ndindex(v.shape):
        p, m = v.copy(), v.copy()
        p[i] += eps
        m[i] -= eps
        g[i] = (f(p) - f(m)) / (2 * eps)
    return g


def test_recurrence_gradient_is_the_finite_difference():
    rng = np.random.default_rng(2)
    T, D = 6, 3
    v = dict(a=rng.uniform(0.2, 1, (T, D)), x=rng.standard_normal((T, D)),
             b=rng.standard_normal((T, D)), h0=rng.standard_normal(D))
    dy, dh = rng.standard_normal((T, D)), rng.standard_normal(D)

    def loss(**kw):
        y, h = linear_scan_ref.forward(**{**v, **kw})
        return (y * dy).sum() + (h * dh).sum()

    y, _ = linear_scan_ref.forward(**v)
    got = dict(zip(('a', 'x', 'b', 'h0'),
                   linear_scan_ref.backward(v['a'], v['x'], y, dy, v['b'], v['h0'], dh)))
    for name in v:
        np.testing.assert_allclose(got[name], _central(lambda z: loss(**{name: z}), v[name]),
                                   rtol=1e-6, atol=1e-7, err_msg=name)


def test_norm_gradient_is_the_finite_difference():
    rng = np.random.default_rng(3)
    h, w, dy = rng.standard_normal((3, 7)), rng.uniform(0.5, 2, 7), rng.standard_normal((3, 7))
    through = rng.standard_normal((3, 7))
    f = lambda hh, ww: (rmsnorm_ref.forward(hh, ww, 0.01) * dy).sum() + (hh * through).sum()
    d, dw = rmsnorm_ref.backward(h, w, dy, 0.01, through)
    np.testing.assert_allclose(d, _central(lambda z: f(z, w), h), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, _central(lambda z: f(h, z), w), rtol=1e-6, atol=1e-8)
    # unit root mean square, and nothing left along h without eps
    y = rmsnorm_ref.forward(h, np.ones(7), 0.0)
    np.testing.assert_allclose((y * y).mean(1), 1.0, rtol=1e-12)
    d0, _ = rmsnorm_ref.backward(h, np.ones(7), dy, 0.0)
    np.testing.assert_allclose((d0 * h).sum(1), 0.0, atol=1e-12)


def test_e4m3_is_torchs():
    """All finite codes are fixed points, and random values, halfway points
    between neighbours among them, round as torch's conversion does."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    codes = np.unique(codes[np.isfinite(codes)])
    np.testing.assert_array_equal(fp8_ref.e4m3(codes), codes)
    rng = np.random.default_rng(4)
    v = np.concatenate([(codes[1:] + codes[:-1]) / 2, rng.uniform(-448, 448, 4096),
                        rng.standard_normal(4096) * 2.0 ** rng.integers(-12, 8, 4096)])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8_ref.e4m3(v), want)


def test_blocks_and_their_product():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((130, 200)), rng.standard_normal((150, 200))
    sx, sw = fp8_ref.scales(x), fp8_ref.scales(w, True)
    assert sx.shape == (130, 2) and sw.shape == (2, 2)
    assert sw[1, 1] == np.abs(w[128:, 128:]).max() / 448
    qx = fp8_ref.e4m3(x / fp8_ref.spread(sx, *x.shape))
    qw = fp8_ref.e4m3(w / fp8_ref.spread(sw, *w.shape, True))
    assert np.abs(qx).max() == 448.0
    # e4m3 keeps 4 significant bits: within half a step, 2^-4, of each value
    # (values below the normal range: half of 2^-9 scales)
    err = np.abs(qx * fp8_ref.spread(sx, *x.shape) - x)
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * fp8_ref.spread(sx, *x.shape))
            * (1 + 1e-12)).all()
    out, _ = fp8_ref.matmul(qx, sx, qw, sw, True)
    want = sum(sx[7, k] * sw[1, k] * (qx[7, 128 * k:128 * k + 128] * qw[140, 128 * k:128 * k + 128])
               .sum() for k in range(2))
    np.testing.assert_allclose(out[7, 140], want, rtol=1e-12)
