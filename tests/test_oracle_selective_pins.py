"""Pins of the float64 oracles of the selective scan and the short convolution:
closed forms, the layer's own oracle, library sums, and differences.

A central difference at step h is off by h^2/6 times the third derivative plus
eps f / h: with h = 1e-5 and values of order 1 both are below 1e-9; 1e-6 is asked."""
import numpy as np
import pytest

import oracle

rng = np.random.default_rng


def scan_inputs(B, H, N, G, L, seed):
    g = rng(seed)
    return dict(u=g.normal(size=(B, H, L)), delta=g.normal(size=(B, H, L)),
                Bm=g.normal(size=(B, G, N, L)), Cm=g.normal(size=(B, G, N, L)),
                log_re=g.uniform(0.2, 1.2, (H, N)), D=g.normal(size=H),
                dt_bias=g.normal(size=H), z=g.normal(size=(B, H, L)),
                x0=g.normal(size=(B, H, N)))


def test_constant_steps_are_the_layers_real_modes():
    """Steps of one length and constant B and C: the layer with log_re sqrt(dt) and no phase."""
    g = rng(0)
    B, H, N, L = 2, 3, 4, 30
    u, log_re, W, D = (g.normal(size=s) for s in ((B, H, L), (H, N), N, H))
    dt = 0.3
    delta = np.full((B, H, L), np.log(np.expm1(dt)))
    ones = np.ones((B, 1, N, L))
    y, x = oracle.selective_scan(u, delta, ones, ones * W[None, None, :, None], log_re, D)
    ref = oracle.dlr_recurrence(u, log_re[None] * np.sqrt(dt), np.zeros((1, H, N)),
                                np.broadcast_to(W * dt, (1, H, N)).astype(complex), D[None])
    assert np.allclose(y, ref, rtol=1e-12, atol=1e-12)


def test_one_step_written_out():
    s = scan_inputs(1, 2, 3, 1, 1, 1)
    y, x = oracle.selective_scan(**s)
    for h in range(2):
        v = s["delta"][0, h, 0] + s["dt_bias"][h]
        dt = np.log(1 + np.exp(v))
        xs = [np.exp(-s["log_re"][h, n] ** 2 * dt) * s["x0"][0, h, n]
              + dt * s["Bm"][0, 0, n, 0] * s["u"][0, h, 0] for n in range(3)]
        z = s["z"][0, h, 0]
        out = sum(s["Cm"][0, 0, n, 0] * xs[n] for n in range(3)) + s["D"][h] * s["u"][0, h, 0]
        assert np.allclose(x[0, h], xs, rtol=1e-14)
        assert np.isclose(y[0, h, 0], out * z / (1 + np.exp(-z)), rtol=1e-14)


def test_a_masked_step_changes_nothing_and_groups_are_channels_apart():
    s = scan_inputs(1, 4, 3, 2, 9, 2)
    s["delta"][..., 4] = -np.inf
    y, x = oracle.selective_scan(**s)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    cut = {k: v[..., keep] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in s.items()}
    y2, x2 = oracle.selective_scan(**cut)
    assert np.array_equal(x, x2) and np.array_equal(y[..., keep], y2)
    for g in range(2):
        hs = slice(2 * g, 2 * g + 2)
        one = {k: (v[:, g:g + 1] if k in ("Bm", "Cm") else v[hs] if k in ("log_re", "D", "dt_bias")
                   else v[:, hs]) for k, v in s.items()}
        y3, x3 = oracle.selective_scan(**one)
        assert np.array_equal(y[:, hs], y3) and np.array_equal(x[:, hs], x3)


def test_rows_end_at_their_length_and_parts_continue():
    s = scan_inputs(3, 2, 3, 1, 12, 3)
    lens = [0, 5, 12]
    y, x = oracle.selective_scan(lens=lens, **s)
    cut = lambda d, b, lo, hi: {k: (v[b:b + 1, ..., lo:hi] if k in ("u", "delta", "Bm", "Cm", "z")
                                    else v[b:b + 1] if k == "x0" else v) for k, v in d.items()}
    for b, n in enumerate(lens):
        yy, xx = oracle.selective_scan(**cut(s, b, 0, n))
        assert np.array_equal(y[b, :, :n], yy[0]) and not y[b, :, n:].any()
        assert np.array_equal(x[b], xx[0])
    first = cut(s, 2, 0, 7)
    y1, x1 = oracle.selective_scan(**first)
    rest = cut(s, 2, 7, 12)
    rest["x0"] = x1
    y2, x2 = oracle.selective_scan(**rest)
    assert np.array_equal(np.concatenate([y1, y2], -1)[0], y[2]) and np.array_equal(x2[0], x[2])


@pytest.mark.parametrize("bare", [False, True])
@pytest.mark.parametrize("lens", [None, [0, 3, 6]])
def test_selective_gradients_against_differences(lens, bare):
    s = scan_inputs(3, 4, 2, 2, 6, 4)
    if bare:
        s["z"] = s["D"] = s["dt_bias"] = s["x0"] = None
    g = rng(5)
    dy, dx = g.normal(size=(3, 4, 6)), g.normal(size=(3, 4, 2))

    def f(**kw):
        y, x = oracle.selective_scan(lens=lens, **{**s, **kw})
        return (y * dy).sum() + (x * dx).sum()

    got = oracle.selective_backward(dy=dy, dx=dx, lens=lens, **s)
    for name, key in (("u", "du"), ("delta", "ddelta"), ("z", "dz"), ("Bm", "dB"), ("Cm", "dC"),
                      ("log_re", "dlog_re"), ("D", "dD"), ("dt_bias", "ddt_bias"), ("x0", "dx0")):
        if s[name] is None:
            assert name == "x0" or got[key] is None
            continue
        flat = s[name].ravel()
        for k in range(flat.size):
            e = np.zeros_like(flat)
            e[k] = 1e-5
            e = e.reshape(s[name].shape)
            ref = (f(**{name: s[name] + e}) - f(**{name: s[name] - e})) / 2e-5
            assert abs(ref - got[key].ravel()[k]) < 1e-6, (name, k, ref, got[key].ravel()[k])


def test_convolution_is_the_librarys():
    g = rng(6)
    B, H, K, L = 2, 3, 4, 11
    u, w, b, x0 = (g.normal(size=s) for s in ((B, H, L), (H, K), H, (B, H, K - 1)))
    y, end = oracle.short_conv(u, w, b, False, x0)
    for i in range(B):
        for h in range(H):
            e = np.concatenate([x0[i, h], u[i, h]])
            ref = np.convolve(e, w[h][::-1], mode="valid") + b[h]
            assert np.allclose(y[i, h], ref, rtol=1e-13, atol=1e-13)
            assert np.array_equal(end[i, h], e[-(K - 1):])
    y2, _ = oracle.short_conv(u, w, b, True, x0)
    assert np.allclose(y2, y / (1 + np.exp(-y)), rtol=1e-13)


def test_convolution_in_parts_and_short_rows():
    g = rng(7)
    u, w, x0 = g.normal(size=(2, 2, 9)), g.normal(size=(2, 5)), g.normal(size=(2, 2, 4))
    y, end = oracle.short_conv(u, w, x0=x0)
    y1, mid = oracle.short_conv(u[..., :2], w, x0=x0)
    assert np.array_equal(mid, np.concatenate([x0[..., 2:], u[..., :2]], -1))
    y2, end2 = oracle.short_conv(u[..., 2:], w, x0=mid)
    assert np.array_equal(np.concatenate([y1, y2], -1), y) and np.array_equal(end, end2)
    y3, e3 = oracle.short_conv(u, w, x0=x0, lens=[0, 3])
    assert not y3[0].any() and np.array_equal(e3[0], x0[0])
    assert np.array_equal(y3[1, :, :3], y[1, :, :3]) and not y3[1, :, 3:].any()


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("lens", [None, [0, 2, 6]])
def test_convolution_gradients_against_differences(lens, silu):
    g = rng(8)
    K = 4
    s = dict(u=g.normal(size=(3, 2, 6)), w=g.normal(size=(2, K)), bias=g.normal(size=2),
             x0=g.normal(size=(3, 2, K - 1)))
    dy, dx = g.normal(size=(3, 2, 6)), g.normal(size=(3, 2, K - 1))

    def f(**kw):
        y, x = oracle.short_conv(silu=silu, lens=lens, **{**s, **kw})
        return (y * dy).sum() + (x * dx).sum()

    got = oracle.short_conv_backward(dy=dy, dx=dx, silu=silu, lens=lens, **s)
    for name, key in (("u", "du"), ("w", "dw"), ("bias", "dbias"), ("x0", "dx0")):
        flat = s[name].ravel()
        for k in range(flat.size):
            e = np.zeros_like(flat)
            e[k] = 1e-5
            e = e.reshape(s[name].shape)
            ref = (f(**{name: s[name] + e}) - f(**{name: s[name] - e})) / 2e-5
            assert abs(ref - got[key].ravel()[k]) < 1e-6, (name, k, ref, got[key].ravel()[k])
