"""Pins of the float64 oracles of the gated recurrence, the 8-bit checkpoints
and the residual norm: closed forms, the layer's own oracle, and differences.

A central difference at step h is off by h^2/6 times the third derivative plus
eps f / h: with h = 1e-5 and values of order 1 both are below 1e-9; 1e-6 is asked."""
import numpy as np
import pytest

import oracle

rng = np.random.default_rng


def test_open_gate_is_the_layers_real_mode():
    """sigmoid(r) -> 1: x_t = lambda x + sqrt(1 - lambda^2) sigmoid(i) u with
    lambda = exp(-log_re^2), the layer's recurrence for one real mode."""
    g = rng(0)
    B, H, L = 2, 3, 40
    log_re = g.uniform(0.1, 1.0, H)
    u, i = g.normal(size=(2, B, H, L))
    y, x = oracle.gated_recurrence(u, np.full((B, H, L), 800.0), i, log_re)
    lam = np.exp(-log_re ** 2)
    v = np.sqrt(1 - lam ** 2)[None, :, None] / (1 + np.exp(-i)) * u
    ref = oracle.dlr_recurrence(v, log_re[None, :, None], np.zeros((1, H, 1)),
                                np.ones((1, H, 1), dtype=complex), np.zeros((1, H)))
    assert np.allclose(y, ref, rtol=1e-13, atol=1e-13)
    assert np.allclose(x, ref[..., -1], rtol=1e-13, atol=1e-13)


def test_shut_gate_keeps_the_state_and_zero_decay_drives_nothing():
    g = rng(1)
    u, i = g.normal(size=(2, 1, 2, 9))
    x0 = g.normal(size=(1, 2))
    y, x = oracle.gated_recurrence(u, np.full((1, 2, 9), -800.0), i, [0.5, 1.0], x0)
    assert np.array_equal(y, np.repeat(x0[..., None], 9, -1)) and np.array_equal(x, x0)
    y, _ = oracle.gated_recurrence(u, g.normal(size=(1, 2, 9)), i, [0.0, 0.0], x0)
    assert np.array_equal(y, np.repeat(x0[..., None], 9, -1))


def test_rows_end_at_their_length():
    g = rng(2)
    u, r, i = g.normal(size=(3, 3, 2, 12))
    x0 = g.normal(size=(3, 2))
    lens = [0, 5, 12]
    y, x = oracle.gated_recurrence(u, r, i, [0.4, 0.9], x0, lens)
    for b, n in enumerate(lens):
        yy, xx = oracle.gated_recurrence(u[b:b + 1, :, :n], r[b:b + 1, :, :n], i[b:b + 1, :, :n],
                                         [0.4, 0.9], x0[b:b + 1])
        assert np.array_equal(y[b, :, :n], yy[0]) and not y[b, :, n:].any()
        assert np.array_equal(x[b], xx[0])


@pytest.mark.parametrize("lens", [None, [0, 3, 7]])
def test_gated_gradients_against_differences(lens):
    g = rng(3)
    B, H, L = 3, 2, 7
    v = dict(u=g.normal(size=(B, H, L)), r=g.normal(size=(B, H, L)), i=g.normal(size=(B, H, L)),
             log_re=g.uniform(0.2, 1.2, H), x0=g.normal(size=(B, H)))
    dy, dx = g.normal(size=(B, H, L)), g.normal(size=(B, H))

    def f(**kw):
        y, x = oracle.gated_recurrence(lens=lens, **{**v, **kw})
        return (y * dy).sum() + (x * dx).sum()

    got = dict(zip(("u", "r", "i", "log_re", "x0"), oracle.gated_backward(
        v["u"], v["r"], v["i"], v["log_re"], dy, dx, v["x0"], lens)))
    for name, d in got.items():
        flat = v[name].ravel()
        for k in range(flat.size):
            e = np.zeros_like(flat)
            e[k] = 1e-5
            e = e.reshape(v[name].shape)
            ref = (f(**{name: v[name] + e}) - f(**{name: v[name] - e})) / 2e-5
            assert abs(ref - d.ravel()[k]) < 1e-6, (name, k, ref, d.ravel()[k])


def test_kept_states_do_not_change_the_gradients():
    g = rng(4)
    B, H, L = 1, 2, 1100
    u, r, i, dy = g.normal(size=(4, B, H, L))
    y, _ = oracle.gated_recurrence(u, r, i, [0.1, 0.6])
    starts = np.concatenate([np.zeros((B, H, 1)), y[..., 511::512]], -1)
    a = oracle.gated_backward(u, r, i, [0.1, 0.6], dy)
    b = oracle.gated_backward(u, r, i, [0.1, 0.6], dy, starts=starts)
    assert all(np.array_equal(p, q) for p, q in zip(a, b))


def test_ckpt8_closed_forms():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 2] = 127.0, 0.5, 1.5     # scale 1: halves go to even
    x[0, 64], x[0, 65] = 127.25, 1.0                # past 127: scale 2
    x[0, 128] = -3.0 * 2.0 ** 90                    # a group of two steps: 96 2^85
    x[1, 70] = np.inf
    got = oracle.ckpt8(x)
    assert got[0, 0] == 127.0 and got[0, 1] == 0.0 and got[0, 2] == 2.0
    assert got[0, 64] == 128.0 and got[0, 65] == 0.0  # 63.625 -> 64, 0.5 -> 0
    assert got[0, 128] == -3.0 * 2.0 ** 90
    assert np.isnan(got[1, 64:128]).all() and not got[1, :64].any() and not got[1, 128:].any()
    v = rng(5).normal(size=(3, 200))
    assert np.max(np.abs(oracle.ckpt8(v) - v)) <= np.max(np.abs(v)) / 127.0


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("form", ["all", "no gate", "norm only", "stream only"])
def test_resnorm_gradients_against_differences(layer, form):
    g = rng(6)
    B, H, L = 2, 5, 3
    shape = (B, H, L)
    v = dict(x=g.normal(size=shape), y=g.normal(size=shape) + 0.3, g=g.normal(size=shape),
             w_post=g.normal(size=H), scale=g.normal(size=H), w_pre=g.normal(size=H))
    do, dn = g.normal(size=shape), g.normal(size=shape)
    if form == "no gate":
        v["g"] = None
    if form == "norm only":
        v["y"] = v["g"] = None
    if form == "stream only":
        dn = None

    def f(**kw):
        w = {**v, **kw}
        o = w["x"] if w["y"] is None else oracle.resnorm_stream(
            w["x"], w["y"], w["g"], w["w_post"], w["scale"], layer, 1e-3)
        n = oracle.resnorm_out(o, w["w_pre"], layer, 1e-3)
        return (do * o).sum() + (0.0 if dn is None else (dn * n).sum())

    o = v["x"] if v["y"] is None else oracle.resnorm_stream(v["x"], v["y"], v["g"], v["w_post"],
                                                            v["scale"], layer, 1e-3)
    got = dict(zip(("x", "y", "g", "w_post", "scale", "w_pre"), oracle.resnorm_backward(
        o, v["y"], v["g"], v["w_post"], v["scale"], v["w_pre"], do, dn, layer, 1e-3)))
    for name, d in got.items():
        assert (d is None) == (v[name] is None or (v["y"] is None and name in ("w_post", "scale")))
        if d is None:
            continue
        flat = v[name].ravel()
        for k in range(flat.size):
            e = np.zeros_like(flat)
            e[k] = 1e-5
            e = e.reshape(v[name].shape)
            ref = (f(**{name: v[name] + e}) - f(**{name: v[name] - e})) / 2e-5
            assert abs(ref - d.ravel()[k]) < 1e-6, (name, k, ref, d.ravel()[k])


def test_resnorm_of_one_value_everywhere():
    """A column of equal values: the layer norm is 0, the rms norm 1 (eps = 0)."""
    o = np.full((1, 4, 2), 3.0)
    assert not oracle.resnorm_out(o, np.ones(4), True, 1e-6).any()
    assert np.array_equal(oracle.resnorm_out(o, np.ones(4), False, 0.0), np.ones((1, 4, 2)))
