"""Float64 oracle for the residual norm.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.

Over the H channels (axis 1) of x, y, g [B,H,L]:
  norm(a) = (a - m) / sqrt(mean((a - m)^2) + eps),  m = mean(a) or (rms) 0,
  o = x + scale norm(y) w_post silu(g),  n = norm(o) w_pre,
and the gradients of f = sum(do o) + sum(dn n), the norm's as the product with
its Jacobian.  stored: the stream as rounded to the activations' type, which
the second norm and the gradients are taken at.

magnitude=True: every term's absolute value instead (see oracle.gated).
"""

import numpy as np


def _norm(a, layer, eps):
    m = a.mean(axis=1, keepdims=True) if layer else np.zeros_like(a[:, :1])
    f = 1.0 / np.sqrt(((a - m) ** 2).mean(axis=1, keepdims=True) + eps)
    return a - m, f


def _wide(a, layer):
    """|a| plus, where the mean is taken off, the mean of |a|: the terms of
    a - mean(a) by their absolute values."""
    return np.abs(a) + (np.abs(a).mean(axis=1, keepdims=True) if layer else 0.0)


def _vec(w):
    return np.asarray(w, dtype=np.float64)[None, :, None]


def _silu(g):
    s = 1.0 / (1.0 + np.exp(-g))
    return g * s, s * (1.0 + g * (1.0 - s))


def resnorm_stream(x, y, g, w_post, scale, layer, eps, magnitude=False):
    """o [B,H,L] (float64, not rounded)."""
    x, y = np.asarray(x, dtype=np.float64), np.asarray(y, dtype=np.float64)
    c, f = _norm(y, layer, eps)
    silu = np.ones_like(x) if g is None else _silu(np.asarray(g, dtype=np.float64))[0]
    if magnitude:
        return np.abs(x) + np.abs(_vec(scale) * _vec(w_post) * silu) * _wide(y, layer) * f
    return x + _vec(scale) * (c * f * _vec(w_post)) * silu


def resnorm_out(stored, w_pre, layer, eps, magnitude=False):
    """n [B,H,L] from the stored stream."""
    o = np.asarray(stored, dtype=np.float64)
    c, f = _norm(o, layer, eps)
    if magnitude:
        return _wide(o, layer) * f * np.abs(_vec(w_pre))
    return c * f * _vec(w_pre)


def _through(grad, c, f, layer, magnitude, wide):
    """The norm's transposed Jacobian times grad; wide: _wide(a) for magnitudes."""
    if magnitude:
        grad = np.abs(grad)
        out = f * (grad + wide * f * (grad * wide * f).mean(axis=1, keepdims=True))
        return out + (f * grad.mean(axis=1, keepdims=True) if layer else 0.0)
    out = f * (grad - c * f * (grad * c * f).mean(axis=1, keepdims=True))
    return out - (f * grad.mean(axis=1, keepdims=True) if layer else 0.0)


def resnorm_backward(stored, y, g, w_post, scale, w_pre, do, dn, layer, eps, magnitude=False):
    """dx, dy, dg [B,H,L], dw_post, dscale, dw_pre [H] (None where there is no
    such input)."""
    ab = np.abs if magnitude else (lambda t: t)
    o = np.asarray(stored, dtype=np.float64)
    t = np.zeros_like(o) if do is None else ab(np.asarray(do, dtype=np.float64))
    dw_pre = np.zeros(o.shape[1])
    if dn is not None:
        c, f = _norm(o, layer, eps)
        wide = _wide(o, layer)
        dn = np.asarray(dn, dtype=np.float64)
        t = t + _through(dn * _vec(w_pre), c, f, layer, magnitude, wide)
        dw_pre = (ab(dn) * (wide if magnitude else c) * f).sum(axis=(0, 2))
    if y is None:
        return t, None, None, None, None, dw_pre
    y = np.asarray(y, dtype=np.float64)
    c, f = _norm(y, layer, eps)
    wide = _wide(y, layer)
    yh = (wide if magnitude else c) * f
    if g is None:
        silu, dsilu = np.ones_like(o), np.zeros_like(o)
    else:
        g = np.asarray(g, dtype=np.float64)
        silu, dsilu = _silu(g)
        if magnitude:
            s = 1.0 / (1.0 + np.exp(-g))
            silu, dsilu = np.abs(silu), s * (1.0 + np.abs(g) * (1.0 - s))
    wp, sc = ab(_vec(w_post)), ab(_vec(scale))
    dy = _through(t * sc * wp * silu, c, f, layer, magnitude, wide)
    dg = None if g is None else t * sc * wp * yh * dsilu
    return (t, dy, dg, (t * sc * silu * yh).sum(axis=(0, 2)), (t * wp * silu * yh).sum(axis=(0, 2)),
            dw_pre)
