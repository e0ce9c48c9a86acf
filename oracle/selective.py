"""Float64 oracle for the selective scan and the short causal convolution.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.

The scan, for every (b, h) and its N modes, g the channel's group:
  dt_t = softplus(delta_t + dt_bias),  x_t = exp(-log_re^2 dt_t) x_{t-1} + dt_t B_t[g] u_t,
  y_t = (sum_n C_t[g] x_t + D u_t) silu(z_t),
stepped one after another; steps at or past lens[b] are skipped (y is 0 there).
Gradients of f = sum(dy y) + sum(dx x_end) by the chain rule, stepping back.

Every function also returns (magnitude=True) the same sums with every term's
absolute value: what a rounding of relative size e anywhere in the computation
can move the result by, per e.
"""

import numpy as np


def _sig(x):
    return np.exp(-np.logaddexp(0.0, -x))


def _live(lens, B, L):
    if lens is None:
        return np.ones((B, 1, L), dtype=bool)
    return np.arange(L)[None, None, :] < np.clip(np.asarray(lens), 0, L)[:, None, None]


def _f64(t, live=None):
    t = np.asarray(t, dtype=np.float64)
    return t if live is None else np.where(live, t, 0.0)


def _parts(u, delta, Bm, Cm, log_re, dt_bias, lens):
    B, H, L = np.shape(u)
    G, N = np.shape(Bm)[1:3]
    live = _live(lens, B, L)
    u, delta = _f64(u, live), _f64(delta, live)
    if dt_bias is not None:
        delta = delta + _f64(dt_bias)[None, :, None]
    dt = np.where(live, np.logaddexp(0.0, delta), 0.0)
    rep = lambda t: np.repeat(_f64(t, live[:, :, None]), H // G, axis=1)  # [B,H,N,L]
    re2 = _f64(log_re) ** 2
    return live, u, delta, dt, rep(Bm), rep(Cm), re2


def selective_scan(u, delta, Bm, Cm, log_re, D=None, dt_bias=None, z=None, x0=None, lens=None,
                   magnitude=False):
    """y [B,H,L] and the state after the last live step [B,H,N]."""
    B, H, L = np.shape(u)
    N = np.shape(Bm)[2]
    live, u, delta, dt, Bh, Ch, re2 = _parts(u, delta, Bm, Cm, log_re, dt_bias, lens)
    x = np.zeros((B, H, N)) if x0 is None else _f64(x0).copy()
    d = np.zeros(H) if D is None else _f64(D)
    if magnitude:
        u, Bh, Ch, x, d = np.abs(u), np.abs(Bh), np.abs(Ch), np.abs(x), np.abs(d)
    y = np.zeros((B, H, L))
    for t in range(L):
        x = np.exp(-re2[None] * dt[..., t, None]) * x + (dt * u)[..., t, None] * Bh[..., t]
        y[..., t] = (Ch[..., t] * x).sum(-1) + d[None] * u[..., t]
    if z is not None:
        z = _f64(z, live)
        s = z * _sig(z)
        y = y * (np.abs(s) if magnitude else s)
    return np.where(live, y, 0.0), x


def selective_backward(u, delta, Bm, Cm, log_re, dy, D=None, dt_bias=None, z=None, dx=None, x0=None,
                       lens=None, magnitude=False):
    """A dict du, ddelta, dz [B,H,L], dB, dC [B,G,N,L], dlog_re [H,N], dD, ddt_bias [H], dx0
    [B,H,N] (None where there is no such input)."""
    B, H, L = np.shape(u)
    G, N = np.shape(Bm)[1:3]
    live, u, delta, dt, Bh, Ch, re2 = _parts(u, delta, Bm, Cm, log_re, dt_bias, lens)
    m = np.abs if magnitude else (lambda t: t)
    x = np.zeros((B, H, N)) if x0 is None else m(_f64(x0)).copy()
    d = np.zeros(H) if D is None else m(_f64(D))
    u, Bh, Ch = m(u), m(Bh), m(Ch)
    dy = m(_f64(dy, live))
    states, decayed = np.zeros((B, H, N, L)), np.zeros((B, H, N, L))
    a = np.exp(-re2[None, :, :, None] * dt[:, :, None])
    for t in range(L):
        decayed[..., t] = a[..., t] * x
        x = decayed[..., t] + (dt * u)[..., t, None] * Bh[..., t]
        states[..., t] = x
    out = dict(dz=None)
    p = dy
    if z is not None:
        zz = _f64(z, live)
        s = _sig(zz)
        slope = m(s) + m(zz * s * _sig(-zz)) if magnitude else s + zz * s * _sig(-zz)
        total = (Ch * states).sum(2) + d[None, :, None] * u
        out["dz"] = np.where(live, dy * total * slope, 0.0)
        p = np.where(live, dy * m(zz * s), 0.0)
    G_ = np.zeros((B, H, N)) if dx is None else m(_f64(dx)).copy()
    q, w = np.zeros((B, H, L)), np.zeros((B, H, L))
    dB, dC = np.zeros((B, H, N, L)), np.zeros((B, H, N, L))
    dlog = np.zeros((B, H, N))
    for t in range(L - 1, -1, -1):
        G_ = G_ + Ch[..., t] * p[..., t, None]
        wt = G_ * decayed[..., t]
        q[..., t] = (G_ * Bh[..., t]).sum(-1)
        w[..., t] = (re2[None] * wt).sum(-1)
        dB[..., t] = G_ * (dt * u)[..., t, None]
        dC[..., t] = p[..., t, None] * states[..., t]
        dlog += wt * dt[..., t, None]
        G_ = a[..., t] * G_
    step = (u * q + w if magnitude else u * q - w) * _sig(delta)
    group = lambda t: t.reshape(B, G, H // G, N, L).sum(2)
    out["du"] = np.where(live, dt * q + d[None, :, None] * p, 0.0)
    out["ddelta"] = np.where(live, step, 0.0)
    out["dB"], out["dC"] = group(dB), group(dC)
    lr = _f64(log_re)
    out["dlog_re"] = (2.0 * np.abs(lr) if magnitude else -2.0 * lr) * dlog.sum(0)
    out["dD"] = None if D is None else (p * u).sum((0, 2))
    out["ddt_bias"] = None if dt_bias is None else out["ddelta"].sum((0, 2))
    out["dx0"] = G_
    return out


def _extended(u, x0, K, live):
    B, H, L = np.shape(u)
    past = np.zeros((B, H, K - 1)) if x0 is None else _f64(x0)
    return np.concatenate([past, _f64(u, live)], axis=2)


def short_conv(u, w, bias=None, silu=True, x0=None, lens=None, magnitude=False):
    """y_t = act(bias + sum_k w_k e_{t+k}), e the K - 1 inputs x0 followed by u: y [B,H,L] and the
    last K - 1 of e up to the last live step."""
    B, H, L = np.shape(u)
    K = np.shape(w)[1]
    live = _live(lens, B, L)
    e, w = _extended(u, x0, K, live), _f64(w)
    b = np.zeros(H) if bias is None else _f64(bias)
    pre, mag = np.zeros((B, H, L)), np.zeros((B, H, L))
    for t in range(L):
        pre[..., t] = b + (w[None] * e[..., t:t + K]).sum(-1)
        mag[..., t] = np.abs(b) + np.abs(w[None] * e[..., t:t + K]).sum(-1)
    # silu' is at most 1.1 in absolute value, silu at most its argument
    y = mag * 1.1 if magnitude else (pre * _sig(pre) if silu else pre)
    n = np.full(B, L) if lens is None else np.clip(np.asarray(lens), 0, L)
    end = np.stack([e[b_, :, n[b_]:n[b_] + K - 1] for b_ in range(B)]) if B else e[:, :, :K - 1]
    return np.where(live, y, 0.0), np.abs(end) if magnitude else end


def short_conv_backward(u, w, dy, bias=None, silu=True, x0=None, dx=None, lens=None,
                        magnitude=False):
    """A dict du [B,H,L], dw [H,K], dbias [H], dx0 [B,H,K-1]."""
    B, H, L = np.shape(u)
    K = np.shape(w)[1]
    live = _live(lens, B, L)
    e, w = _extended(u, x0, K, live), _f64(w)
    b = np.zeros(H) if bias is None else _f64(bias)
    p = _f64(dy, live).copy()
    if silu:
        for t in range(L):
            pre = b + (w[None] * e[..., t:t + K]).sum(-1)
            if magnitude:
                mag = np.abs(b) + np.abs(w[None] * e[..., t:t + K]).sum(-1)
                # silu'' is at most 1/2 in absolute value
                p[..., t] = np.abs(p[..., t]) * (_sig(pre) + np.abs(pre * _sig(pre) * _sig(-pre))
                                                 + 0.5 * mag)
            else:
                p[..., t] *= _sig(pre) + pre * _sig(pre) * _sig(-pre)
    if magnitude:
        p, e, w = np.abs(p), np.abs(e), np.abs(w)
    de, dw = np.zeros_like(e), np.zeros((H, K))
    for t in range(L):
        de[..., t:t + K] += w[None] * p[..., t, None]
        dw += (p[..., t, None] * e[..., t:t + K]).sum(0)
    if dx is not None and K > 1:
        for b_ in range(B):
            n = L if lens is None else int(np.clip(lens[b_], 0, L))
            de[b_, :, n:n + K - 1] += np.abs(_f64(dx)[b_]) if magnitude else _f64(dx)[b_]
    return dict(du=np.where(live, de[..., K - 1:], 0.0), dw=dw, dbias=p.sum((0, 2)),
                dx0=de[..., :K - 1])
