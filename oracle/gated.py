"""Float64 oracle for the gated linear recurrence and the 8-bit checkpoints.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.

The map, for every (b, h), with q = sigmoid(r), s = sigmoid(i):
  a_t = exp(-log_re^2 q_t),  x_t = a_t x_{t-1} + sqrt(1 - a_t^2) s_t u_t,  y_t = x_t,
stepped one after another; steps at or past lens[b] are skipped (y is 0 there).
Gradients of f = sum(dy y) + sum(dx x_end) by the chain rule, stepping back:
  G_t = dy_t + a_{t+1} G_{t+1};  d/da = G_t x_{t-1},  d/db = G_t.

Every function also returns (magnitude=True) the same sums with every term's
absolute value: what a rounding of relative size e anywhere in the computation
can move the result by, per e.
"""

import numpy as np

CHUNK = 512
GROUP = 64


def _sig(x):
    out = np.empty_like(x)
    pos = x >= 0
    out[pos] = 1.0 / (1.0 + np.exp(-x[pos]))
    e = np.exp(x[~pos])
    out[~pos] = e / (1.0 + e)
    return out


def _live(lens, B, L):
    if lens is None:
        return np.ones((B, 1, L), dtype=bool)
    return np.arange(L)[None, None, :] < np.clip(np.asarray(lens), 0, L)[:, None, None]


def _parts(u, r, i, log_re, live):
    u, r, i = (np.where(live, np.asarray(t, dtype=np.float64), 0.0) for t in (u, r, i))
    lr = np.asarray(log_re, dtype=np.float64)[None, :, None]
    q, s = _sig(r), _sig(i)
    z = lr * lr * q
    a = np.where(live, np.exp(-z), 1.0)
    w = np.where(live, -np.expm1(-2.0 * z), 0.0)
    return u, q, s, _sig(-r), _sig(-i), a, np.sqrt(w), lr


def gated_recurrence(u, r, i, log_re, x0=None, lens=None, magnitude=False):
    """y [B,H,L] and the state after the last live step [B,H]."""
    u = np.asarray(u)
    B, H, L = u.shape
    live = _live(lens, B, L)
    u, q, s, _, _, a, beta, _ = _parts(u, r, i, log_re, live)
    b = beta * s * u
    x = np.zeros((B, H)) if x0 is None else np.asarray(x0, dtype=np.float64).copy()
    if magnitude:
        b, x = np.abs(b), np.abs(x)
    y = np.zeros((B, H, L))
    for t in range(L):
        x = a[..., t] * x + b[..., t]
        y[..., t] = np.where(live[..., t], x, 0.0)
    return y, x


def gated_backward(u, r, i, log_re, dy, dx=None, x0=None, lens=None, starts=None,
                   magnitude=False):
    """du, dr, di [B,H,L], dlog_re [H], dx0 [B,H].  starts [B,H,ceil(L/512)]:
    states taken up again at every chunk (an 8-bit checkpoint's backward pass);
    None: the recurrence's own."""
    u = np.asarray(u)
    B, H, L = u.shape
    live = _live(lens, B, L)
    u, q, s, nq, ns, a, beta, lr = _parts(u, r, i, log_re, live)
    b = beta * s * u
    dy = np.where(live, np.asarray(dy, dtype=np.float64), 0.0)
    x = np.zeros((B, H)) if x0 is None else np.asarray(x0, dtype=np.float64).copy()
    c = np.zeros((B, H)) if dx is None else np.asarray(dx, dtype=np.float64).copy()
    if magnitude:
        u, b, dy, x, c = (np.abs(t) for t in (u, b, dy, x, c))
        starts = None if starts is None else np.abs(starts)
    prev = np.zeros((B, H, L))
    for t in range(L):
        if starts is not None and t % CHUNK == 0:
            x = np.asarray(starts, dtype=np.float64)[..., t // CHUNK]
        prev[..., t] = x
        x = a[..., t] * x + b[..., t]
    G = np.zeros((B, H, L))
    for t in range(L - 1, -1, -1):
        G[..., t] = dy[..., t] + c
        c = a[..., t] * G[..., t]
    sign = 1.0 if magnitude else -1.0
    ratio = np.divide(a * a, beta, out=np.zeros_like(a), where=beta > 0)
    G = np.where(live, G, 0.0)
    dz = G * s * u * ratio + sign * a * G * prev
    dlog = 2.0 * np.asarray(log_re, dtype=np.float64) * (dz * q).sum(axis=(0, 2))
    if magnitude:
        dlog = np.abs(dlog)
    return G * beta * s, dz * lr * lr * q * nq, G * beta * u * s * ns, dlog, c


def ckpt8(x, largest=float(np.finfo(np.float32).max)):
    """The values the 8-bit form of x [..., L] stands for: per group of 64 steps
    whole multiples, at most 127 in size, of the smallest power of two (not
    below 2^-126) that reaches the largest; NaN where a group holds Inf or NaN.
    largest: the largest value of x's type; a multiple past it is one lower."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros_like(x)
    L = x.shape[-1]
    for lo in range(0, L, GROUP):
        v = x[..., lo:lo + GROUP]
        top = np.max(np.abs(v), axis=-1, keepdims=True)
        e = np.full(top.shape, -126)
        fin = np.isfinite(top)
        while True:  # one power at a time: no logarithm to round
            low = fin & (top > 127.0 * np.exp2(e.astype(np.float64)))
            if not low.any():
                break
            e = e + low
        scale = np.exp2(e.astype(np.float64))
        with np.errstate(invalid="ignore"):
            q = np.rint(v / scale)
            q = np.where(np.abs(q) * scale > largest, q - np.sign(q), q)
            out[..., lo:lo + GROUP] = np.where(fin, q * scale, np.nan)
    return out
