"""Inputs and tolerances shared by the GPU tests of the selective scan and the
short convolution.

Tolerance of a float32 computation: as in seq_cases.py, c 2^-23 times the same
sums with every term's absolute value, plus half a step of the output's type.
c counts roundings (each 2^-24):
* selective forward: a step size 16 (exponential, reciprocal, series), a drive
  3, the exponent of a decay carries the step size's 16 and two more (times the
  exponent, which costs more than it weighs past 2: 36), the lane's steps in
  two passes 32, the lanes' joins 10, the gate 30, the skip 2, the read-out's N
  modes N + 4: below 134 + N; 6 for every tile of 128 steps the state is
  carried over (its entry, four joins, the decay's product);
* selective backward: its products take two such sums, and the sums over a
  group's rows and a lane's steps 32 + H / 32 more;
* short convolution: K products, the gate 20: 2 (K + 20) covers both passes;
  its weights' gradients add up at most 8 + L / 8 terms in a lane and 6 joins.
"""
import numpy as np

from seq_cases import dtype_of, lens_of, spoil_padding, torch_


def c_selective(N, L):
    return 67 + N / 2 + 6 * (-(-L // 256))


def c_selective_back(H, N, L):
    return 2 * c_selective(N, L) + 16 + H / 64


def c_conv(K):
    return K + 20


def c_conv_sums(K, L):
    return K + 28 + L / 16


def selective_inputs(B, H, N, G, L, dtype, seed, gate=True, skip=True, bias=True, joint=False,
                     ragged=False):
    """A dict of GPU tensors: u, delta, z, dy [B,H,L], Bm, Cm [B,G,N,L] in dtype, log_re [H,N], D,
    dt_bias [H], x0, dx [B,H,N], lens."""
    torch = torch_()
    g = np.random.default_rng(seed)
    dt = dtype_of(dtype)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda()

    def part(rows, first, *shape):
        v = g.normal(size=(B,) + shape + (L,))
        if not joint:
            return up(v).to(dt)
        p = torch.full((B, rows, L), float("nan"), dtype=dt, device="cuda")
        n = int(np.prod(shape))
        p[:, first:first + n] = up(v).to(dt).reshape(B, n, L)
        return p[:, first:first + n].unflatten(1, shape)

    s = dict(u=part(2 * H, 0, H), delta=part(H + 3, 2, H), Bm=part(2 * G * N + 5, 5, G, N),
             Cm=part(2 * G * N + 5, 5 + G * N, G, N), z=part(2 * H, H, H) if gate else None,
             log_re=up(g.uniform(0.05, 1.5, (H, N)) * g.choice([-1, 1], (H, N))),
             D=up(g.normal(size=H)) if skip else None,
             dt_bias=up(g.uniform(-4.0, 0.5, H)) if bias else None,
             x0=up(g.normal(size=(B, H, N))), dx=up(g.normal(size=(B, H, N))),
             dy=up(g.normal(size=(B, H, L))).to(dt), lens=lens_of(B, L, seed) if ragged else None)
    if ragged:
        for k in ("u", "delta", "z", "dy"):
            if s[k] is not None:
                spoil_padding(s[k], s["lens"])
        for k in ("Bm", "Cm"):
            for b, n in enumerate(s["lens"].tolist()):
                s[k][b, :, :, n:] = float("inf")
    return s


def conv_inputs(B, H, K, L, dtype, seed, bias=True, joint=False, ragged=False):
    """u, dy [B,H,L] in dtype, w [H,K], bias [H], x0, dx [B,H,K-1] and lens on the GPU."""
    torch = torch_()
    g = np.random.default_rng(seed)
    dt = dtype_of(dtype)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda()
    u = up(g.normal(size=(B, (2 if joint else 1) * H, L))).to(dt)
    s = dict(u=u[:, H:] if joint else u, w=up(g.normal(size=(H, K))),
             bias=up(g.normal(size=H)) if bias else None, x0=up(g.normal(size=(B, H, K - 1))),
             dx=up(g.normal(size=(B, H, K - 1))), dy=up(g.normal(size=(B, H, L))).to(dt),
             lens=lens_of(B, L, seed) if ragged else None)
    if ragged:
        spoil_padding(s["u"], s["lens"])
        spoil_padding(s["dy"], s["lens"])
    return s
