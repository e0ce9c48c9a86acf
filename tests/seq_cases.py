"""Inputs and tolerances shared by the GPU tests of the gated recurrence, the
8-bit checkpoints and the residual norm.

Tolerance of a float32 computation: c 2^-23 times the same sums with every
term's absolute value (the oracle's magnitude=True), plus half a step of the
output's type.  c counts roundings (each 2^-24, the hardware's exp2, reciprocal
and square root 2^-23):
* gated forward: a gate's chain of exp2, reciprocal and products leaves b within
  some 60 roundings of its own (the exponent of exp(-x) carries |x| log2(e) of
  them, |x| <= 10 here), eight steps of decay in a lane 24, six levels of the
  wave's scan 18, the second pass over the lane 16: below 128 = 2 * 64; a
  further 12 for every tile of 512 steps the state is carried over;
* gated backward: its products take two such sums, 2 (128 + 12 tiles);
* residual norm: the sums over H run over at most H / 16 terms in a row, a
  dozen more in the joins (two sums and their mean for the layer norm), the
  factor 4, the gate 30, the products 10: 2 (48 + H / 16).
"""
import numpy as np

from long_convolution_sequence_amd import binding as bd

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SUB = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half a subnormal step
STEP = 2.0 ** -23


def torch_():
    import torch
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def dtype_of(name):
    torch = torch_()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def say(*a):
    print(*a, flush=True)


def np64(t):
    return t.detach().double().cpu().numpy()


def c_gated(L):
    return 64 + 6 * (-(-L // 512))


def c_norm(H):
    return 48 + H / 16


def close(got, ref, mag, c, dtype, what):
    """got (a tensor) against ref, elementwise."""
    g = np64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all(), what + ": not finite"
    near = c * STEP * mag
    # double rounding: half a step of what the computation may have reached
    tol = near + HALF[dtype] * (np.abs(ref) + near) + SUB[dtype]
    err = np.abs(g - ref)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    say("  %-8s worst error / tolerance %.3f" % (what, worst))
    assert worst <= 1.0, (what, worst, np.unravel_index(np.argmax(err / tol), err.shape))


def gated_inputs(B, H, L, dtype, seed, joint=False):
    """u, r, i, dy [B,H,L] in dtype, log_re [H], x0, dx [B,H] on the GPU."""
    torch = torch_()
    g = np.random.default_rng(seed)
    dt = dtype_of(dtype)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda()
    s = dict(log_re=up(np.exp(g.uniform(np.log(0.015), np.log(2.0), H)) * g.choice([-1, 1], H)),
             x0=up(g.normal(size=(B, H))), dx=up(g.normal(size=(B, H))),
             dy=up(g.normal(size=(B, H, L))).to(dt))
    gates = [np.clip(g.normal(size=(B, H, L)) * sd, -10, 10) for sd in (1.0, 2.0, 2.0)]
    if joint:
        p = up(np.concatenate(gates, axis=1)).to(dt)
        s["u"], s["r"], s["i"] = p[:, :H], p[:, H:2 * H], p[:, 2 * H:]
    else:
        s["u"], s["r"], s["i"] = (up(a).to(dt) for a in gates)
    return s


def lens_of(B, L, seed):
    """0, 1, L and odd lengths between, as far as B goes."""
    torch = torch_()
    g = np.random.default_rng(seed)
    lens = [L, 0, 1][:B] + [int(g.integers(0, L + 1)) for _ in range(max(0, B - 3))]
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


def spoil_padding(t, lens):
    """NaN behind every row's end (in place)."""
    for b, n in enumerate(lens.tolist()):
        t[b, :, n:] = float("nan")


def norm_inputs(B, H, L, dtype, seed, joint=False):
    torch = torch_()
    g = np.random.default_rng(seed)
    dt = dtype_of(dtype)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda()
    s = {k: up(g.normal(size=(B, H, L)) * sd + m).to(dt)
         for k, sd, m in (("x", 2.0, 0.5), ("y", 0.7, 0.3), ("do", 1.0, 0.0), ("dn", 1.0, 0.0))}
    gate = np.clip(g.normal(size=(B, H, L)) * 2.0, -10, 10)
    if joint:
        p = up(np.concatenate([np.zeros_like(gate), gate], axis=1)).to(dt)
        s["g"] = p[:, H:]
    else:
        s["g"] = up(gate).to(dt)
    s["w_post"], s["scale"], s["w_pre"] = (up(g.normal(size=H) + m) for m in (1.0, 0.3, 1.0))
    return s


KINDS = {"state": bd.CKPT_STATE, "int8": bd.CKPT_INT8}
