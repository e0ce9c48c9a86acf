"""GPU parity of the residual norm with its output in 8 bits against the float64
oracle.

The stream is compared as the residual norm's tests do.  The scale of a step is
its largest |n| over M and the values are off by at most half a step of their 8
bits (1/2 for whole numbers; 2^-4 of the value, or half of 2^-9 below 2^-6, for
e4m3), both on top of a float32 computation's own roundings (seq_cases.c_norm).
"""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from seq_cases import STEP, c_norm, close, dtype_of, lens_of, norm_inputs, np64, say, spoil_padding, torch_

pytestmark = pytest.mark.gpu

EPS = 1e-5
FORMS = {"int8": bd.Q8_INT8, "e4m3": bd.Q8_E4M3}
MOST = {"int8": 127.0, "e4m3": 448.0}

# (B, H, L, type, form, what): channels around a lane's four and every layout's most, lengths
# around a strip; what: p with the norm after the layer, g its gate, a the sum alone, n the norm
# alone, l layer norms, r rows of several lengths, j the gate a slice of a joint projection
SHAPES = [
    (2, 1, 3, "f32", "int8", "n"), (2, 3, 33, "bf16", "e4m3", "pg"), (3, 4, 31, "f16", "int8", "ar"),
    (2, 255, 16, "f32", "e4m3", "pgl"), (3, 256, 17, "bf16", "int8", "pgrj"), (2, 257, 32, "f16", "e4m3", "a"),
    (2, 511, 40, "bf16", "int8", "nlr"), (3, 512, 64, "f32", "int8", "pr"), (2, 515, 63, "bf16", "e4m3", "al"),
    (2, 1024, 65, "bf16", "int8", "pgj"), (1, 1030, 100, "f16", "e4m3", "pglr"), (2, 2048, 33, "bf16", "int8", "a"),
    (2, 2049, 15, "f32", "int8", "pg"), (1, 4096, 70, "bf16", "e4m3", "ar"), (2, 4099, 18, "f16", "int8", "pgr"),
    (1, 8192, 35, "bf16", "int8", "pgl"), (1, 8191, 9, "f32", "e4m3", "n"), (40, 96, 2, "bf16", "int8", "a"),
    (3, 100, 5000, "bf16", "e4m3", "ar"),
    (1, 1, 1, "f32", "int8", "a"), (5, 7, 1, "bf16", "e4m3", "pgr"), (9, 512, 1, "f16", "int8", "pgl"),
    (6, 513, 1, "f32", "e4m3", "ar"), (3, 2048, 1, "bf16", "int8", "n"), (4, 2055, 1, "bf16", "int8", "pgrj"),
    (64, 4096, 1, "bf16", "int8", "a"), (2, 8192, 1, "f32", "e4m3", "pgl"),
]
IDS = ["B%dH%dL%d-%s-%s-%s" % s for s in SHAPES]


def prepared(B, H, L, dtype, form, what, seed):
    say("case: B=%d H=%d L=%d %s %s %s seed=%d" % (B, H, L, dtype, form, what, seed))
    s = norm_inputs(B, H, L, dtype, seed, "j" in what)
    s["lens"] = lens_of(B, L, seed) if "r" in what else None
    if "r" in what:
        for k in ("x", "y", "g"):
            spoil_padding(s[k], s["lens"])
    if "p" not in what:
        s["w_post"] = s["scale"] = None
    if "g" not in what:
        s["g"] = None
    if "n" in what:
        s["y"] = None
    s["norm"] = bd.NORM_LAYER if "l" in what else bd.NORM_RMS
    s["form"] = FORMS[form]
    return s


def run(s, stats=False, **kw):
    fn = bd.resnorm8_forward_stats if stats else bd.resnorm8_forward
    return fn(s["x"], s["y"], s["g"], s["w_post"], s["scale"], s["w_pre"], norm=s["norm"], eps=EPS,
              form=s["form"], lens=s["lens"], **kw)


def check_bits(q, qs, stored, w_pre, layer, form, live, what=""):
    """q, qs against the norm of the stored stream [B,H,L]; live [B,L]."""
    n = oracle.resnorm_out(stored, w_pre, layer, EPS).transpose(0, 2, 1)
    mag = oracle.resnorm_out(stored, w_pre, layer, EPS, magnitude=True).transpose(0, 2, 1)
    c = c_norm(stored.shape[1])
    near = c * STEP * mag
    s = np64(qs)
    top = np.abs(n).max(-1)
    err = np.abs(s - np.where(live, top / MOST[form], 0.0))
    tol = np.where(live, (near.max(-1) + 4 * STEP * top) / MOST[form], 0.0)
    assert (err <= tol).all(), (what, "scale", float(np.max(err - tol)))
    v = np64(q.float())
    assert np.abs(v).max(initial=0.0) <= MOST[form]
    assert not v[~live].any()
    half = 0.5 if form == "int8" else np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10)
    bound = half * s[..., None] * (1 + 8 * STEP) + near + 4 * STEP * np.abs(n)
    off = np.where(live[..., None], np.abs(v * s[..., None] - n), 0.0)
    worst = float(np.max(off / np.maximum(bound, 1e-300), initial=0.0))
    say("  values   worst error / tolerance %.3f" % worst)
    assert worst <= 1.0, (what, worst)
    # the largest value of a live step takes the whole range
    full = np.abs(v).max(-1)
    assert (full[live & (top > 0)] == MOST[form]).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    B, H, L, dtype, form, what = shape
    torch = torch_()
    s = prepared(*shape, seed=H + L)
    o, q, qs, stats = run(s, stats=True)
    layer = s["norm"] == bd.NORM_LAYER
    assert tuple(q.shape) == (B, L, H) and tuple(qs.shape) == (B, L)
    lens = np.full(B, L) if s["lens"] is None else s["lens"].cpu().numpy()
    live = np.arange(L)[None] < lens[:, None]
    zero = lambda t: np.nan_to_num(np64(t)) * live[:, None]
    if s["y"] is None:
        assert o is None
        stored = zero(s["x"])
    else:
        if s["w_post"] is not None:
            g = None if s["g"] is None else zero(s["g"])
            a = [zero(s["x"]), zero(s["y"]), g, np64(s["w_post"]), np64(s["scale"]), layer, EPS]
            ref, mag = (oracle.resnorm_stream(*a, magnitude=m) for m in (False, True))
        else:
            ref = zero(s["x"]) + zero(s["y"])
            mag = np.abs(zero(s["x"])) + np.abs(zero(s["y"]))
        close(o, ref * live[:, None], mag, c_norm(H), dtype, "o")
        stored = np64(o)
    check_bits(q, qs, stored, np64(s["w_pre"]), layer, form, live)
    # the statistics are the backward pass's: as the residual norm's own
    if s["y"] is None or s["w_post"] is not None:
        _, _, theirs = bd.resnorm_forward_stats(s["x"], s["y"], s["g"], s["w_post"], s["scale"],
                                                s["w_pre"], norm=s["norm"], eps=EPS, lens=s["lens"])
        rows = slice(None) if s["y"] is not None else slice(stats.shape[0] // 2, None)
        a, b = np64(stats[rows]), np64(theirs[rows])
        assert (np.abs(a - b) <= 2 * c_norm(H) * STEP * np.maximum(np.abs(b), 1.0)).all()
    again = run(s)
    assert torch.equal(q.view(torch.int8), again[1].view(torch.int8)) and torch.equal(qs, again[2])
