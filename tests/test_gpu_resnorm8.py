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
    (2, 63, 34, "bf16", "int8", "pgl"), (3, 64, 21, "f32", "e4m3", "pgr"), (2, 65, 48, "f16", "int8", "al"),
    (2, 127, 33, "bf16", "e4m3", "nl"), (3, 128, 31, "f16", "int8", "pgj"), (2, 129, 64, "f32", "int8", "ar"),
    (2, 1023, 20, "f32", "int8", "pgl"), (2, 1025, 37, "f32", "e4m3", "al"), (1, 2047, 50, "bf16", "int8", "pgl"),
    (2, 2048, 17, "f32", "int8", "pgr"),
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


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("H,L", [(40, 9), (600, 3), (2500, 1), (100, 1)])
def test_steps_without_numbers(H, L, form):
    """A step that holds Inf or NaN stands for NaN, one of zeros for 0, its neighbours for what
    they were."""
    torch = torch_()
    s = prepared(6, H, L, "bf16", form, "a", seed=H)
    _, q0, s0 = run(s)
    s["x"][1, H // 2, L // 2] = float("inf")
    s["x"][2, 0, 0] = float("nan")
    s["x"][3, :, L - 1] = s["y"][3, :, L - 1] = 0.0
    s["x"][4, :, 0] *= 1e-38
    s["y"][4, :, 0] = 0.0
    _, q, qs = run(s)
    touched = torch.zeros(6, L, dtype=torch.bool, device="cuda")
    touched[1, L // 2] = touched[2, 0] = touched[3, L - 1] = touched[4, 0] = True
    assert torch.isnan(qs[1, L // 2]) and torch.isnan(qs[2, 0])
    assert qs[3, L - 1] == 0.0 and qs[4, 0] == 0.0
    assert not q.float()[touched].any()
    assert torch.equal(q.view(torch.int8)[~touched], q0.view(torch.int8)[~touched])
    assert torch.equal(qs[~touched], s0[~touched])


@pytest.mark.parametrize("H,L", [(40, 33), (700, 9), (700, 1)])
def test_rows_of_no_steps_with_any_parameters(H, L):
    torch = torch_()
    s = prepared(3, H, L, "f32", "int8", "pgr", seed=5)
    s["lens"][:] = torch.tensor([0, 0, 0], dtype=torch.int32)
    for k in ("w_post", "scale", "w_pre"):
        s[k].fill_(float("nan"))
    o, q, qs = run(s)
    assert not o.any() and not q.any() and not qs.any()


@pytest.mark.parametrize("L", [33, 1])
def test_captured_and_replayed_on_streams(L):
    torch = torch_()
    s = prepared(3, 300, L, "bf16", "e4m3", "pg", seed=7)
    run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(s)
    other = torch.cuda.Stream()
    for rep in range(4):
        new = prepared(3, 300, L, "bf16", "e4m3", "pg", seed=40 + rep)
        for k in ("x", "y", "g", "w_post", "scale", "w_pre"):
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        torch.cuda.synchronize()
        eager = run(s, stream=other)
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("L", [40, 1])
def test_gradients_of_the_sum_through_the_norms_backward_pass(L, layer):
    """o = x + y, n = norm(o) w: the statistics with the residual norm's backward pass, called
    without y, give the gradient of both."""
    torch = torch_()
    B, H = 3, 70
    s = prepared(B, H, L, "f32", "int8", "al" if layer else "a", seed=9)
    o, _, _, stats = run(s, stats=True)
    g = bd.resnorm_backward(o, None, None, stats, None, None, s["w_pre"], s["do"], s["dn"],
                            norm=s["norm"])
    one = np.zeros((B, H, L))
    args = (np64(o), one + 1.0, None, np.ones(H), np.zeros(H), np64(s["w_pre"]), np64(s["do"]),
            np64(s["dn"]), layer, EPS)
    ref = oracle.resnorm_backward(*args)
    mag = oracle.resnorm_backward(*args, magnitude=True)
    close(g["dx"], ref[0], mag[0], 2 * c_norm(H), "f32", "dx")
    close(g["dw_pre"], ref[-1], mag[-1], 2 * c_norm(H) + B * L, "f32", "dw_pre")


def test_binding_refuses():
    torch = torch_()
    s = prepared(2, 8, 20, "bf16", "int8", "pg", seed=1)
    x, y, g, wp, sc, wr = (s[k] for k in ("x", "y", "g", "w_post", "scale", "w_pre"))
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, None, None, wr)  # a gate without the norm it follows
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, None, None, sc, wr)
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, None, g, None, None, wr)
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, wp, sc, None)
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, wp, sc, wr, form=2)
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, wp, sc, wr, q=torch.empty(2, 8, 20, dtype=torch.int8,
                                                              device="cuda"))
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, wp, sc, wr, form=bd.Q8_E4M3,
                            q=torch.empty(2, 20, 8, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x, y, g, wp, sc, wr, qs=torch.empty(2, 8, device="cuda"))
    with pytest.raises(TypeError):
        bd.resnorm8_forward(x, y.float(), g, wp, sc, wr)
    with pytest.raises(ValueError):
        bd.resnorm8_forward(x[..., ::2], y[..., ::2], None, wp, sc, wr)
    with pytest.raises(bd.DSSMError):
        bd.resnorm8_forward(x, y, g, wp, sc, wr, o=x)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last steps of the last row against the same steps alone."""
    torch = torch_()
    B, H, L = 2, 1100, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, H, L, device="cuda", generator=gen, dtype=torch.bfloat16)
    w = torch.randn(H, device="cuda", generator=gen)
    _, q, qs = bd.resnorm8_forward(x, None, None, None, None, w)
    tail = x[1:, :, L - 64:].contiguous()
    _, q2, s2 = bd.resnorm8_forward(tail, None, None, None, None, w)
    assert torch.equal(q[1:, L - 64:], q2) and torch.equal(qs[1:, L - 64:], s2)
