"""GPU parity of the selective scan (a sequence, streaming, one token, backward)
against the float64 oracle."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from selective_cases import c_selective, c_selective_back, selective_inputs
from seq_cases import close, np64, say, torch_

pytestmark = pytest.mark.gpu

# (B, H, N, G, L, type, what): lengths around the borders of a lane, a short tile and a tile;
# modes around a stage's eight; channels around a wave's four and a workgroup's rows; few rows,
# whose modes are shared by four waves and whose steps are cut into segments; many rows
SHAPES = [
    (2, 3, 1, 1, 1, "f32", "gsb"), (3, 4, 4, 2, 2, "bf16", "gsbr"), (2, 5, 3, 1, 3, "f16", "sb"),
    (3, 6, 16, 3, 4, "f32", "gr"), (2, 33, 8, 1, 5, "bf16", "gsbj"), (4, 7, 9, 1, 15, "f32", "sbr"),
    (2, 32, 17, 2, 16, "f16", "gsb"), (3, 31, 7, 1, 17, "f32", "br"), (2, 4, 16, 1, 63, "bf16", "gsb"),
    (4, 8, 5, 4, 64, "f32", "gsbr"), (3, 34, 3, 2, 65, "f32", "gsbj"), (4, 12, 16, 1, 255, "bf16", "gbr"),
    (2, 9, 8, 1, 256, "f32", "gsb"), (3, 10, 4, 2, 257, "f32", "sbr"), (2, 3, 2, 1, 300, "f16", "gsb"),
    (3, 5, 64, 1, 513, "f32", "gsbr"), (1, 2, 128, 1, 700, "bf16", "gsb"), (2, 130, 13, 2, 1001, "f16", "r"),
    (3, 66, 16, 1, 2049, "f32", "gsbrj"), (1, 4, 16, 1, 9000, "f32", "gsb"), (1, 3, 2, 1, 5000, "f32", "sb"),
    (2, 2, 33, 2, 6000, "bf16", "gsbr"), (2, 2048, 5, 1, 300, "f32", "gsb"), (3, 1400, 3, 2, 270, "bf16", "gsbr"),
    (600, 9, 4, 1, 20, "f32", "gsbr"), (4, 1030, 11, 1, 258, "f16", "gsb"),
]
IDS = ["B%dH%dN%dG%dL%d-%s-%s" % s for s in SHAPES]
GRADS = ("du", "ddelta", "dz", "dB", "dC", "dlog_re", "dD", "ddt_bias", "dx0")


def prepared(B, H, N, G, L, dtype, what, seed):
    say("case: B=%d H=%d N=%d G=%d L=%d %s %s seed=%d" % (B, H, N, G, L, dtype, what, seed))
    return selective_inputs(B, H, N, G, L, dtype, seed, gate="g" in what, skip="s" in what,
                            bias="b" in what, joint="j" in what, ragged="r" in what)


def args_of(s):
    return [s[k] for k in ("u", "delta", "Bm", "Cm", "log_re")]


def options_of(s):
    return {k: s[k] for k in ("D", "dt_bias", "z", "lens")}


def reference(s, back=False, **kw):
    a = [np.nan_to_num(np64(t), posinf=0.0) for t in args_of(s)]
    o = {k: None if s[k] is None else np.nan_to_num(np64(s[k])) for k in ("D", "dt_bias", "z", "x0")}
    o["lens"] = None if s["lens"] is None else s["lens"].cpu().numpy()
    if back:
        return oracle.selective_backward(*a, np.nan_to_num(np64(s["dy"])), dx=np64(s["dx"]), **o, **kw)
    return oracle.selective_scan(*a, **o, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_state(shape):
    B, H, N, G, L, dtype, what = shape
    torch = torch_()
    s = prepared(*shape, seed=L + H)
    xo = torch.full_like(s["x0"], float("nan"))
    y = bd.selective_forward(*args_of(s), x=s["x0"], x_out=xo, **options_of(s))
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(y, ref, mag, c_selective(N, L), dtype, "y")
    close(xo, end, mend, c_selective(N, L), "f32", "state")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    B, H, N, G, L, dtype, what = shape
    torch = torch_()
    s = prepared(*shape, seed=2 * L + H)
    y, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=torch.empty_like(s["x0"]),
                                        **options_of(s))
    plain = bd.selective_forward(*args_of(s), x=s["x0"], x_out=torch.empty_like(s["x0"]),
                                 **options_of(s))
    assert torch.equal(y, plain)
    got = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], **options_of(s))
    ref, mag = reference(s, True), reference(s, True, magnitude=True)
    for n in GRADS:
        if ref[n] is None:
            assert got[n] is None
            continue
        t = "f32" if n in ("dlog_re", "dD", "ddt_bias", "dx0") else dtype
        close(got[n], ref[n], mag[n], c_selective_back(H, N, L), t, n)
    again = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], **options_of(s))
    for n in GRADS:
        assert got[n] is None or torch.equal(got[n], again[n]), n + " differs between two calls"


@pytest.mark.parametrize("B,H,N,G,dtype,what", [
    (1, 1, 1, 1, "f32", "gsb"), (5, 6, 3, 2, "bf16", "gsbr"), (8, 64, 16, 1, "bf16", "gsb"),
    (3, 10, 17, 5, "f16", "sr"), (2, 33, 64, 1, "f32", "gbr"), (4, 7, 128, 1, "bf16", "b"),
    (300, 130, 16, 1, "f32", "gsbr"), (2, 5, 5, 1, "f16", "gsb")])
def test_step(B, H, N, G, dtype, what):
    torch = torch_()
    s = prepared(B, H, N, G, 1, dtype, what, seed=B + H + N)
    flat = {k: None if s[k] is None else s[k][..., 0].contiguous()
            for k in ("u", "delta", "Bm", "Cm", "z")}
    x = s["x0"].clone()
    y = bd.selective_step(flat["u"], flat["delta"], flat["Bm"], flat["Cm"], s["log_re"], x,
                          D=s["D"], dt_bias=s["dt_bias"], z=flat["z"], lens=s["lens"])
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(y, ref[..., 0], mag[..., 0], c_selective(N, 1), dtype, "y")
    close(x, end, mend, c_selective(N, 1), "f32", "state")
    if s["lens"] is not None:
        idle = (s["lens"] <= 0).cpu().numpy()
        assert np.array_equal(np64(x)[idle], np64(s["x0"])[idle]) and not np64(y)[idle].any()
