"""GPU parity of the short causal convolution (a sequence, streaming, one token,
backward) against the float64 oracle."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from selective_cases import c_conv, c_conv_sums, conv_inputs
from seq_cases import close, np64, say, torch_

pytestmark = pytest.mark.gpu

# (B, H, K, L, type, what): lengths around a lane's steps, a wave's tile with its helping lane
# and a workgroup's; more taps than steps; few rows, cut into segments
SHAPES = [
    (2, 3, 4, 1, "f32", "ab"), (3, 5, 8, 2, "bf16", "abr"), (4, 3, 3, 7, "f16", "br"),
    (2, 3, 4, 8, "f32", "ab"), (3, 7, 2, 9, "bf16", "ar"), (3, 2, 1, 64, "f32", "abr"),
    (4, 3, 5, 65, "f16", "abj"), (5, 3, 4, 300, "f32", "abr"), (2, 3, 6, 504, "bf16", "ab"),
    (2, 3, 7, 505, "f32", "b"), (3, 3, 8, 511, "f32", "abr"), (3, 3, 4, 512, "f16", "abrj"),
    (3, 3, 4, 513, "f32", "abr"), (2, 3, 8, 1008, "f32", "ab"), (4, 5, 4, 1009, "bf16", "abr"),
    (2, 3, 3, 2048, "f32", "a"), (3, 2, 4, 2049, "f16", "abr"), (1, 1, 7, 20000, "f32", "ab"),
    (4, 131, 4, 2100, "bf16", "abrj"), (8, 1024, 4, 1030, "f32", "ab"), (3000, 3, 4, 9, "f32", "abr"),
]
IDS = ["B%dH%dK%dL%d-%s-%s" % s for s in SHAPES]


def prepared(B, H, K, L, dtype, what, seed):
    say("case: B=%d H=%d K=%d L=%d %s %s seed=%d" % (B, H, K, L, dtype, what, seed))
    s = conv_inputs(B, H, K, L, dtype, seed, bias="b" in what, joint="j" in what,
                    ragged="r" in what)
    s["act"] = bd.ACT_SILU if "a" in what else bd.ACT_NONE
    return s


def reference(s, back=False, **kw):
    o = dict(bias=None if s["bias"] is None else np64(s["bias"]), silu=s["act"] == bd.ACT_SILU,
             x0=np64(s["x0"]), lens=None if s["lens"] is None else s["lens"].cpu().numpy(), **kw)
    u = np.nan_to_num(np64(s["u"]))
    if back:
        return oracle.short_conv_backward(u, np64(s["w"]), np.nan_to_num(np64(s["dy"])),
                                          dx=np64(s["dx"]), **o)
    return oracle.short_conv(u, np64(s["w"]), **o)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_state(shape):
    B, H, K, L, dtype, what = shape
    torch = torch_()
    s = prepared(*shape, seed=L + H)
    x = s["x0"].clone()
    y = bd.shortconv_forward(s["u"], s["w"], s["bias"], s["act"], x=x, lens=s["lens"])
    ref, end = reference(s)
    mag, _ = reference(s, magnitude=True)
    close(y, ref, mag, c_conv(K), dtype, "y")
    # the state is a copy of the last inputs
    assert np.array_equal(np64(x), end)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    B, H, K, L, dtype, what = shape
    torch = torch_()
    s = prepared(*shape, seed=2 * L + H)
    call = lambda: bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], s["act"], x=s["x0"],
                                         dx=s["dx"], lens=s["lens"])
    got = call()
    ref, mag = reference(s, True), reference(s, True, magnitude=True)
    for n, t, c in (("du", dtype, 2 * c_conv(K)), ("dw", "f32", 2 * c_conv_sums(K, L)),
                    ("dbias", "f32", 2 * c_conv_sums(K, L)), ("dx0", "f32", 2 * c_conv(K))):
        if n == "dbias" and s["bias"] is None:
            assert got[n] is None
        elif got[n].numel():
            close(got[n], ref[n], mag[n], c, t, n)
    again = call()
    for n in got:
        assert got[n] is None or torch.equal(got[n], again[n]), n + " differs between two calls"


@pytest.mark.parametrize("B,H,K,dtype,what", [
    (1, 1, 1, "f32", "ab"), (5, 6, 2, "bf16", "abr"), (64, 300, 4, "bf16", "ab"),
    (3, 10, 8, "f16", "ar"), (2, 33, 5, "f32", "b")])
def test_step(B, H, K, dtype, what):
    torch = torch_()
    s = prepared(B, H, K, 1, dtype, what, seed=B + H + K)
    x = s["x0"].clone()
    y = bd.shortconv_step(s["u"][..., 0].contiguous(), s["w"], s["bias"], x, s["act"],
                          lens=s["lens"])
    ref, end = reference(s)
    mag, _ = reference(s, magnitude=True)
    close(y, ref[..., 0], mag[..., 0], c_conv(K), dtype, "y")
    assert np.array_equal(np64(x), end)
