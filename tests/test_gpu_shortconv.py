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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 4, 8])
def test_stream_in_parts_and_tokens(K, dtype):
    """Parts of a sequence, some shorter than the taps, then single tokens, from the state the last
    left: the same numbers as in one call."""
    torch = torch_()
    s = prepared(3, 37, K, 700, dtype, "ab", seed=11)
    whole = bd.shortconv_forward(s["u"], s["w"], s["bias"], s["act"], x=s["x0"],
                                 x_out=torch.empty_like(s["x0"]))
    x = s["x0"].clone()
    ys = []
    for lo, hi in ((0, 1), (1, 4), (4, 600), (600, 697)):
        ys.append(bd.shortconv_forward(s["u"][..., lo:hi].contiguous(), s["w"], s["bias"], s["act"],
                                       x=x))
    for t in range(697, 700):
        ys.append(bd.shortconv_step(s["u"][..., t].contiguous(), s["w"], s["bias"], x,
                                    s["act"])[..., None])
    assert torch.equal(torch.cat(ys, -1), whole)
    assert np.array_equal(np64(x), reference(s)[1])


def test_without_a_state_and_empty_sequences():
    torch = torch_()
    s = prepared(2, 3, 4, 20, "f32", "ab", seed=3)
    a = bd.shortconv_forward(s["u"], s["w"], s["bias"])
    b = bd.shortconv_forward(s["u"], s["w"], s["bias"], x=torch.zeros_like(s["x0"]))
    assert torch.equal(a, b)
    none = s["u"][..., :0].contiguous()
    xo = torch.full_like(s["x0"], float("nan"))
    assert bd.shortconv_forward(none, s["w"], s["bias"], x=s["x0"], x_out=xo).numel() == 0
    assert torch.equal(xo, s["x0"])
    g = bd.shortconv_backward(none, none, s["w"], s["bias"], x=s["x0"], dx=s["dx"])
    assert torch.equal(g["dx0"], s["dx"]) and not g["dw"].any() and not g["dbias"].any()
    g = bd.shortconv_backward(s["dy"][:0], s["u"][:0], s["w"], s["bias"])
    assert not g["dw"].any() and not g["dbias"].any()
    # without gradients of the state on either side
    g = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"])
    h = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], x=torch.zeros_like(s["x0"]),
                              dx=torch.zeros_like(s["dx"]))
    for k in g:
        assert torch.equal(g[k], h[k]), k


@pytest.mark.parametrize("L", [9, 700])
def test_empty_rows_with_any_parameters(L):
    torch = torch_()
    s = prepared(2, 3, 4, L, "f32", "ab", seed=5)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    s["w"].fill_(float("nan"))
    s["bias"].fill_(float("inf"))
    x = s["x0"].clone()
    assert not bd.shortconv_forward(s["u"], s["w"], s["bias"], x=x, lens=lens).any()
    assert torch.equal(x, s["x0"])
    g = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], x=s["x0"], dx=s["dx"], lens=lens)
    assert torch.equal(g["dx0"], s["dx"])
    for k in ("du", "dw", "dbias"):
        assert not g[k].any(), k


@pytest.mark.parametrize("L", [40, 3000])
def test_captured_and_replayed_on_streams(L):
    """A captured forward and backward pass, replayed on new inputs with eager work on another
    stream between the replays."""
    torch = torch_()
    s = prepared(2, 6, 4, L, "bf16", "ab", seed=31)
    s["xT"] = torch.empty_like(s["x0"])

    def both(stream=None):
        y = bd.shortconv_forward(s["u"], s["w"], s["bias"], x=s["x0"], x_out=s["xT"], stream=stream)
        g = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], x=s["x0"], dx=s["dx"],
                                  stream=stream)
        return [y, s["xT"]] + [g[k] for k in ("du", "dw", "dbias", "dx0")]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    other = torch.cuda.Stream()
    for rep in range(4):
        new = prepared(2, 6, 4, L, "bf16", "ab", seed=40 + rep)
        for k in ("u", "dy", "x0", "dx", "w", "bias"):
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        torch.cuda.synchronize()
        eager = both(other)
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b), rep


def test_a_bad_row_stays_its_own_and_gradients_into_a_slice():
    torch = torch_()
    for L in (5, 40, 700):
        s = prepared(3, 5, 4, L, "bf16", "ab", seed=L)
        ref = bd.shortconv_forward(s["u"], s["w"], s["bias"])
        t = s["u"].clone()
        t[1, 2, L // 2] = float("nan")
        y = bd.shortconv_forward(t, s["w"], s["bias"])
        hit = torch.isnan(y)
        assert hit.sum() == min(4, L - L // 2) and hit[1, 2, L // 2:L // 2 + 4].all()
        assert torch.equal(y[~hit], ref[~hit])
        a = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"])
        buf = torch.full((3, 11, L), 7.0, dtype=torch.bfloat16, device="cuda")
        b = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], du=buf[:, 5:10])
        for k in a:
            assert torch.equal(a[k], b[k]), k
        assert (buf[:, :5] == 7.0).all() and (buf[:, 10:] == 7.0).all()


def test_binding_refuses():
    torch = torch_()
    s = prepared(2, 4, 3, 64, "bf16", "ab", seed=61)
    u, w, b = s["u"], s["w"], s["bias"]
    with pytest.raises(TypeError):
        bd.shortconv_forward(u.double(), w, b)
    with pytest.raises(TypeError):
        bd.shortconv_forward(u, w.bfloat16(), b)
    with pytest.raises(ValueError):
        bd.shortconv_forward(u, w[:3].contiguous(), b)
    with pytest.raises(ValueError):
        bd.shortconv_forward(u, w[:, 0].contiguous(), b)
    with pytest.raises(ValueError):
        bd.shortconv_forward(u, w, b[:3].contiguous())
    with pytest.raises(ValueError):
        bd.shortconv_forward(u, w, b, x=s["x0"][..., :1].contiguous())
    with pytest.raises(ValueError):
        bd.shortconv_forward(u[..., 0], w, b)
    with pytest.raises(ValueError):
        bd.shortconv_step(u, w, b, s["x0"])
    with pytest.raises(TypeError):
        bd.shortconv_step(u[..., 0].contiguous(), w, b, None)
    with pytest.raises(ValueError):
        bd.shortconv_forward(u.transpose(1, 2).contiguous().transpose(1, 2), w, b)
    with pytest.raises(bd.DSSMError):
        bd.shortconv_forward(u, w, b, act=3)
    with pytest.raises(bd.DSSMError):
        bd.shortconv_forward(u, torch.zeros(4, 9, device="cuda"), b)
    with pytest.raises(bd.DSSMError):
        bd.shortconv_forward(u, w, b, y=u)
    with pytest.raises(ValueError):
        bd.shortconv_backward(s["dy"], u[:, :3], w, b)


def test_offsets_past_32_bits():
    torch = torch_()
    H, L = 130, 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(1, H, L, device="cuda", generator=gen, dtype=torch.bfloat16)
    w = torch.randn(H, 4, device="cuda", generator=gen)
    y = bd.shortconv_forward(u, w)
    last = (u[:, H - 2:].contiguous(), w[H - 2:].contiguous())
    assert torch.equal(y[:, H - 2:], bd.shortconv_forward(*last))
    g = bd.shortconv_backward(y, u, w)
    h = bd.shortconv_backward(y[:, H - 2:].contiguous(), *last)
    assert torch.equal(g["du"][:, H - 2:], h["du"])
    # other segments: sums of 2^24 terms in another order
    err = (g["dw"][H - 2:] - h["dw"]).abs()
    size = (y[:, H - 2:].float().abs().mean() * 2 * 2 ** 24) * 2.0 ** -23 * 64
    assert (err <= size).all()
