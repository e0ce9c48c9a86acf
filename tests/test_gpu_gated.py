"""GPU parity of the gated recurrence (forward, streaming, one token, backward
from kept states and from 8 bits) against the float64 oracle."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from seq_cases import (KINDS, STEP, c_gated, close, dtype_of, gated_inputs, lens_of, np64, say,
                       spoil_padding, torch_)

pytestmark = pytest.mark.gpu

# (B, H, L, type, ragged): rows inside a lane, inside a wave, over several tiles of one wave
# (many rows), of four waves, and split into segments; lengths around every border
SHAPES = [
    (2, 3, 1, "f32", False), (3, 5, 7, "bf16", True), (4, 3, 8, "f16", True), (2, 3, 9, "f32", False),
    (3, 7, 63, "bf16", True), (3, 2, 64, "f32", True), (4, 3, 65, "f16", False),
    (5, 3, 300, "f32", True), (2, 3, 511, "bf16", False), (3, 3, 512, "f32", True),
    (3, 3, 513, "f32", True), (4, 5, 2047, "f16", True), (2, 3, 2048, "bf16", False),
    (2, 3, 2049, "f32", False), (3, 2, 6145, "f32", True), (1, 1, 20000, "f32", False),
    (4, 131, 2100, "bf16", True), (4, 2049, 530, "f16", True), (8, 1024, 1030, "f32", False),
    # the most channels, many batch rows
    (2, 65535, 3, "bf16", True), (40000, 3, 9, "f16", True),
    # many segments, and segments of several tiles
    (1, 2, 150000, "f32", False), (3, 85, 30000, "bf16", True),
]
IDS = ["B%dH%dL%d-%s%s" % (b, h, l, t, "-ragged" if r else "") for b, h, l, t, r in SHAPES]


def prepared(B, H, L, dtype, ragged, seed, joint=False):
    say("case: B=%d H=%d L=%d %s ragged=%d seed=%d" % (B, H, L, dtype, ragged, seed))
    s = gated_inputs(B, H, L, dtype, seed, joint)
    s["lens"] = lens_of(B, L, seed) if ragged else None
    if ragged:
        for k in ("u", "r", "i", "dy"):
            spoil_padding(s[k], s["lens"])
    return s


def gate8(t):
    """A gate's logit as an 8-bit checkpoint bounds it."""
    return np.clip(t, -31.75, 31.75)


def reference(s, **kw):
    a = [np64(s[k]) for k in ("u", "r", "i", "log_re")]
    lens = None if s["lens"] is None else s["lens"].cpu().numpy()
    if s["lens"] is not None:
        a[:3] = [np.nan_to_num(t) for t in a[:3]]
    return oracle.gated_recurrence(*a, x0=np64(s["x0"]), lens=lens, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_state(shape):
    B, H, L, dtype, ragged = shape
    torch = torch_()
    s = prepared(*shape, seed=L + H, joint=L % 2 == 1)
    xo = torch.full_like(s["x0"], float("nan"))
    y = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"], x_out=xo, lens=s["lens"])
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(y, ref, mag, c_gated(L), dtype, "y")
    close(xo, end, mend, c_gated(L), "f32", "state")


@pytest.mark.parametrize("kind", ["state", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, kind):
    B, H, L, dtype, ragged = shape
    torch = torch_()
    s = prepared(*shape, seed=2 * L + H, joint=L % 2 == 0)
    k = KINDS[kind]
    y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], k, x=s["x0"],
                                    x_out=torch.empty_like(s["x0"]), lens=s["lens"])
    plain = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"],
                             x_out=torch.empty_like(s["x0"]), lens=s["lens"])
    assert torch.equal(y, plain)
    kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == "state" else {}
    got = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], lens=s["lens"], **kept)
    lens = None if s["lens"] is None else s["lens"].cpu().numpy()
    u, r, i, dy = (np.nan_to_num(np64(s[n])) for n in ("u", "r", "i", "dy"))
    nch = -(-L // 512)
    # the states a checkpoint begins with are the forward pass's own
    starts = np64(ckpt[:4 * B * H * nch].view(torch.float32).view(B, H, nch))
    if kind == "int8":
        u, r, i = oracle.ckpt8(u), oracle.ckpt8(gate8(r)), oracle.ckpt8(gate8(i))
    args = (u, r, i, np64(s["log_re"]), dy, np64(s["dx"]), np64(s["x0"]), lens, starts)
    ref = oracle.gated_backward(*args)
    mag = oracle.gated_backward(*args, magnitude=True)
    for n, v, m, t in zip(("du", "dr", "di", "dlog_re", "dx0"), ref, mag,
                          (dtype, dtype, dtype, "f32", "f32")):
        close(got[n], v, m, 2 * c_gated(L), t, n)
    if ragged:
        for b, n in enumerate(lens):
            assert not np64(got["du"])[b, :, n:].any()
    again = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], lens=s["lens"], **kept)
    for n in got:
        assert torch.equal(got[n], again[n]), n + " differs between two calls"


def test_kept_states_are_the_forward_passes():
    torch = torch_()
    s = prepared(2, 3, 1700, "f32", False, seed=5)
    _, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"],
                                    x_out=torch.empty_like(s["x0"]))
    y, _ = reference(s)
    mag, _ = reference(s, magnitude=True)
    got = ckpt[:4 * 6 * 4].view(torch.float32).view(2, 3, 4)
    assert torch.equal(got[..., 0], s["x0"])
    for c in (1, 2, 3):
        close(got[..., c], y[..., c * 512 - 1], mag[..., c * 512 - 1], c_gated(1700), "f32", "start")


def test_eight_bits_hold_what_the_oracle_says():
    """The three blobs of a checkpoint decode to the oracle's values, bit for bit."""
    torch = torch_()
    for L, ragged in ((70, True), (1000, False), (5, True)):
        s = prepared(3, 4, L, "bf16", ragged, seed=L)
        _, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], bd.CKPT_INT8,
                                        lens=s["lens"])
        off = (4 * 12 * -(-L // 512) + 255) // 256 * 256
        n = bd.ckpt8_size((3, 4, L))
        for k, name in enumerate(("u", "r", "i")):
            got = bd.ckpt8_unpack(ckpt[off + k * n:off + (k + 1) * n], (3, 4, L), torch.float32)
            ref = np.nan_to_num(np64(s[name]))
            assert np.array_equal(np64(got), oracle.ckpt8(ref if name == "u" else gate8(ref))), name


@pytest.mark.parametrize("kind", ["state", "int8"])
@pytest.mark.parametrize("mask", [float("-inf"), None, float("inf")])
def test_masked_gates(mask, kind):
    """Steps shut or opened by an infinite logit or the type's lowest value, whole
    groups and rows of them: a shut step keeps the state and has no gradient of
    its input; everything is finite and, from 8 bits too, the oracle's."""
    torch = torch_()
    B, H, L = 2, 3, 700
    s = prepared(B, H, L, "bf16", False, seed=71)
    value = torch.finfo(torch.bfloat16).min if mask is None else mask
    shut = torch.rand(B, 1, L, device="cuda") < 0.2
    shut[0, 0, 64:200] = True
    shut[1] = True
    for k in ("r", "i"):
        s[k] = s[k].masked_fill(shut, value)
    k = KINDS[kind]
    y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], k, x=s["x0"],
                                    x_out=torch.empty_like(s["x0"]))
    big = lambda t: np.clip(np64(t), -1e30, 1e30)
    a = [np64(s["u"]), big(s["r"]), big(s["i"]), np64(s["log_re"])]
    ref, _ = oracle.gated_recurrence(*a, x0=np64(s["x0"]))
    mag, _ = oracle.gated_recurrence(*a, x0=np64(s["x0"]), magnitude=True)
    close(y, ref, mag, c_gated(L), "bf16", "y")
    kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == "state" else {}
    got = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], **kept)
    starts = np64(ckpt[:4 * B * H * 2].view(torch.float32).view(B, H, 2))
    if kind == "int8":
        a[:3] = oracle.ckpt8(a[0]), oracle.ckpt8(gate8(a[1])), oracle.ckpt8(gate8(a[2]))
    elif value < 0:
        assert not got["du"][shut.expand_as(y)].any()
    args = a + [np64(s["dy"]), np64(s["dx"]), np64(s["x0"]), None, starts]
    # a logit of 31.75 carries 31.75 log2(e) roundings of its exponent, twice
    c = 2 * (c_gated(L) + 100)
    for n, v, m in zip(("du", "dr", "di", "dlog_re", "dx0"), oracle.gated_backward(*args),
                       oracle.gated_backward(*args, magnitude=True)):
        close(got[n], v, m, c, "f32" if n in ("dlog_re", "dx0") else "bf16", n)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_stream_in_parts_and_tokens(dtype):
    """Parts of a sequence, then single tokens, from the state the last left."""
    torch = torch_()
    B, H, L = 3, 37, 700
    s = prepared(B, H, L, dtype, False, seed=11)
    x = s["x0"].clone()
    ys = []
    for lo, hi in ((0, 1), (1, 600), (600, 697)):
        part = [s[k][:, :, lo:hi].contiguous() for k in ("u", "r", "i")]
        ys.append(bd.gated_forward(*part, s["log_re"], x=x))
    for t in range(697, 700):
        tok = [s[k][:, :, t].contiguous() for k in ("u", "r", "i")]
        ys.append(bd.gated_step(*tok, s["log_re"], x)[..., None])
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(torch.cat(ys, -1), ref, mag, c_gated(L) + 40, dtype, "y")
    close(x, end, mend, c_gated(L) + 40, "f32", "state")


@pytest.mark.parametrize("B,H,dtype", [(1, 1, "f32"), (5, 63, "bf16"), (3, 1000, "f16"),
                                       (64, 4096, "bf16"), (7, 2049, "f32"), (3, 65535, "f16")])
def test_step(B, H, dtype):
    """One token: slices of a joint projection, idle streams, old states kept."""
    torch = torch_()
    s = prepared(B, H, 1, dtype, False, seed=B + H, joint=True)
    u, r, i = (s[k][..., 0] for k in ("u", "r", "i"))
    s["lens"] = torch.tensor([b % 3 for b in range(B)], dtype=torch.int32, device="cuda")
    for b in range(0, B, 3):
        for t in (u, r, i):
            t[b] = float("nan")
    xo = torch.empty_like(s["x0"])
    before = s["x0"].clone()
    y = bd.gated_step(u, r, i, s["log_re"], s["x0"], x_out=xo, lens=s["lens"])
    assert torch.equal(s["x0"], before)
    s["lens"] = s["lens"].clamp(max=1)
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(y[..., None], ref, mag, 64, dtype, "y")
    close(xo, end, mend, 64, "f32", "state")
    assert torch.equal(xo[::3], before[::3])
    y2 = bd.gated_step(u, r, i, s["log_re"], s["x0"], lens=s["lens"])
    assert torch.equal(y2, y) and torch.equal(s["x0"], xo)


def test_no_state_and_empty_sequences():
    torch = torch_()
    s = prepared(2, 3, 100, "f32", False, seed=3)
    y = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"])
    z = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=torch.zeros_like(s["x0"]))
    assert torch.equal(y, z)
    none = s["u"][..., :0].contiguous()
    xo = torch.full_like(s["x0"], float("nan"))
    y, ckpt = bd.gated_forward_ckpt(none, none, none, s["log_re"], x=s["x0"], x_out=xo)
    assert y.shape == (2, 3, 0) and torch.equal(xo, s["x0"])
    g = bd.gated_backward(none, ckpt, bd.CKPT_STATE, s["log_re"], u=none, r=none, i=none,
                          dx=s["dx"])
    assert torch.equal(g["dx0"], s["dx"]) and not g["dlog_re"].any()
    none = s["u"][:0].contiguous()
    y, ckpt = bd.gated_forward_ckpt(none, none, none, s["log_re"])
    g = bd.gated_backward(none, ckpt, bd.CKPT_STATE, s["log_re"], u=none, r=none, i=none)
    assert y.shape == (0, 3, 100) and g["du"].shape == (0, 3, 100)
    assert g["dlog_re"].shape == (3,) and not g["dlog_re"].any()


def test_extreme_gates_and_parameters():
    """log_re of 0 and tiny ones (no decay, no drive), gates open and shut beyond
    exp's range: finite, and the oracle's values."""
    torch = torch_()
    B, H, L = 2, 6, 530
    s = prepared(B, H, L, "f32", False, seed=9)
    s["log_re"][:] = torch.tensor([0.0, -0.0, 1e-22, 1e-12, 3e-4, 30.0])
    s["r"][0, :, :100], s["r"][0, :, 100:200] = 200.0, -200.0
    s["i"][1, :, :100], s["i"][1, :, 100:200] = 200.0, -200.0
    y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"],
                                    x_out=torch.empty_like(s["x0"]))
    ref, _ = reference(s)
    mag, _ = reference(s, magnitude=True)
    # 1 - a^2 below 2^-126 counts as 0, so sqrt(1 - a^2) is off by up to 2^-63 in every step: at
    # most L values of u, G or u G below 2^6 add that up where nothing decays.  close() multiplies
    # a magnitude by c STEP, so the sum is divided by it.
    lost = L * 2.0 ** 6 * 2.0 ** -63
    # exp(-r log2(e)) at |r| = 200 carries 2 * 200 more roundings of its exponent
    c = c_gated(L) + 400
    close(y, ref, mag + lost / (c * STEP), c, "f32", "y")
    got = bd.gated_backward(s["dy"], ckpt, bd.CKPT_STATE, s["log_re"], u=s["u"], r=s["r"],
                            i=s["i"], dx=s["dx"])
    starts = np64(ckpt[:4 * B * H * 2].view(torch.float32).view(B, H, 2))
    args = tuple(np64(s[k]) for k in ("u", "r", "i", "log_re", "dy", "dx", "x0")) + (None, starts)
    r, m = oracle.gated_backward(*args), oracle.gated_backward(*args, magnitude=True)
    for n, v, g in zip(("du", "dr", "di", "dlog_re", "dx0"), r, m):
        if n == "dlog_re":  # the channels whose 1 - a^2 is below float32's range count it as 0
            assert torch.isfinite(got[n]).all() and not got[n][:2].any()
            close(got[n][3:], v[3:], g[3:], 2 * c, "f32", n)
        else:
            close(got[n], v, g + lost / (2 * c * STEP), 2 * c, "f32", n)


@pytest.mark.parametrize("L", [40, 700, 5000])
def test_parameters_past_float32(L):
    """log_re whose square float32 does not hold: no step remembers another, and
    what is masked stays 0."""
    torch = torch_()
    B, H = 3, 3
    s = prepared(B, H, L, "f32", True, seed=13)
    s["log_re"][:] = torch.tensor([1e20, -3e38, float("inf")])
    s["r"].clamp_(-5, 5)
    y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"],
                                    x_out=torch.empty_like(s["x0"]), lens=s["lens"])
    got = bd.gated_backward(s["dy"], ckpt, bd.CKPT_STATE, s["log_re"], u=s["u"], r=s["r"],
                            i=s["i"], lens=s["lens"])
    for b, n in enumerate(s["lens"].tolist()):
        u, i, dy = (np64(s[k])[b, :, :n] for k in ("u", "i", "dy"))
        sig = 1.0 / (1.0 + np.exp(-i))
        close(y[b, :, :n], sig * u, np.abs(sig * u), c_gated(L), "f32", "y")
        close(got["du"][b, :, :n], sig * dy, np.abs(sig * dy), 2 * c_gated(L), "f32", "du")
        assert not got["dr"][b].any()
        for t in (y, got["du"], got["di"]):
            assert not t[b, :, n:].any()


@pytest.mark.parametrize("B,H,L", [(1, 2, 60000), (2, 100, 20000), (3, 5, 2100)])
def test_streaming_in_place_over_split_rows(B, H, L):
    """A state that is overwritten by the row's last segment is the one its
    first segments started from."""
    torch = torch_()
    s = prepared(B, H, L, "bf16", False, seed=17)
    s["log_re"].fill_(0.02)  # the state before the row is remembered to its end
    xo = torch.empty_like(s["x0"])
    y = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"], x_out=xo)
    x = s["x0"].clone()
    y2 = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=x)
    assert torch.equal(y, y2) and torch.equal(x, xo)


def test_a_bad_row_stays_its_own():
    """NaN and Inf in one row's inputs leave every other row as it was."""
    torch = torch_()
    for L in (5, 40, 700):
        s = prepared(3, 5, L, "f32", False, seed=L)
        ref = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"])
        for k, v in (("u", float("inf")), ("r", float("nan")), ("i", float("nan"))):
            t = s[k].clone()
            t[1, 2, L // 2] = v
            y = bd.gated_forward(*[t if n == k else s[n] for n in ("u", "r", "i")], s["log_re"])
            assert not torch.isfinite(y[1, 2, L // 2])
            y[1, 2] = ref[1, 2]
            assert torch.equal(y, ref)


def test_gradients_into_slices_of_one_buffer():
    torch = torch_()
    B, H, L = 3, 10, 130
    s = prepared(B, H, L, "bf16", False, seed=21, joint=True)
    _, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"])
    kept = dict(u=s["u"], r=s["r"], i=s["i"])
    a = bd.gated_backward(s["dy"], ckpt, bd.CKPT_STATE, s["log_re"], **kept)
    buf = torch.full((B, 3 * H + 1, L), 7.0, dtype=torch.bfloat16, device="cuda")
    b = bd.gated_backward(s["dy"], ckpt, bd.CKPT_STATE, s["log_re"], du=buf[:, :H],
                          dr=buf[:, H:2 * H], di=buf[:, 2 * H:3 * H], **kept)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert (buf[:, 3 * H:] == 7.0).all()


@pytest.mark.parametrize("shape", [(2, 3, 300), (2, 3, 9000)])
def test_captured_and_replayed(shape):
    """A captured forward and backward pass, replayed on new inputs with eager
    work between the replays."""
    torch = torch_()
    B, H, L = shape
    s = prepared(B, H, L, "bf16", False, seed=31)

    def both():
        y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], bd.CKPT_INT8,
                                        x=s["x0"], x_out=s["xT"])
        g = bd.gated_backward(s["dy"], ckpt, bd.CKPT_INT8, s["log_re"], dx=s["dx"])
        return [y, s["xT"]] + [g[k] for k in ("du", "dr", "di", "dlog_re", "dx0")]

    s["xT"] = torch.empty_like(s["x0"])
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for rep in range(4):
        new = prepared(B, H, L, "bf16", False, seed=40 + rep)
        for k in ("u", "r", "i", "dy", "x0", "dx", "log_re"):
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, both()):
            assert torch.equal(a, b), rep


def test_on_another_stream():
    torch = torch_()
    s = prepared(2, 4, 3000, "f32", False, seed=51)
    ref = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], stream=st)
    st.synchronize()
    assert torch.equal(y, ref)


def test_two_streams_at_once():
    """Calls under way on two streams, their workspaces the binding's own."""
    torch = torch_()
    sets = [prepared(2, 5, 9000, "f32", False, seed=52 + k) for k in range(2)]

    def both(s, stream=None):
        y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], bd.CKPT_INT8,
                                        stream=stream)
        g = bd.gated_backward(s["dy"], ckpt, bd.CKPT_INT8, s["log_re"], stream=stream)
        return [y] + [g[k] for k in ("du", "dr", "di", "dlog_re", "dx0")]

    ref = [both(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(8):
        for k in range(2):
            got[k].append(both(sets[k], streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(run, ref[k]))


def test_binding_refuses():
    torch = torch_()
    s = prepared(2, 4, 64, "bf16", False, seed=61)
    u, r, i, lr = s["u"], s["r"], s["i"], s["log_re"]
    with pytest.raises(TypeError):
        bd.gated_forward(u, r.float(), i, lr)
    with pytest.raises(TypeError):
        bd.gated_forward(u.double(), r.double(), i.double(), lr)
    with pytest.raises(TypeError):
        bd.gated_forward(u, r, i, lr.bfloat16())
    for bad in (r[:, :, :32], r.transpose(1, 2).contiguous().transpose(1, 2), r.cpu(),
                torch.empty(2, 8, 64, dtype=r.dtype, device="cuda")[:, ::2]):
        with pytest.raises((ValueError, TypeError)):
            bd.gated_forward(u, bad, i, lr)
    wide = torch.zeros(2, 12, 64, dtype=r.dtype, device="cuda")
    with pytest.raises(ValueError):  # another batch stride than u's
        bd.gated_forward(u, wide[:, :4], i, lr)
    with pytest.raises(ValueError):
        bd.gated_forward(wide[:, :4], wide[:, 4:8], i, lr)
    with pytest.raises(ValueError):
        bd.gated_forward(u.expand(2, 4, 64), r[:1].expand(2, 4, 64), i, lr)
    with pytest.raises(ValueError):
        bd.gated_forward(u, r, i, lr[:3].contiguous())
    with pytest.raises(TypeError):
        bd.gated_forward(u, r, i, lr, lens=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        bd.gated_forward(u, r, i, lr, lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        bd.gated_forward(u, r, i, lr, y=torch.empty(2, 64, 4, dtype=u.dtype, device="cuda"))
    with pytest.raises(bd.DSSMError):
        bd.gated_forward(u, r, i, lr, y=u)
    with pytest.raises(bd.DSSMError) as e:
        bd.gated_forward(u, r, i, lr, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bd.DSSM_ERR_WORKSPACE
    _, ckpt = bd.gated_forward_ckpt(u, r, i, lr)
    with pytest.raises(ValueError):
        bd.gated_backward(s["dy"], ckpt, bd.CKPT_STATE, lr)
    with pytest.raises(ValueError):
        bd.gated_backward(s["dy"], ckpt, bd.CKPT_INT8, lr)  # too small for 8 bits
    with pytest.raises(ValueError):
        bd.gated_backward(s["dy"], ckpt, bd.CKPT_INT8, lr, u=u, r=r, i=i)
    with pytest.raises(ValueError):
        bd.gated_step(u, r, i, lr, s["x0"])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last channels of a long bank against the same
    channels alone (other segments: the same up to roundings), forward, 8 bits
    and backward."""
    torch = torch_()
    H, L = 130, 1 << 24
    say("case: B=1 H=%d L=%d bf16" % (H, L))
    log_re = torch.full((H,), 0.2, device="cuda")
    big = {k: torch.zeros(1, H, L, dtype=torch.bfloat16, device="cuda") for k in ("u", "r", "i", "dy")}
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in big.values():
        t[0, -2:] = torch.randn(2, L, generator=gen, device="cuda").to(t.dtype)
    small = {k: t[:, -2:].contiguous() for k, t in big.items()}
    for kind in (bd.CKPT_STATE, bd.CKPT_INT8):
        out = []
        for s, lr in ((big, log_re), (small, log_re[-2:].contiguous())):
            y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], lr, kind)
            kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == bd.CKPT_STATE else {}
            g = bd.gated_backward(s["dy"], ckpt, kind, lr, **kept)
            out.append([t[:, -2:].clone() for t in (y, g["du"], g["dr"], g["di"])])
            del y, ckpt, g
        for name, a, b in zip(("y", "du", "dr", "di"), *out):
            # one rounding to bf16 may fall on either side: 2^-7 of the value, or of what
            # float32 leaves of values of order 1
            d = (a.float() - b.float()).abs()
            worst = float((d / (2.0 ** -7 * b.float().abs() + 1e-5)).max())
            say("  kind %d %-3s worst difference / bound %.3f" % (kind, name, worst))
            assert worst <= 1.0, (kind, name, worst)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,H,L", [(1, 64, 1), (1, 64, 300), (1, 64, 600), (2, 200, 2100), (2, 4096, 600)])
def test_drive_of_one_open_step(B, H, L, dtype):
    """One open step among shut ones leaves sqrt(1 - a^2) sigmoid(i) u in the state
    to float32's digits, whatever the activations' type.

    In half steps h = 2^-24, x = 2 log_re^2 sigmoid(r): the exponent's two products
    and its constant 3 h; the series of 1 - exp(-x) another 5 h (its first
    coefficient, its last sum and product, h for the terms before, h for the one
    left out); the root halves these 8 h and adds 2 h of its own; sigmoid(0) = 1/2,
    u = 1 and the shut steps are exact.  6 h in all, and one for products of them."""
    torch = torch_()
    say("case: B=%d H=%d L=%d %s" % (B, H, L, dtype))
    dt = dtype_of(dtype)
    x = torch.linspace(0.02, 0.49, H, dtype=torch.float64)
    log_re = x.sqrt().float()
    ref = (0.5 * torch.sqrt(-torch.expm1(-log_re.double() ** 2))).expand(B, H).numpy()
    u, i = torch.ones(B, H, L, device="cuda").to(dt), torch.zeros(B, H, L, device="cuda").to(dt)
    r = torch.full((B, H, L), float("-inf"), device="cuda").to(dt)
    r[..., L // 3] = 0.0

    def near(got, what):
        worst = float(np.max(np.abs(np64(got) - ref) / (7 * 2.0 ** -24 * ref)))
        say("  %-6s worst error / tolerance %.3f" % (what, worst))
        assert worst <= 1.0, (what, worst)

    end = torch.empty(B, H, device="cuda")
    lr = log_re.cuda()
    y, ckpt = bd.gated_forward_ckpt(u, r, i, lr, x_out=end)
    near(end, "state")
    for c in range(1, -(-L // 512)):
        if c * 512 > L // 3:
            near(ckpt[:4 * B * H * -(-L // 512)].view(torch.float32).view(B, H, -1)[..., c], "kept")
    if dtype == "f32":
        near(y[..., -1], "y")
    if L == 1:
        state = torch.zeros(B, H, device="cuda")
        bd.gated_step(u[..., 0], r[..., 0], i[..., 0], lr, state)
        near(state, "token")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [float("-inf"), None])
def test_steps_shut_by_the_recurrence_gate_alone(mask, dtype):
    """With i open and u large, a row shut by r keeps its state and, from kept
    states, has no gradient but dx0; from 8 bits its drive is at most 2^-22
    |log_re| sigmoid(i) u (r counts as -31.75, sqrt(2 sigmoid(-31.75)) = 2^-22.4:
    the factor 2^0.4 holds all roundings, the type's among them), and so are the
    gradients: with G = dx, du = G drive / u, di = G drive (1 - sigmoid(i)),
    dr = G drive / 2, dlog_re = sum G drive / log_re."""
    torch = torch_()
    B, H, L = 2, 5, 700
    s = prepared(B, H, L, dtype, False, seed=73)
    s["dy"].zero_()
    s["r"].fill_(torch.finfo(s["r"].dtype).min if mask is None else mask)
    s["u"].mul_(1000.0)
    G = np.abs(np64(s["dx"]))[..., None]
    u, i, lr = np.abs(np64(s["u"])), np64(s["i"]), np.abs(np64(s["log_re"]))[None, :, None]
    # u and i as 8 bits hold them: at most half a unit of their group's largest more
    u = u + np.abs(u).max() / 127
    sig = 1.0 / (1.0 + np.exp(-(i + np.abs(i).max() / 127)))
    drive = 2.0 ** -22 * lr * sig * u
    for kind in ("state", "int8"):
        k = KINDS[kind]
        y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], k, x=s["x0"],
                                        x_out=torch.empty_like(s["x0"]))
        assert torch.equal(y, s["x0"][..., None].to(y.dtype).expand(B, H, L))
        kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == "state" else {}
        got = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], **kept)
        if kind == "state":
            assert torch.equal(got["dx0"], s["dx"])
            assert not any(got[n].any() for n in ("du", "dr", "di", "dlog_re"))
            continue
        assert np.allclose(np64(got["dx0"]), np64(s["dx"]), rtol=2.0 ** -20, atol=0)
        bounds = dict(du=G * drive / u, di=G * drive, dr=G * (drive / 2 + lr * lr * 2.0 ** -45 *
                                                              np.abs(np64(y)).max()))
        for n, b in bounds.items():
            worst = float((np.abs(np64(got[n])) / b).max())
            say("  %-7s largest / bound %.3f" % (n, worst))
            assert worst <= 1.0, (n, worst)
        b = (G * (drive / lr + 2 * lr * 2.0 ** -45 * np.abs(np64(y)).max())).sum(axis=(0, 2))
        worst = float((np.abs(np64(got["dlog_re"])) / b).max())
        say("  dlog_re largest / bound %.3f" % worst)
        assert worst <= 1.0, worst


@pytest.mark.parametrize("kind,dtype", [("state", "f32"), ("int8", "bf16")])
@pytest.mark.parametrize("tiles,rest", [(255, 77), (256, 5), (511, 900)])
def test_many_segments_remember_each_other(tiles, rest, kind, dtype):
    """A few rows of just over 255, 256 and 511 tiles of 2048 steps: 256 segments of
    one tile, 129 and 256 of two.  Each channel is driven in one tile alone (the
    last one by the state before the row) and read back in another, and forgets
    nearly nothing in between, so what every segment passes on is seen by itself
    at the far end, in either direction."""
    torch = torch_()
    B, H, L = 1, 8, tiles * 2048 + rest
    s = prepared(B, H, L, dtype, False, seed=75)
    first = [0, 1, 3, 75, 76, 128, 254, None]
    far = [tiles, tiles, 200, 254, 0, 2, 1, tiles]
    driven = torch.zeros(B, H, L, dtype=torch.bool, device="cuda")
    asked = torch.zeros_like(driven)
    for h in range(H):
        if first[h] is not None:
            driven[:, h, first[h] * 2048:(first[h] + 1) * 2048] = True
        asked[:, h, far[h] * 2048:(far[h] + 1) * 2048] = True
    # one sign each, so that a sum is as large as its terms
    s["u"] = s["u"].abs() * driven
    s["dy"] = s["dy"].abs() * asked
    s["x0"] = s["x0"].abs() * torch.tensor([0.0] * 7 + [1.0], device="cuda")
    s["dx"] = s["dx"].abs() * torch.tensor([1.0] + [0.0] * 7, device="cuda")
    s["log_re"] = torch.full((H,), 1e-3, device="cuda") * torch.tensor([1.0, -1.0] * 4, device="cuda")
    k = KINDS[kind]
    end = torch.empty_like(s["x0"])
    y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], k, x=s["x0"], x_out=end)
    ref, last = reference(s)
    mag, mlast = reference(s, magnitude=True)
    close(y, ref, mag, c_gated(L), dtype, "y")
    close(end, last, mlast, c_gated(L), "f32", "state")
    kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == "state" else {}
    got = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], **kept)
    u, r, i = (np64(s[n]) for n in ("u", "r", "i"))
    if kind == "int8":
        u, r, i = oracle.ckpt8(u), oracle.ckpt8(gate8(r)), oracle.ckpt8(gate8(i))
    nch = -(-L // 512)
    starts = np64(ckpt[:4 * B * H * nch].view(torch.float32).view(B, H, nch))
    args = (u, r, i, np64(s["log_re"]), np64(s["dy"]), np64(s["dx"]), np64(s["x0"]), None, starts)
    ref, mag = oracle.gated_backward(*args), oracle.gated_backward(*args, magnitude=True)
    for n, v, m in zip(("du", "dr", "di", "dlog_re", "dx0"), ref, mag):
        close(got[n], v, m, 2 * c_gated(L), "f32" if n in ("dlog_re", "dx0") else dtype, n)


@pytest.mark.parametrize("L", [1, 5, 40, 300, 700, 2100, 9000])
def test_empty_rows_with_any_parameters(L):
    """An empty row passes its state and its state's gradient through and has no
    other, whatever its channels' parameters; without a live step the parameters'
    gradients are 0."""
    torch = torch_()
    B, H = 3, 3
    s = prepared(B, H, L, "f32", False, seed=77)
    s["log_re"][:] = torch.tensor([float("nan"), float("inf"), 0.3])
    for lens in ([L, 0, 0], [0, 0, 0]):
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for kind, k in KINDS.items():
            end = torch.empty_like(s["x0"])
            y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], k, x=s["x0"],
                                            x_out=end, lens=lens)
            kept = dict(u=s["u"], r=s["r"], i=s["i"]) if kind == "state" else {}
            got = bd.gated_backward(s["dy"], ckpt, k, s["log_re"], dx=s["dx"], lens=lens, **kept)
            empty = lens == 0
            assert torch.equal(end[empty], s["x0"][empty])
            assert torch.equal(got["dx0"][empty], s["dx"][empty])
            for t in (y, got["du"], got["dr"], got["di"]):
                assert not t[empty].any()
            if empty.all():
                assert not got["dlog_re"].any()
