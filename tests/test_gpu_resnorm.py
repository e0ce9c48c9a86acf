"""GPU parity of the residual norm and of the 8-bit checkpoints against the
float64 oracle, and a block run as it would be used."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from seq_cases import (c_norm, close, dtype_of, gated_inputs, lens_of, norm_inputs, np64, say,
                       spoil_padding, torch_)

pytestmark = pytest.mark.gpu

# (B, H, L, type, layer norm, ragged): single steps, rows shorter than a strip, odd rows,
# the forms' borders in channels (forward 16 to 128, 256, 512; backward 32 to 128, 256, 512, 1024)
# and past them up to the most
SHAPES = [
    (1, 1, 1, "f32", False, False), (3, 17, 1, "bf16", True, True), (5, 2048, 1, "f16", False, False),
    (2, 2049, 1, "bf16", False, False), (2, 8192, 1, "f32", True, False),
    (2, 3, 2, "f32", True, False), (3, 5, 7, "bf16", False, True), (2, 128, 64, "f16", False, False),
    (2, 129, 65, "bf16", True, True), (3, 130, 100, "f32", False, True), (2, 256, 33, "f32", True, False),
    (2, 513, 71, "bf16", False, False), (1, 1024, 130, "f32", True, False),
    (2, 1025, 40, "f16", False, True), (1, 2048, 37, "bf16", True, False),
    (1, 2050, 21, "f32", False, False), (1, 4096, 18, "bf16", False, False),
    (1, 4100, 9, "f16", True, False), (1, 8192, 11, "f32", False, False),
    (4, 24, 3000, "bf16", False, True),
    # single steps: a wave's channels, and just past a wave's and a workgroup's
    (5, 512, 1, "f32", True, True), (3, 700, 1, "f16", True, True), (2, 4097, 1, "bf16", True, False),
    # many batch rows of one and of few steps
    (9000, 5, 1, "bf16", True, True), (5000, 40, 3, "f32", False, True),
    # few channels: wide strips
    (3, 9, 70000, "bf16", True, True), (4, 30, 33001, "f16", False, False),
    (2, 61, 65600, "f32", True, False), (3, 33, 700, "f32", False, True),
    # the most channels in strips as wide as they get, the most shared memory
    (256, 8192, 2, "bf16", True, True),
    # strips as wide as they get where channels are looped over
    (5, 514, 6700, "f16", True, True), (4, 1030, 4100, "bf16", False, False),
]
IDS = ["B%dH%dL%d-%s-%s%s" % (b, h, l, t, "layer" if n else "rms", "-ragged" if r else "")
       for b, h, l, t, n, r in SHAPES]
EPS = 1e-5


def norm_of(layer):
    return bd.NORM_LAYER if layer else bd.NORM_RMS


def prepared(B, H, L, dtype, layer, ragged, seed, joint=False):
    say("case: B=%d H=%d L=%d %s layer=%d ragged=%d seed=%d" % (B, H, L, dtype, layer, ragged, seed))
    s = norm_inputs(B, H, L, dtype, seed, joint)
    s["lens"] = lens_of(B, L, seed) if ragged else None
    if ragged:
        for k in ("x", "y", "g", "do", "dn"):
            spoil_padding(s[k], s["lens"])
    return s


def masked(a, s):
    """a with zeros behind the rows' ends."""
    a = np.nan_to_num(a)
    if s["lens"] is not None:
        for b, n in enumerate(s["lens"].tolist()):
            a[b, :, n:] = 0.0
    return a


@pytest.mark.parametrize("form", ["all", "no gate", "norm only", "stream only"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward_and_backward(shape, form):
    B, H, L, dtype, layer, ragged = shape
    torch = torch_()
    s = prepared(*shape, seed=H + L, joint=True)
    x, y, g, wo, sc, wp = (s[k] for k in ("x", "y", "g", "w_post", "scale", "w_pre"))
    do, dn = s["do"], s["dn"]
    if form == "no gate":
        g = None
        do = None
    if form == "norm only":
        y = g = None
    if form == "stream only":
        wp = dn = None
    norm = norm_of(layer)
    o, n, stats = bd.resnorm_forward_stats(x, y, g, wo, sc, wp, norm=norm, eps=EPS, lens=s["lens"])
    o2, n2 = bd.resnorm_forward(x, y, g, wo, sc, wp, norm=norm, eps=EPS, lens=s["lens"])
    for a, b in ((o, o2), (n, n2)):
        assert (a is None and b is None) or torch.equal(a, b)
    f = lambda t: None if t is None else masked(np64(t), s)
    w = [None if t is None else np64(t) for t in (wo, sc, wp)]
    c = c_norm(H)
    if y is None:
        assert o is None
        o = x
    else:
        args = (f(x), f(y), f(g), w[0], w[1], layer, EPS)
        close(o, masked(oracle.resnorm_stream(*args), s), oracle.resnorm_stream(*args, magnitude=True),
              c, dtype, "o")
    if wp is not None:
        args = (f(o), w[2], layer, EPS)
        close(n, masked(oracle.resnorm_out(*args), s), oracle.resnorm_out(*args, magnitude=True), c,
              dtype, "n")
    got = bd.resnorm_backward(o, y, g, stats, wo, sc, wp, do, dn, norm=norm, lens=s["lens"])
    args = (f(o), f(y), f(g), w[0], w[1], w[2], f(do), f(dn), layer, EPS)
    ref = oracle.resnorm_backward(*args)
    mag = oracle.resnorm_backward(*args, magnitude=True)
    # the parameters' sums: a strip's steps by shuffles, up to 8192 strips one after another
    # over 512 workgroups: 16 in a row, and the strips' own dozen
    for k, v, m in zip(("dx", "dy", "dg", "dw_post", "dscale", "dw_pre"), ref, mag):
        if v is None:
            assert got[k] is None, k
        else:
            close(got[k], v, m, 2 * c + 30, "f32" if k[1] == "w" or k == "dscale" else dtype, k)
    again = bd.resnorm_backward(o, y, g, stats, wo, sc, wp, do, dn, norm=norm, lens=s["lens"])
    for k in got:
        assert got[k] is None or torch.equal(got[k], again[k]), k + " differs between two calls"


def test_one_token_is_a_sequence_of_one():
    torch = torch_()
    s = prepared(6, 300, 1, "bf16", False, False, seed=2)
    args = (s["w_post"], s["scale"], s["w_pre"])
    o, n = bd.resnorm_forward(s["x"], s["y"], s["g"], *args)
    flat = {k: s[k][..., 0] for k in ("x", "y", "g", "do", "dn")}
    o2, n2, stats = bd.resnorm_forward_stats(flat["x"], flat["y"], flat["g"], *args)
    assert torch.equal(o[..., 0], o2) and torch.equal(n[..., 0], n2)
    a = bd.resnorm_backward(o, s["y"], s["g"], stats, *args, s["do"], s["dn"])
    b = bd.resnorm_backward(o2, flat["y"], flat["g"], stats, *args, flat["do"], flat["dn"])
    for k in a:
        assert torch.equal(a[k].reshape(b[k].shape), b[k]), k


def test_bad_columns_stay_their_own():
    """NaN and Inf in one step's channel leave every other step as it was; a
    column of zeros with eps = 0 gives NaN there only."""
    torch = torch_()
    s = prepared(2, 40, 70, "f32", True, False, seed=4)
    args = (s["w_post"], s["scale"], s["w_pre"])
    ref = bd.resnorm_forward(s["x"], s["y"], s["g"], *args, norm=bd.NORM_LAYER)
    for k, v in (("x", float("nan")), ("y", float("inf")), ("g", float("nan"))):
        t = s[k].clone()
        t[1, 7, 33] = v
        got = bd.resnorm_forward(*[t if n == k else s[n] for n in ("x", "y", "g")], *args,
                                 norm=bd.NORM_LAYER)
        for a, b in zip(got, ref):
            assert not torch.isfinite(a[1, 7, 33])
            a[1, :, 33] = b[1, :, 33]
            assert torch.equal(a, b)
    x = s["x"].clone()
    x[0, :, 5] = 0.0
    _, n = bd.resnorm_forward(x, None, None, None, None, s["w_pre"], eps=0.0)
    assert torch.isnan(n[0, :, 5]).all() and torch.isfinite(n[0, :, :5]).all()
    lens = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    _, n = bd.resnorm_forward(x, None, None, None, None, s["w_pre"], eps=0.0, lens=lens)
    assert torch.isfinite(n).all() and not n[0, :, 3:].any() and not n[1].any()


@pytest.mark.parametrize("H", [40, 600])
def test_layer_norm_far_from_zero_and_with_outliers(H):
    """Means a thousand times the spread, and a channel (the first, the last) a
    thousand times the others: no digits of the variance are lost beyond those
    of float32 values of that size."""
    torch = torch_()
    for case in ("mean", "first", "last"):
        s = prepared(2, H, 40, "f32", True, False, seed=H)
        for t in (s["x"], s["y"]):
            if case == "mean":
                t += 1000.0
            else:
                t[:, 0 if case == "first" else -1] *= 1000.0
        w = (s["w_post"], s["scale"], s["w_pre"])
        o, n = bd.resnorm_forward(s["x"], s["y"], s["g"], *w, norm=bd.NORM_LAYER, eps=EPS)
        a = [np64(t) for t in (s["x"], s["y"], s["g"]) + w[:2]] + [True, EPS]
        close(o, oracle.resnorm_stream(*a), oracle.resnorm_stream(*a, magnitude=True), c_norm(H),
              "f32", "o")
        a = [np64(o), np64(w[2]), True, EPS]
        close(n, oracle.resnorm_out(*a), oracle.resnorm_out(*a, magnitude=True), c_norm(H), "f32",
              "n")


@pytest.mark.parametrize("H,L", [(40, 70), (1100, 30), (300, 1)])
def test_large_gates(H, L):
    """Gates open and shut far beyond exp's range: silu' is 1 and 0 there, not
    what is left of the difference of two large numbers."""
    torch = torch_()
    s = prepared(2, H, L, "f32", False, False, seed=H)
    sizes = torch.tensor([0.0, 17.3, -17.3, 60.1, -60.1, 1000.3, -1000.3, 3.0e6, 1e30, -1e30,
                          torch.finfo(torch.float32).min], device="cuda")
    s["g"].copy_(sizes[torch.randint(0, 11, s["g"].shape, device="cuda")])
    s["do"] *= 2.0 ** -20  # times a gate of 1e30 it stays finite in float32
    w = (s["w_post"], s["scale"] * 2.0 ** -20, s["w_pre"])
    # a column's o is as large as its largest gate; of the gradients dg alone is looked at
    o, _, stats = bd.resnorm_forward_stats(s["x"], s["y"], s["g"], w[0], w[1], None, eps=EPS)
    got = bd.resnorm_backward(o, s["y"], s["g"], stats, w[0], w[1], None, s["do"], None)
    a = [np64(t) for t in (s["x"], s["y"], s["g"]) + w[:2]] + [False, EPS]
    # exp(-g) carries |g| log2(e) roundings of its exponent where it is not 0 or infinite
    c = c_norm(H) + 100
    with np.errstate(over="ignore"):
        close(o, oracle.resnorm_stream(*a), oracle.resnorm_stream(*a, magnitude=True), c, "f32", "o")
        a = [np64(t) for t in (o, s["y"], s["g"]) + w] + [np64(s["do"]), None, False, EPS]
        ref, mag = (oracle.resnorm_backward(*a, magnitude=m) for m in (False, True))
    assert torch.equal(got["dx"], s["do"])
    close(got["dg"], ref[2], mag[2], 2 * c + 30, "f32", "dg")


def test_no_steps():
    torch = torch_()
    s = prepared(2, 9, 4, "f32", False, False, seed=6)
    w = (s["w_post"], s["scale"], s["w_pre"])
    for cut in ((slice(0, 0),), (slice(None), slice(None), slice(0, 0))):
        z = s["x"][cut].contiguous()
        o, n, stats = bd.resnorm_forward_stats(z, z, z, *w)
        got = bd.resnorm_backward(o, z, z, stats, *w, z, z)
        for k in ("dw_post", "dscale", "dw_pre"):
            assert got[k].shape == (9,) and not got[k].any()


def test_captured_and_replayed():
    torch = torch_()
    s = prepared(2, 200, 300, "f16", True, False, seed=8)
    keys = ("x", "y", "g", "do", "dn", "w_post", "scale", "w_pre")

    def both():
        w = (s["w_post"], s["scale"], s["w_pre"])
        o, n, stats = bd.resnorm_forward_stats(s["x"], s["y"], s["g"], *w, norm=bd.NORM_LAYER)
        g = bd.resnorm_backward(o, s["y"], s["g"], stats, *w, s["do"], s["dn"], norm=bd.NORM_LAYER)
        return [o, n] + list(g.values())

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for rep in range(4):
        new = prepared(2, 200, 300, "f16", True, False, seed=80 + rep)
        for k in keys:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, both()):
            assert torch.equal(a, b), rep


def test_resnorm_binding_refuses():
    torch = torch_()
    s = prepared(2, 20, 30, "f16", False, False, seed=10)
    x, y, g, w = s["x"], s["y"], s["g"], (s["w_post"], s["scale"], s["w_pre"])
    for bad in ((x, y.float(), g), (x, y[:, :10], g), (x.transpose(1, 2), y.transpose(1, 2), None),
                (x, None, g), (x[0, 0], None, None), (x, y.cpu(), g)):
        with pytest.raises((ValueError, TypeError)):
            bd.resnorm_forward(*bad, *w)
    with pytest.raises(ValueError):
        bd.resnorm_forward(x, None, None, None, None, None)
    with pytest.raises(ValueError):
        bd.resnorm_forward(x, y, g, s["w_post"][:5].contiguous(), *w[1:])
    with pytest.raises((ValueError, TypeError)):
        bd.resnorm_forward(x, y, g, None, *w[1:])
    o, n, stats = bd.resnorm_forward_stats(x, y, g, *w)
    with pytest.raises(ValueError):  # the layer norm keeps twice as much
        bd.resnorm_backward(o, y, g, stats, *w, s["do"], s["dn"], norm=bd.NORM_LAYER)
    with pytest.raises(bd.DSSMError):
        bd.resnorm_backward(o, y, g, stats, *w, None, None)


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1,), (7,), (64,), (65,), (3, 100), (2, 3, 1000), (5, 1), (4, 16384),
                                   (3000, 130)])
def test_ckpt8_round_trip(shape, dtype):
    """Bit for bit what the oracle decodes, rounded once to the type."""
    torch = torch_()
    say("case:", shape, dtype)
    g = np.random.default_rng(sum(shape))
    x = g.normal(size=shape) * np.exp(g.uniform(-6, 6, size=shape[:-1] + (1,)))
    x = torch.from_numpy(x.astype(np.float32)).cuda().to(dtype_of(dtype))
    blob = bd.ckpt8_pack(x)
    assert blob.numel() == max(bd.ckpt8_size(shape), 256)
    ref = torch.from_numpy(oracle.ckpt8(np64(x)))
    assert torch.equal(bd.ckpt8_unpack(blob, shape, torch.float32).cpu(), ref.float())
    assert torch.equal(bd.ckpt8_unpack(blob, shape, x.dtype).cpu(), ref.to(x.dtype))


def test_ckpt8_borders():
    """Powers of two, 127 and just past it, zeros, subnormals, the largest
    values, Inf and NaN."""
    torch = torch_()
    rows = [[0.0] * 64, [-0.0] * 64, [127.0, 1.5, 0.5, -2.5] + [0.0] * 60,
            [127.00001, 1.0] + [0.0] * 62, [127.5, 3.0] + [0.0] * 62,
            [1e-45, 1e-40] + [0.0] * 62, [2.0 ** -126, 2.0 ** -127] + [0.0] * 62,
            [3.4028235e38, 1e38] + [1.0] * 62, [2.0 ** k for k in range(-32, 32)],
            [float("inf"), 1.0] + [0.0] * 62, [float("nan"), 1.0] + [0.0] * 62,
            [float("-inf"), float("nan")] + [5.0] * 62]
    x = torch.tensor(rows, dtype=torch.float32, device="cuda")
    x = torch.cat([x, torch.ones(len(rows), 3, device="cuda")], 1)  # a second, short group
    got = np64(bd.ckpt8_unpack(bd.ckpt8_pack(x), x.shape, torch.float32))
    ref = oracle.ckpt8(np64(x))
    assert np.array_equal(got, ref, equal_nan=True)
    assert np.isnan(got[-3:, :64]).all() and (got[:, 64:] == 1.0).all()
    for name, largest in (("f16", 65504.0), ("bf16", 3.3895313892515355e38)):
        x = torch.full((2, 64), largest, dtype=dtype_of(name), device="cuda")
        x[1] = -x[1]
        got = np64(bd.ckpt8_unpack(bd.ckpt8_pack(x), x.shape, x.dtype))
        assert np.isfinite(got).all() and np.array_equal(got, oracle.ckpt8(np64(x), largest))


def test_ckpt8_refuses():
    torch = torch_()
    x = torch.zeros(4, 70, device="cuda")
    with pytest.raises(ValueError):
        bd.ckpt8_pack(x.t())
    with pytest.raises(TypeError):
        bd.ckpt8_pack(x.double())
    with pytest.raises(ValueError):
        bd.ckpt8_pack(x, blob=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        bd.ckpt8_unpack(bd.ckpt8_pack(x), (400, 70), torch.float32)
    with pytest.raises(TypeError):
        bd.ckpt8_unpack(bd.ckpt8_pack(x), (4, 70), torch.int32)
    assert bd.ckpt8_unpack(bd.ckpt8_pack(x[:0]), (0, 70), torch.float32).shape == (0, 70)


# ---------------------------------------------------------------------------
# a block, as it would be used
# ---------------------------------------------------------------------------

def test_block_trains_and_decodes():
    """Norm, joint projection, gated recurrence, gate and residual, next norm: a
    training step's gradients against differences of its own float64 form, and
    the same weights run token by token against the whole sequence."""
    torch = torch_()
    B, H, L = 2, 24, 90
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s, sd=1.0: torch.randn(*s, generator=gen, device="cuda") * sd
    w_in = rand(4 * H, H, sd=H ** -0.5)
    prm = dict(w0=1 + rand(H, sd=0.1), w_post=1 + rand(H, sd=0.1), scale=rand(H, sd=0.5),
               w_pre=1 + rand(H, sd=0.1), log_re=rand(H, sd=0.5))
    x, do, dn = rand(B, H, L), rand(B, H, L), rand(B, H, L)
    # forward
    _, n0, st0 = bd.resnorm_forward_stats(x, None, None, None, None, prm["w0"])
    p = torch.matmul(w_in, n0)
    u, r, i, g = (p[:, k * H:(k + 1) * H] for k in range(4))
    y, ckpt = bd.gated_forward_ckpt(u, r, i, prm["log_re"])
    o, n, st1 = bd.resnorm_forward_stats(x, y, g, prm["w_post"], prm["scale"], prm["w_pre"])
    # backward
    dp = torch.empty_like(p)
    d1 = bd.resnorm_backward(o, y, g, st1, prm["w_post"], prm["scale"], prm["w_pre"], do, dn,
                             dg=dp[:, 3 * H:])
    d2 = bd.gated_backward(d1["dy"], ckpt, bd.CKPT_STATE, prm["log_re"], u=u, r=r, i=i,
                           du=dp[:, :H], dr=dp[:, H:2 * H], di=dp[:, 2 * H:3 * H])
    dw_in = sum(torch.matmul(dp[b], n0[b].t().contiguous()) for b in range(B))
    dn0 = torch.matmul(w_in.t().contiguous(), dp)
    d0 = bd.resnorm_backward(x, None, None, st0, None, None, prm["w0"], d1["dx"], dn0)
    got = dict(x=d0["dx"], w_in=dw_in, w0=d0["dw_pre"], w_post=d1["dw_post"], scale=d1["dscale"],
               w_pre=d1["dw_pre"], log_re=d2["dlog_re"])

    def f(v):
        n0 = oracle.resnorm_out(v["x"], v["w0"], False, 1e-6)
        p = np.einsum("kh,bhl->bkl", v["w_in"], n0)
        y, _ = oracle.gated_recurrence(p[:, :H], p[:, H:2 * H], p[:, 2 * H:3 * H], v["log_re"])
        o = oracle.resnorm_stream(v["x"], y, p[:, 3 * H:], v["w_post"], v["scale"], False, 1e-6)
        n = oracle.resnorm_out(o, v["w_pre"], False, 1e-6)
        return (np64(do) * o).sum() + (np64(dn) * n).sum()

    at = {k: np64(v) for k, v in dict(prm, x=x, w_in=w_in).items()}
    for k, d in got.items():
        e = np.random.default_rng(len(k)).normal(size=at[k].shape)
        h = 1e-5
        ref = (f({**at, k: at[k] + h * e}) - f({**at, k: at[k] - h * e})) / (2 * h)
        mine = float((np64(d) * e).sum())
        # a float32 gradient off by 2^-16 of its size in every entry, at random signs, and the
        # difference's own 1e-6 of its terms
        size = float(np.sqrt(((np64(d) * e) ** 2).sum()))
        say("  %-7s %.6e by differences %.6e" % (k, mine, ref))
        assert abs(mine - ref) <= 8 * 2.0 ** -16 * size + 1e-5 * abs(ref) + 1e-5, k
    # token by token
    state = torch.zeros(B, H, device="cuda")
    for t in range(L):
        xt = x[..., t].contiguous()
        _, nt = bd.resnorm_forward(xt, None, None, None, None, prm["w0"])
        pt = torch.matmul(nt, w_in.t().contiguous())
        ut, rt, it, gt = (pt[:, k * H:(k + 1) * H] for k in range(4))
        yt = bd.gated_step(ut, rt, it, prm["log_re"], state)
        ot, nt = bd.resnorm_forward(xt, yt, gt, prm["w_post"], prm["scale"], prm["w_pre"])
        # float32 throughout, states over 90 steps: some 2^-14 of values of order 1
        assert (ot - o[..., t]).abs().max() < 2.0 ** -14 and (nt - n[..., t]).abs().max() < 2.0 ** -13


def test_norm_offsets_past_32_bits():
    """More than 2^31 elements: the last steps of a long call against the same
    steps alone."""
    torch = torch_()
    H, L, n = 2100, 1 << 20, 96
    say("case: B=1 H=%d L=%d bf16" % (H, L))
    gen = torch.Generator(device="cuda").manual_seed(5)
    big = torch.zeros(1, H, L, dtype=torch.bfloat16, device="cuda")
    big[..., -n:] = torch.randn(1, H, n, generator=gen, device="cuda").to(big.dtype)
    w = torch.rand(H, generator=gen, device="cuda") + 0.5
    small = big[..., -n:].contiguous()
    end = lambda t: t[..., -n:].contiguous()
    o, m, stats = bd.resnorm_forward_stats(big, big, None, w, w, w)
    o2, _ = bd.resnorm_forward(small, small, None, w, w, w)
    # the backward passes from the same values, so that only sums' orders differ
    g = bd.resnorm_backward(o, big, None, stats, w, w, w, m, big)
    g2 = bd.resnorm_backward(end(o), small, None, end(stats), w, w, w, end(m), small)
    _, n1 = bd.resnorm_forward(big, None, None, None, None, w)
    _, n2 = bd.resnorm_forward(small, None, None, None, None, w)
    pairs = dict(o=(o, o2), n=(n1, n2), dx=(g["dx"], g2["dx"]), dy=(g["dy"], g2["dy"]))
    for name, (a, b) in pairs.items():
        d = (end(a).float() - b.float()).abs()
        # one rounding to bf16 may fall on either side (2^-7 of the value), or of what float32
        # leaves of terms of order 1 to 10
        worst = float((d / (2.0 ** -7 * b.float().abs() + 1e-4)).max())
        say("  %-3s worst difference / bound %.3f" % (name, worst))
        assert worst <= 1.0, (name, worst)
    x = big
    y = bd.ckpt8_unpack(bd.ckpt8_pack(x), x.shape, x.dtype)
    z = bd.ckpt8_unpack(bd.ckpt8_pack(x[0, -3:]), (3, L), x.dtype)
    assert torch.equal(y[0, -3:], z)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("H,L", [(40, 70), (300, 70), (600, 70), (1100, 70), (40, 1), (300, 1),
                                 (1100, 1), (5000, 1)])
def test_steps_behind_a_row_stay_zero_with_any_parameters(H, L, layer):
    """Infinite and NaN parameters, and finite ones whose product is past float32:
    outputs and gradients behind the rows' ends are 0 all the same, and without a
    live step the parameters' gradients too."""
    torch = torch_()
    s = prepared(3, H, L, "f32", layer, True, seed=H + L)
    s["w_post"][1], s["scale"][1] = 1e30, 1e30
    s["scale"][2], s["w_post"][3] = float("nan"), float("-inf")
    s["w_pre"][4], s["w_pre"][-1] = float("inf"), float("nan")
    w = (s["w_post"], s["scale"], s["w_pre"])
    norm = norm_of(layer)
    for lens in (s["lens"], torch.zeros_like(s["lens"])):
        for gate in (s["g"], None):
            o, n, stats = bd.resnorm_forward_stats(s["x"], s["y"], gate, *w, norm=norm, lens=lens)
            got = bd.resnorm_backward(o, s["y"], gate, stats, *w, s["do"], s["dn"], norm=norm,
                                      lens=lens)
            got.update(o=o, n=n)
            for k, t in got.items():
                if t is None:
                    continue
                if t.dim() == 1:
                    live = lens.max() > 0
                    assert live or not t.any(), k
                else:
                    for b, m in enumerate(lens.tolist()):
                        assert not t[b, :, m:].any(), (k, b, m)
