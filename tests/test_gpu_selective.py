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
# whose steps are cut into segments; many rows
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,N,G", [(37, 5, 1), (6, 16, 2)])
def test_stream_in_parts_and_tokens(H, N, G, dtype):
    """Parts of a sequence, then single tokens, from the state the last left."""
    torch = torch_()
    B, L = 3, 700
    s = prepared(B, H, N, G, L, dtype, "gsb", seed=11)
    x = s["x0"].clone()
    ys = []
    prm = dict(D=s["D"], dt_bias=s["dt_bias"])
    cut = lambda k, lo, hi: s[k][..., lo:hi].contiguous()
    for lo, hi in ((0, 1), (1, 65), (65, 600), (600, 697)):
        part = [cut(k, lo, hi) for k in ("u", "delta", "Bm", "Cm")]
        ys.append(bd.selective_forward(*part, s["log_re"], z=cut("z", lo, hi), x=x, **prm))
    for t in range(697, 700):
        tok = [s[k][..., t].contiguous() for k in ("u", "delta", "Bm", "Cm")]
        ys.append(bd.selective_step(*tok, s["log_re"], x, z=s["z"][..., t].contiguous(),
                                    **prm)[..., None])
    ref, end = reference(s)
    mag, mend = reference(s, magnitude=True)
    close(torch.cat(ys, -1), ref, mag, c_selective(N, L) + 40, dtype, "y")
    close(x, end, mend, c_selective(N, L) + 40, "f32", "state")


@pytest.mark.parametrize("B,H,N,L", [(1, 2, 16, 30000), (2, 40, 7, 3000), (3, 5, 4, 300),
                                     (600, 8, 3, 140)])
def test_streaming_in_place(B, H, N, L):
    """A state that is overwritten by the row's last segment is the one its first
    segments started from."""
    torch = torch_()
    s = prepared(B, H, N, 1, L, "bf16", "sb", seed=17)
    s["log_re"].fill_(0.01)  # the state before the row is remembered to its end
    xo = torch.empty_like(s["x0"])
    y = bd.selective_forward(*args_of(s), x=s["x0"], x_out=xo, **options_of(s))
    x = s["x0"].clone()
    y2 = bd.selective_forward(*args_of(s), x=x, **options_of(s))
    assert torch.equal(y, y2) and torch.equal(x, xo)


def test_no_state_and_empty_sequences():
    torch = torch_()
    s = prepared(2, 6, 4, 2, 50, "f32", "gsb", seed=19)
    o = options_of(s)
    a = bd.selective_forward(*args_of(s), **o)
    b = bd.selective_forward(*args_of(s), x=torch.zeros_like(s["x0"]),
                             x_out=torch.empty_like(s["x0"]), **o)
    assert torch.equal(a, b)
    # no steps: the state passes, the gradients of nothing are zero
    e = {k: s[k][..., :0].contiguous() for k in ("u", "delta", "Bm", "Cm", "z", "dy")}
    five = [e["u"], e["delta"], e["Bm"], e["Cm"], s["log_re"]]
    prm = dict(D=s["D"], dt_bias=s["dt_bias"], z=e["z"])
    xo = torch.full_like(s["x0"], float("nan"))
    y, ckpt = bd.selective_forward_ckpt(*five, x=s["x0"], x_out=xo, **prm)
    assert y.shape == (2, 6, 0) and torch.equal(xo, s["x0"])
    g = bd.selective_backward(e["dy"], ckpt, *five, dx=s["dx"], **prm)
    assert torch.equal(g["dx0"], s["dx"])
    for k in ("dlog_re", "dD", "ddt_bias"):
        assert not g[k].any()
    # no rows
    none = [t[:0] for t in args_of(s)[:4]] + [s["log_re"]]
    prm["z"] = s["z"][:0]
    y, ckpt = bd.selective_forward_ckpt(*none, **prm)
    g = bd.selective_backward(s["dy"][:0], ckpt, *none, **prm)
    assert y.numel() == 0 and not g["dlog_re"].any() and not g["dD"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("L", [40, 300, 5000])
def test_masked_steps_change_nothing(L, dtype):
    """delta at -infinity or the type's lowest value: the step keeps the state, its output reads
    it, and its gradients are 0; the rest is as without the step."""
    torch = torch_()
    s = prepared(2, 5, 6, 1, L, dtype, "gsb", seed=L)
    g = np.random.default_rng(L)
    shut = torch.from_numpy(g.random(L) < 0.3).cuda()
    shut[:3] = True
    s["delta"][:, :, shut] = float("-inf")
    s["delta"][:, :, 1] = torch.finfo(s["delta"].dtype).min
    y, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=torch.empty_like(s["x0"]),
                                        **options_of(s))
    ref, _ = reference(s)
    mag, _ = reference(s, magnitude=True)
    close(y, ref, mag, c_selective(6, L), dtype, "y")
    got = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], **options_of(s))
    ref, mag = reference(s, True), reference(s, True, magnitude=True)
    for n in GRADS:
        t = "f32" if n in ("dlog_re", "dD", "ddt_bias", "dx0") else dtype
        close(got[n], ref[n], mag[n], c_selective_back(5, 6, L), t, n)
    assert not got["ddelta"][:, :, shut].any() and not got["dB"][..., shut].any()


@pytest.mark.parametrize("L", [30, 200, 4000])
def test_empty_rows_with_any_parameters(L):
    """Steps behind a row's end are 0, an empty row passes its state and gradient through and adds
    nothing to the parameters', whatever they hold."""
    torch = torch_()
    s = prepared(2, 4, 3, 1, L, "f32", "gsb", seed=5)
    s["lens"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    for k in ("log_re", "D", "dt_bias"):
        s[k].fill_(float("nan"))
    xo = torch.empty_like(s["x0"])
    y, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=xo, **options_of(s))
    assert torch.equal(xo, s["x0"]) and not y.any()
    g = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], **options_of(s))
    assert torch.equal(g["dx0"], s["dx"])
    for k in set(GRADS) - {"dx0"}:
        assert not g[k].any(), k


@pytest.mark.parametrize("L", [20, 300])
def test_parameters_past_float32(L):
    """log_re whose square float32 does not hold: no step remembers another."""
    torch = torch_()
    s = prepared(2, 3, 2, 1, L, "f32", "b", seed=13)
    s["log_re"][:] = torch.tensor([[1e20, -3e38], [float("inf"), 1e25], [2e19, 1e30]])
    y, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=torch.empty_like(s["x0"]),
                                        **options_of(s))
    u, delta, Bm, Cm = (np64(s[k]) for k in ("u", "delta", "Bm", "Cm"))
    dt = np.logaddexp(0, delta + np64(s["dt_bias"])[None, :, None])
    ref = (Cm * Bm).sum(2) * dt * u
    close(y, ref, np.abs(Cm * Bm).sum(2) * dt * np.abs(u), c_selective(2, L), "f32", "y")
    g = bd.selective_backward(s["dy"], ckpt, *args_of(s), **options_of(s))
    assert not g["dlog_re"].any() and not g["dx0"].any()
    dy = np64(s["dy"])
    close(g["du"], (Cm * Bm).sum(2) * dt * dy, np.abs(Cm * Bm).sum(2) * dt * np.abs(dy),
          c_selective_back(3, 2, L), "f32", "du")


def test_a_bad_row_stays_its_own():
    """NaN and Inf in one row's inputs leave every other row as it was."""
    torch = torch_()
    for L in (5, 40, 700, 6000):
        s = prepared(2, 7, 5, 1, L, "f32", "gsb", seed=L)
        o = options_of(s)
        ref, ckpt = bd.selective_forward_ckpt(*args_of(s), **o)
        back = bd.selective_backward(s["dy"], ckpt, *args_of(s), **o)
        for k, v in (("u", float("inf")), ("delta", float("nan")), ("z", float("nan"))):
            t = s[k].clone()
            t[1, 2, L // 2] = v
            bad = {**s, k: t}
            y, ckpt = bd.selective_forward_ckpt(*args_of(bad), **options_of(bad))
            assert not torch.isfinite(y[1, 2, L // 2])
            y[1, 2] = ref[1, 2]
            assert torch.equal(y, ref)
            g = bd.selective_backward(bad["dy"], ckpt, *args_of(bad), **options_of(bad))
            for n in ("du", "ddelta", "dz", "dx0"):
                g[n][1, 2] = back[n][1, 2]
                assert torch.equal(g[n], back[n]), (k, n)
            assert torch.equal(g["dB"][0], back["dB"][0]) and torch.equal(g["dC"][0], back["dC"][0])


def test_slowest_modes():
    """Modes that remember the whole row: decays next to 1 do not add up their roundings."""
    torch = torch_()
    s = prepared(1, 3, 4, 1, 40000, "f32", "b", seed=23)
    s["log_re"].copy_(torch.tensor([0.002, 0.01, 0.03, 0.1]).cuda().expand(3, 4))
    s["dt_bias"].fill_(-2.0)
    s["delta"].mul_(0.1)
    xo = torch.empty_like(s["x0"])
    y = bd.selective_forward(*args_of(s), x=s["x0"], x_out=xo, **options_of(s))
    ref, end = reference(s)
    rel = np.linalg.norm(np64(y) - ref) / np.linalg.norm(ref)
    rel_x = np.linalg.norm(np64(xo) - end) / np.linalg.norm(end)
    say("  relative error of y %.2e, of the state %.2e" % (rel, rel_x))
    # 313 tiles of 7 joins, each rounded once (2^-24): 1.3e-4 at worst, and the root of their
    # number of it where they do not all fall on one side
    assert rel < 2.0 ** -24 * 4 * np.sqrt(313 * 7) and rel_x < 2.0 ** -24 * 4 * np.sqrt(313 * 7)


def test_gradients_into_slices_of_one_buffer():
    torch = torch_()
    B, H, N, G, L = 3, 10, 4, 2, 130
    s = prepared(B, H, N, G, L, "bf16", "gsbj", seed=21)
    _, ckpt = bd.selective_forward_ckpt(*args_of(s), **options_of(s))
    a = bd.selective_backward(s["dy"], ckpt, *args_of(s), **options_of(s))
    buf = torch.full((B, 3 * H + 1, L), 7.0, dtype=torch.bfloat16, device="cuda")
    proj = torch.full((B, 2 * G * N + 3, L), 7.0, dtype=torch.bfloat16, device="cuda")
    b = bd.selective_backward(s["dy"], ckpt, *args_of(s), du=buf[:, :H], ddelta=buf[:, H:2 * H],
                              dz=buf[:, 2 * H:3 * H], dB=proj[:, :G * N].unflatten(1, (G, N)),
                              dC=proj[:, G * N:2 * G * N].unflatten(1, (G, N)), **options_of(s))
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert (buf[:, 3 * H:] == 7.0).all() and (proj[:, 2 * G * N:] == 7.0).all()


@pytest.mark.parametrize("shape", [(2, 6, 5, 2, 40), (2, 6, 5, 2, 300), (1, 4, 16, 1, 9000)])
def test_captured_and_replayed(shape):
    """Two captured graphs of a forward and backward pass that share a workspace, replayed in turn
    on new inputs with eager work between the replays."""
    torch = torch_()
    B, H, N, G, L = shape
    s = prepared(*shape, "bf16", "gsb", seed=31)
    s["xT"] = torch.empty_like(s["x0"])
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")

    def both():
        y, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=s["xT"], workspace=ws,
                                            **options_of(s))
        g = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], workspace=ws,
                                  **options_of(s))
        return [y, s["xT"]] + [g[k] for k in GRADS]

    both()
    torch.cuda.synchronize()
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held.append(both())
    for rep in range(4):
        new = prepared(*shape, "bf16", "gsb", seed=40 + rep)
        for k in ("u", "delta", "Bm", "Cm", "z", "dy", "x0", "dx", "log_re", "D", "dt_bias"):
            s[k].copy_(new[k])
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held[rep % 2]]
        graphs[1 - rep % 2].replay()
        for a, b, c in zip(got, both(), held[1 - rep % 2]):
            assert torch.equal(a, b) and torch.equal(c, b), rep


def test_on_other_streams_at_once():
    torch = torch_()
    sets = [prepared(2, 5, 6, 1, L, "f32", "gsb", seed=52 + L) for L in (60, 9000)]

    def both(s, stream=None):
        y, ckpt = bd.selective_forward_ckpt(*args_of(s), stream=stream, **options_of(s))
        g = bd.selective_backward(s["dy"], ckpt, *args_of(s), stream=stream, **options_of(s))
        return [y] + [g[k] for k in GRADS]

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


def test_gradients_against_differences():
    """The device's gradients along random directions against central differences of its own
    float32 outputs: step 1e-2, values of order 1, sums of 500 terms with roundings of 1e-6."""
    torch = torch_()
    s = prepared(2, 4, 3, 2, 60, "f32", "gsb", seed=71)
    g = np.random.default_rng(72)

    def f(t):
        xo = torch.empty_like(t["x0"])
        y = bd.selective_forward(*args_of(t), x=t["x0"], x_out=xo, **options_of(t))
        return (np64(y) * np64(s["dy"])).sum() + (np64(xo) * np64(s["dx"])).sum()

    _, ckpt = bd.selective_forward_ckpt(*args_of(s), x=s["x0"], x_out=torch.empty_like(s["x0"]),
                                        **options_of(s))
    got = bd.selective_backward(s["dy"], ckpt, *args_of(s), dx=s["dx"], **options_of(s))
    for name, key in (("u", "du"), ("delta", "ddelta"), ("z", "dz"), ("Bm", "dB"), ("Cm", "dC"),
                      ("log_re", "dlog_re"), ("D", "dD"), ("dt_bias", "ddt_bias"), ("x0", "dx0")):
        d = torch.from_numpy(g.normal(size=tuple(s[name].shape)).astype(np.float32)).cuda()
        d /= d.norm()
        h = 1e-2
        num = (f({**s, name: s[name] + h * d}) - f({**s, name: s[name] - h * d})) / (2 * h)
        ana = float((np64(got[key]) * np64(d)).sum())
        scale = float(np.linalg.norm(np64(got[key])))
        say("  %s: %.6f against %.6f" % (name, ana, num))
        # the third derivative's share h^2 / 6 times a few times the gradient's size, and the
        # outputs' roundings, 1e-6 of sums of size 100, over h
        assert abs(num - ana) <= 1e-3 * scale + 1e-2, name


def test_more_gradient_parts_than_workgroups():
    """A group per channel and many modes: dB and dC by workgroups that take turns.  One step
    from no state has dB = C dy dt u and dC = B dy dt u: the step size's rounding (2e-7, its
    polynomial's among it) and four products'."""
    torch = torch_()
    B, H, N = 2, 16400, 128
    gen = torch.Generator("cuda").manual_seed(3)
    u, delta, dy = [torch.randn(B, H, 1, device="cuda", generator=gen) for _ in range(3)]
    Bm, Cm = [torch.randn(B, H, N, 1, device="cuda", generator=gen) for _ in range(2)]
    log_re = torch.rand(H, N, device="cuda", generator=gen)
    y, ckpt = bd.selective_forward_ckpt(u, delta, Bm, Cm, log_re)
    g = bd.selective_backward(dy, ckpt, u, delta, Bm, Cm, log_re)
    drive = (dy.double() * torch.nn.functional.softplus(delta.double()) * u.double())[:, :, None]
    for got, ref in ((g["dB"], Cm.double() * drive), (g["dC"], Bm.double() * drive)):
        assert ((got.double() - ref).abs() <= 2.0 ** -21 * ref.abs()).all()


def test_binding_refuses():
    torch = torch_()
    s = prepared(2, 4, 3, 2, 64, "bf16", "gsb", seed=61)
    u, delta, Bm, Cm, lr = args_of(s)
    with pytest.raises(TypeError):
        bd.selective_forward(u, delta.float(), Bm, Cm, lr)
    with pytest.raises(TypeError):
        bd.selective_forward(u, delta, Bm.float(), Cm.float(), lr)
    with pytest.raises(TypeError):
        bd.selective_forward(u, delta, Bm, Cm, lr.bfloat16())
    with pytest.raises(TypeError):
        bd.selective_forward(u.double(), delta.double(), Bm.double(), Cm.double(), lr)
    for bad in (Bm[..., :32], Bm[:1], Bm[:, :1], Bm.transpose(2, 3), Bm.cpu(), Bm.flatten(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            bd.selective_forward(u, delta, bad, Cm, lr)
    with pytest.raises(ValueError):  # three channels do not make two groups
        bd.selective_forward(u[:, :3].contiguous(), delta[:, :3].contiguous(), Bm, Cm, lr[:3])
    with pytest.raises(ValueError):
        bd.selective_forward(u, delta, Bm, Cm, lr[:, :2].contiguous())
    with pytest.raises(ValueError):
        bd.selective_forward(u, delta, Bm, Cm, lr, D=s["D"][:3].contiguous())
    with pytest.raises(ValueError):
        bd.selective_forward(u, delta, Bm, Cm, lr, x=s["x0"][:, :3].contiguous())
    with pytest.raises(ValueError):
        bd.selective_forward(u, delta, Bm, Cm, lr, lens=torch.zeros(3, dtype=torch.int32,
                                                                    device="cuda"))
    with pytest.raises(bd.DSSMError):
        bd.selective_forward(u, delta, Bm, Cm, lr, y=u)
    _, ckpt = bd.selective_forward_ckpt(u, delta, Bm, Cm, lr)
    with pytest.raises(TypeError):
        bd.selective_backward(s["dy"], None, u, delta, Bm, Cm, lr)
    with pytest.raises(ValueError):
        bd.selective_backward(s["dy"], ckpt, u, delta, Bm, Cm, lr, dz=torch.empty_like(u))
    with pytest.raises(ValueError):
        bd.selective_backward(s["dy"], ckpt[:16], u, delta, Bm, Cm, lr)
    with pytest.raises(bd.DSSMError) as e:
        bd.selective_backward(s["dy"], ckpt, u, delta, Bm, Cm, lr,
                              workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bd.DSSM_ERR_WORKSPACE
    with pytest.raises(ValueError):
        bd.selective_step(u, delta, Bm, Cm, lr, s["x0"])
    many = torch.zeros(1, 1, 200, 4, device="cuda")
    with pytest.raises(bd.DSSMError) as e:
        bd.selective_forward(torch.zeros(1, 2, 4, device="cuda"), torch.zeros(1, 2, 4, device="cuda"),
                             many, many, torch.zeros(2, 200, device="cuda"))
    assert e.value.status == bd.DSSM_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last channels of a long bank against the same channels alone
    (other segments: the same up to roundings)."""
    torch = torch_()
    H, L, N = 132, 1 << 24, 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(1, H, L, device="cuda", generator=gen, dtype=torch.bfloat16)
    delta = torch.randn(1, H, L, device="cuda", generator=gen, dtype=torch.bfloat16)
    Bm, Cm = (torch.randn(1, 1, N, L, device="cuda", generator=gen).to(torch.bfloat16)
              for _ in range(2))
    log_re = torch.full((H, N), 0.3, device="cuda")
    y, ckpt = bd.selective_forward_ckpt(u, delta, Bm, Cm, log_re)
    last = [t[:, H - 4:].contiguous() for t in (u, delta)] + [Bm, Cm, log_re[H - 4:].contiguous()]
    y2, ckpt2 = bd.selective_forward_ckpt(*last)
    say("  forward done")
    # both are roundings (2^-9) of sums whose terms, at most 30 of size 1, carry c 2^-23
    slack = 30 * c_selective(N, 256) * 2.0 ** -23
    near = lambda a, b: ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + slack).all()
    assert near(y[:, H - 4:], y2)
    del y, y2
    g = bd.selective_backward(u, ckpt, u, delta, Bm, Cm, log_re)
    g2 = bd.selective_backward(last[0], ckpt2, *last)
    say("  backward done")
    for k in ("du", "ddelta"):
        # y counts twice: the gradient's sums are of such terms again
        a, b = g[k][:, H - 4:].float(), g2[k].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 30 * slack).all(), k
