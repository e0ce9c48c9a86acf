"""The operators of a selective state space block, case by case, for timing and comparison.

Three operators over activations [B, H, L] (time fastest), as the layer forward takes them:

* the selective scan: per channel N real modes whose step size, drive and read-out come with every
  step, in streaming (a state in and out), one-token and training form:
  dt = softplus(delta + dt_bias), x_t = exp(-log_re^2 dt) x_{t-1} + dt B_t u_t,
  y_t = (sum_n C_t x_t + D u_t) silu(z_t);
* the short causal convolution ahead of it, its last inputs carried as a state, with its gradients;
* the residual sum and norm ahead of the next projection, its output in 8 bits with a scale per
  step, channels fastest, as a product in 8 bits reads it.

`own` false: plain torch operations in 32 bits.  `own` true: the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token for a small batch: latency
        dict(name="scan_token", kind="scan_step", B=8, H=1024, N=16, G=1, L=1, dtype="bf16",
             gate=True, skip=True),
        # one generated token for a server's batch: the states are the traffic
        dict(name="scan_token_server", kind="scan_step", B=256, H=4096, N=16, G=1, L=1,
             dtype="bf16", gate=True, skip=True),
        # prompts of different lengths in one padded batch
        dict(name="scan_prompts", kind="scan", B=4, H=2048, N=16, G=1, L=2048, dtype="bf16",
             gate=True, skip=True, ragged=True),
        # a long sequence of few channels in float32, continued from a state
        dict(name="scan_long", kind="scan", B=1, H=128, N=16, G=1, L=65536, dtype="f32",
             gate=False, skip=True, ragged=False),
        # the largest: a wide layer's training step
        dict(name="scan_train_wide", kind="scan_train", B=4, H=2048, N=16, G=1, L=4096,
             dtype="bf16", gate=True, skip=True, ragged=False),
        # odd sizes, two groups, a padded batch, neither gate nor skip
        dict(name="scan_train_odd", kind="scan_train", B=3, H=130, N=13, G=2, L=1001, dtype="f16",
             gate=False, skip=False, ragged=True),
        # as many modes as the layer's own workloads have, in float32
        dict(name="scan_train_modes", kind="scan_train", B=2, H=256, N=64, G=4, L=4096,
             dtype="f32", gate=True, skip=True, ragged=False),
        # the convolution's part of one generated token
        dict(name="conv_token", kind="conv_step", B=64, H=4096, K=4, L=1, dtype="bf16", act=True),
        # prompts of different lengths in one padded batch
        dict(name="conv_prompts", kind="conv", B=8, H=2048, K=4, L=2048, dtype="bf16", act=True,
             ragged=True),
        # training in float32, odd length and more taps
        dict(name="conv_train", kind="conv_train", B=4, H=1024, K=7, L=8191, dtype="f32",
             act=True, ragged=False),
        # ahead of the next product: one generated token of a server's batch
        dict(name="norm8_token", kind="norm8", B=64, H=4096, L=1, dtype="bf16", layer=False,
             post=False, form="int8"),
        # a wide layer's block, with the gate and norm after the layer, for float8 products
        dict(name="norm8_wide", kind="norm8", B=4, H=2048, L=4096, dtype="bf16", layer=False,
             post=True, form="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["scan_step", "scan", "scan", "scan_train", "scan_train", "conv_step", "conv",
                       "conv_train", "norm8", "norm8"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    case = dict(kind=kind, dtype=dtype)
    token = kind.endswith("_step") or (kind == "norm8" and rng.random() < 0.4)
    if kind.startswith("scan"):
        # state elements: at most half of the largest listed case
        most = 1 << 28
        N = _log_int(rng, 1, 128)
        L = 1 if token else _log_int(rng, 1, 65536 if kind == "scan" else 16384)
        heads = _log_int(rng, 1, min(4096, max(1, min(1 << 25, most // N) // L)))
        G = rng.choice([1, 1, 2, 4]) if heads >= 4 else 1
        H = heads // G * G
        B = _log_int(rng, 1, max(1, min(256 if token else 16, min(1 << 24, most // N) // (L * H))))
        case.update(B=B, H=H, N=N, G=G, L=L, gate=rng.random() < 0.6, skip=rng.random() < 0.7)
        if not token:
            case["ragged"] = rng.random() < 0.5
        return case
    most = 1 << 25
    L = 1 if token else _log_int(rng, 1, 32768)
    H = _log_int(rng, 16, min(8192 if kind == "norm8" else 4096, max(16, most // L)))
    B = _log_int(rng, 1, max(1, min(256 if token else 16, most // (L * H))))
    case.update(B=B, H=H, L=L)
    if kind == "norm8":
        case.update(layer=rng.random() < 0.3, post=rng.random() < 0.5,
                    form=rng.choice(["int8", "e4m3"]))
        return case
    case.update(K=rng.choice([2, 3, 4, 4, 5, 8]), act=rng.random() < 0.7)
    if not token:
        case["ragged"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _make(case, seed):
    """Inputs on the GPU, from the seed alone."""
    B, H, L, kind = case["B"], case["H"], case["L"], case["kind"]
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, mean=0.0, dtype=dt):
        t = torch.randn(*shape, generator=gen, device="cuda")
        return (t * sd + mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def part(rows, first, count, sd=1.0):
        """`count` of the `rows` channels that one joint projection gives, as a slice of them."""
        if L == 1:
            return normal(B, count, sd=sd)
        p = torch.empty(B, rows, L, dtype=dt, device="cuda")
        p[:, first:first + count] = normal(B, count, L, sd=sd)
        return p[:, first:first + count]

    s = {"lens": None}
    if case.get("ragged"):
        # the longest fills the batch, the others end anywhere
        s["lens"] = (uniform(B, lo=0.1) * L).to(torch.int32)
        s["lens"][0] = L
    if kind.startswith("scan"):
        N, G = case["N"], case["G"]
        flat = kind == "scan_step"
        s["u"] = normal(B, H) if flat else normal(B, H, L)
        s["delta"] = normal(B, H, sd=0.7) if flat else normal(B, H, L, sd=0.7)
        # read-in and read-out lie behind a few channels that feed the step sizes
        s["Bm"] = part(8 + 2 * G * N, 8, G * N).unflatten(1, (G, N))
        s["Cm"] = part(8 + 2 * G * N, 8 + G * N, G * N).unflatten(1, (G, N))
        s["z"] = part(2 * H, H, H) if case["gate"] else None
        # modes spread as the layer's real initialisation spreads them, steps of 1e-3 .. 1e-1
        modes = torch.arange(1, N + 1, device="cuda").float()
        s["log_re"] = torch.sqrt(modes)[None] * (1.0 + 0.1 * uniform(H, N, lo=-1.0))
        step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = torch.log(torch.expm1(step)) if case["skip"] else None
        s["D"] = normal(H, dtype=torch.float32) if case["skip"] else None
        if not case["skip"]:
            s["delta"] = (s["delta"].float() - 4.0).to(dt)
        s["x0"] = normal(B, H, N, sd=0.3, dtype=torch.float32)
        if kind == "scan_train":
            s["dy"] = normal(B, H, L)
            s["dx"] = normal(B, H, N, dtype=torch.float32)
    elif kind.startswith("conv"):
        K = case["K"]
        s["u"] = part(2 * H, 0, H)
        s["w"] = uniform(H, K, lo=-1.0) * math.sqrt(1.0 / K)
        s["bias"] = uniform(H, lo=-0.5, hi=0.5)
        # the inputs before the first one, in the activations' type
        s["x0"] = normal(B, H, K - 1).float()
        if kind == "conv_train":
            s["dy"] = normal(B, H, L)
            s["dx"] = normal(B, H, K - 1, dtype=torch.float32)
    else:
        shape = (B, H) if L == 1 else (B, H, L)
        s["x"], s["y"] = normal(*shape, sd=2.0), normal(*shape, sd=0.7, mean=0.1)
        s["w_pre"] = normal(H, sd=0.2, mean=1.0, dtype=torch.float32)
        s["g"] = s["w_post"] = s["scale"] = None
        if case["post"]:
            s["g"] = normal(*shape, sd=1.5)
            s["w_post"] = normal(H, sd=0.2, mean=1.0, dtype=torch.float32)
            s["scale"] = normal(H, sd=0.1, mean=0.3, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    if "x0" in s:
        s["x"] = torch.empty_like(s["x0"])  # the state after the call; x0 is kept, as for a retry
    s["case"] = case
    return s


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------

def _run_own(s):
    from long_convolution_sequence_amd import binding as bd

    case = s["case"]
    kind = case["kind"]
    if kind == "scan_step":
        y = bd.selective_step(s["u"], s["delta"], s["Bm"], s["Cm"], s["log_re"], s["x0"], D=s["D"],
                              dt_bias=s["dt_bias"], z=s["z"], x_out=s["x"])
        return y, s["x"]
    if kind.startswith("scan"):
        prm = dict(D=s["D"], dt_bias=s["dt_bias"], z=s["z"], lens=s["lens"])
        args = (s["u"], s["delta"], s["Bm"], s["Cm"], s["log_re"])
        if kind == "scan":
            return bd.selective_forward(*args, x=s["x0"], x_out=s["x"], **prm), s["x"]
        y, ckpt = bd.selective_forward_ckpt(*args, x=s["x0"], x_out=s["x"], **prm)
        g = bd.selective_backward(s["dy"], ckpt, *args, dx=s["dx"], **prm)
        return (y, s["x"]) + tuple(g[k] for k in ("du", "ddelta", "dB", "dC", "dz", "dlog_re", "dD",
                                                  "ddt_bias", "dx0"))
    act = bd.ACT_SILU if case.get("act") else bd.ACT_NONE
    if kind == "conv_step":
        y = bd.shortconv_step(s["u"], s["w"], s["bias"], s["x0"], act=act, x_out=s["x"])
        return y, s["x"]
    if kind.startswith("conv"):
        y = bd.shortconv_forward(s["u"], s["w"], s["bias"], act=act, x=s["x0"], x_out=s["x"],
                                 lens=s["lens"])
        if kind == "conv":
            return y, s["x"]
        g = bd.shortconv_backward(s["dy"], s["u"], s["w"], s["bias"], act=act, x=s["x0"],
                                  dx=s["dx"], lens=s["lens"])
        return y, s["x"], g["du"], g["dw"], g["dbias"], g["dx0"]
    o, q, qs = bd.resnorm8_forward(
        s["x"], s["y"], s["g"], s["w_post"], s["scale"], s["w_pre"],
        norm=bd.NORM_LAYER if case["layer"] else bd.NORM_RMS, eps=EPS,
        form=bd.Q8_INT8 if case["form"] == "int8" else bd.Q8_E4M3)
    # the values the 8 bits stand for, as a product in bfloat16 would take them
    return o, (q.float() * qs[..., None]).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scan(a, b, x0):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = x0 over the last axis, by doubling, in the type of a;
    32 bits out."""
    b = b.to(a.dtype)
    b = torch.cat([b[..., :1] + a[..., :1] * x0[..., None], b[..., 1:]], -1)
    o = 1
    while o < b.shape[-1]:
        b = torch.cat([b[..., :o], b[..., o:] + a[..., o:] * b[..., :-o]], -1)
        a = torch.cat([a[..., :o], a[..., o:] * a[..., :-o]], -1)
        o *= 2
    return b.float()


def _valid(lens, L, device):
    """[B, 1, L]: which steps are live, or None for all."""
    if lens is None:
        return None
    return (torch.arange(L, device=device)[None, :] < lens[:, None])[:, None, :]


def _only(t, valid):
    return t if valid is None else torch.where(valid, t, torch.zeros_like(t))


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _spread(t, H):
    """[B, G, N, L] -> [B, H, N, L]: every head reads its group's."""
    return t.float().repeat_interleave(H // t.shape[1], dim=1)


def _run_scan_plain(s):
    case = s["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    flat = kind == "scan_step"
    wide = (lambda t: t[..., None]) if flat else (lambda t: t)
    u, delta = wide(s["u"]).float(), wide(s["delta"]).float()
    B, H, L = u.shape
    G = case["G"]
    Bm, Cm = _spread(wide(s["Bm"]), H), _spread(wide(s["Cm"]), H)
    valid = _valid(s["lens"], L, u.device)
    pre = delta if s["dt_bias"] is None else delta + s["dt_bias"][None, :, None]
    step = _only(_softplus(pre), valid)  # past a row's end the state stays
    u = _only(u, valid)
    if valid is not None:
        Bm, Cm = _only(Bm, valid[:, :, None]), _only(Cm, valid[:, :, None])
    re2 = (s["log_re"] * s["log_re"])[None, :, :, None]
    # the slowest modes remember thousands of steps, and as many roundings next to 1 add up
    e = -re2 * step[:, :, None]
    a = torch.exp(e if L == 1 else e.double())
    h = _scan(a, (step * u)[:, :, None] * Bm, s["x0"])
    yh = (Cm * h).sum(2)
    if s["D"] is not None:
        yh = yh + s["D"][None, :, None] * u
    y = yh
    if s["z"] is not None:
        z = wide(s["z"]).float()
        sg = torch.sigmoid(z)
        y = _only(yh * (z * sg), valid)
    y = y.to(dt)
    if flat:
        return y[..., 0], h[..., -1]
    xT = h[..., -1].contiguous()
    if kind == "scan":
        return y, xT
    dy = _only(s["dy"].float(), valid)
    dz = None
    if s["z"] is not None:
        dz = _only(dy * yh * sg * (1.0 + z * (1.0 - sg)), valid).to(dt)
        dy = _only(dy * (z * sg), valid)
    # the state's gradient, from the last step back
    c = Cm * dy[:, :, None]
    c[..., -1] += s["dx"]
    nxt = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    Gr = _scan(nxt.flip(-1), c.flip(-1), torch.zeros_like(s["x0"])).flip(-1)
    a = a.float()
    w = Gr * (a * torch.cat([s["x0"][..., None], h[..., :-1]], -1))  # times the decayed state
    gb = (Gr * Bm).sum(2)
    du = step * gb
    if s["D"] is not None:
        du = du + s["D"][None, :, None] * dy
    dstep = u * gb - (re2 * w).sum(2)
    ddelta = _only(dstep * torch.sigmoid(pre), valid)
    group = lambda t: t.unflatten(1, (G, H // G)).sum(2).to(dt)
    dB = group(Gr * (step * u)[:, :, None])
    dC = group(h * dy[:, :, None])
    total = lambda t: t.double().sum((0, -1))
    dlog = (-2.0 * s["log_re"].double() * total(w * step[:, :, None])).float()
    return (y, xT, _only(du, valid).to(dt), ddelta.to(dt), dB, dC, dz, dlog,
            None if s["D"] is None else total(dy * u).float(),
            None if s["dt_bias"] is None else total(ddelta).float(), a[..., 0] * Gr[..., 0])


def _run_conv_plain(s):
    case = s["case"]
    kind, dt, K = case["kind"], DTYPES[case["dtype"]], case["K"]
    u = s["u"].float()
    if kind == "conv_step":
        u = u[..., None]
    B, H, L = u.shape
    valid = _valid(s["lens"], L, u.device)
    u = _only(u, valid)
    ext = torch.cat([s["x0"], u], -1)
    w = s["w"]
    pre = s["bias"][None, :, None] + sum(w[None, :, k, None] * ext[..., k:k + L] for k in range(K))
    sg = torch.sigmoid(pre)
    y = _only(pre * sg if case["act"] else pre, valid).to(dt)
    if valid is None:
        end = ext[..., L:].contiguous()
    else:
        at = s["lens"].long()[:, None, None] + torch.arange(K - 1, device=u.device)
        end = torch.gather(ext, 2, at.expand(B, H, K - 1))
    if kind == "conv_step":
        return y[..., 0], end
    if kind == "conv":
        return y, end
    dp = _only(s["dy"].float(), valid)
    if case["act"]:
        dp = dp * (sg * (1.0 + pre * (1.0 - sg)))
    dext = torch.zeros_like(ext)
    for k in range(K):
        dext[..., k:k + L] += w[None, :, k, None] * dp
    if valid is None:
        dext[..., L:] += s["dx"]
    else:
        dext.scatter_add_(2, at.expand(B, H, K - 1), s["dx"])
    total = lambda t: t.double().sum((0, -1)).float()
    dw = torch.stack([total(dp * ext[..., k:k + L]) for k in range(K)], -1)
    du = _only(dext[..., K - 1:], valid).to(dt)
    return y, end, du, dw, total(dp), dext[..., :K - 1].contiguous()


def _norm_plain(t, layer):
    d = t - t.mean(1, keepdim=True) if layer else t
    return d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)


def _run_norm8_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x, y = s["x"].float(), s["y"].float()
    flat = x.dim() == 2
    wide = (lambda t: t[..., None]) if flat else (lambda t: t)
    x, y = wide(x), wide(y)
    if case["post"]:
        g = wide(s["g"].float())
        col = lambda t: t[None, :, None]
        y = _norm_plain(y, case["layer"]) * (col(s["w_post"]) * col(s["scale"]))
        y = y * (g * torch.sigmoid(g))
    o = (x + y).to(dt)
    # the norm is of the stream as it is stored
    n = _norm_plain(o.float(), case["layer"]) * s["w_pre"][None, :, None]
    top = 127.0 if case["form"] == "int8" else 448.0
    unit = n.abs().amax(1, keepdim=True) / top
    q = n / unit
    q = torch.round(q) if case["form"] == "int8" else q.to(torch.float8_e4m3fn).float()
    v = (q * unit).to(torch.bfloat16).transpose(1, 2)
    return (o[..., 0], v[:, 0]) if flat else (o, v)


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind.startswith("scan"):
        return _run_scan_plain(state)
    if kind.startswith("conv"):
        return _run_conv_plain(state)
    return _run_norm8_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B, H, L, kind = case["B"], case["H"], case["L"], case["kind"]
    n, e = B * H * L, BYTES[case["dtype"]]
    if kind.startswith("scan"):
        N, bc = case["N"], 2 * B * case["G"] * case["N"] * L * e
        z = 1 if case["gate"] else 0
        prm = 4 * H * N + (8 * H if case["skip"] else 0)
        state = 8 * B * H * N
        if kind != "scan_train":
            # u, delta, z -> y; per mode a product, an exponential, a product and two sums
            return dict(bytes=n * (3 + z) * e + bc + prm + state, flops=n * (7 * N + 20))
        # and dy -> du, ddelta, dz, dB, dC, the parameters' and the state's gradients
        return dict(bytes=n * (6 + 2 * z) * e + 2 * bc + 2 * prm + 2 * state,
                    flops=n * (27 * N + 60))
    if kind.startswith("conv"):
        K = case["K"]
        prm, state = 4 * H * (K + 1), 8 * B * H * (K - 1)
        if kind != "conv_train":
            return dict(bytes=n * 2 * e + prm + state, flops=n * (2 * K + 6))
        return dict(bytes=n * 4 * e + 2 * prm + 2 * state, flops=n * (8 * K + 18))
    post = 1 if case["post"] else 0
    return dict(bytes=n * ((3 + post) * e + 1) + 4 * B * L + 4 * H * (1 + 2 * post),
                flops=n * (8 + 14 * post))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _walk(a, b, start):
    """The recurrence step by step in 64 bits, rows [R, L]: blocks of about sqrt(L) steps side by
    side from zero, then their ends joined in order, then every step given its block's start.
    Returns the states after each step."""
    R, L = a.shape
    T = max(1, math.isqrt(L))
    nb = -(-L // T)
    pad = nb * T - L
    if pad:
        a = torch.cat([a, a.new_ones(R, pad)], 1)
        b = torch.cat([b, b.new_zeros(R, pad)], 1)
    a, b = a.reshape(R, nb, T), b.reshape(R, nb, T)
    h, p = torch.empty_like(b), torch.empty_like(a)
    hs, ps = torch.zeros_like(b[..., 0]), torch.ones_like(a[..., 0])
    for t in range(T):
        hs = hs * a[..., t] + b[..., t]
        ps = ps * a[..., t]
        h[..., t], p[..., t] = hs, ps
    c = start
    for k in range(nb):
        h[:, k].addcmul_(p[:, k], c[:, None])
        c = h[:, k, -1].clone()
    return h.reshape(R, nb * T)[:, :L]


def _exact_scan(case, s):
    """Mode by mode, so that a mode's states are all that is held at once."""
    kind = case["kind"]
    B, H, L, N, G = (case[k] for k in ("B", "H", "L", "N", "G"))
    flat = kind == "scan_step"
    rows = lambda t: t.double().reshape(B * H, L)
    u, delta = rows(s["u"]), rows(s["delta"])
    per_row = lambda t: t.double().repeat(B)[:, None]
    if s["dt_bias"] is not None:
        delta = delta + per_row(s["dt_bias"])
    lens = torch.full((B,), L, device="cuda") if s["lens"] is None else s["lens"].long()
    alive = torch.arange(L, device="cuda")[None] < lens.repeat_interleave(H)[:, None]
    zero = torch.zeros_like(u)
    step = torch.where(alive, torch.logaddexp(delta, zero), zero)
    u = torch.where(alive, u, zero)
    D = torch.zeros(B * H, 1, device="cuda").double() if s["D"] is None else per_row(s["D"])

    def reads(t, n):  # [B, G, N, L] -> [B H, L] of mode n
        t = t.double().reshape(B, G, N, L)[:, :, n]
        t = t[:, :, None].expand(B, G, H // G, L).reshape(B * H, L)
        return torch.where(alive, t, zero)

    gate = slope = None
    if s["z"] is not None:
        z = rows(s["z"])
        ex = torch.exp(-z)
        gate = torch.where(alive, z / (1.0 + ex), zero)
        slope = torch.where(alive, (1.0 + ex + z * ex) / (1.0 + ex) ** 2, zero)
    train = kind == "scan_train"
    total = D * u
    ends = torch.empty(B * H, N, device="cuda", dtype=torch.float64)
    if train:
        dy = torch.where(alive, rows(s["dy"]), zero)
        dp = dy if gate is None else dy * gate
        du, dstep = D * dp, torch.zeros_like(u)
        dB = torch.empty(B, G, N, L, device="cuda", dtype=torch.float64)
        dC, dlog = torch.empty_like(dB), torch.empty(H, N, device="cuda", dtype=torch.float64)
        dx0 = torch.empty_like(ends)
        group = lambda t: t.reshape(B, G, H // G, L).sum(2)
    for n in range(N):
        lr = per_row(s["log_re"][:, n])
        Bn, Cn = reads(s["Bm"], n), reads(s["Cm"], n)
        a = torch.exp(-lr * lr * step)
        x0 = s["x0"][..., n].double().reshape(-1)
        h = _walk(a, step * u * Bn, x0)
        total = total + Cn * h
        ends[:, n] = h[:, -1]
        if not train:
            continue
        c = Cn * dp
        c[:, -1] += s["dx"][..., n].double().reshape(-1)
        back = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        A = _walk(back.flip(1), c.flip(1), torch.zeros_like(x0)).flip(1)
        before = torch.cat([x0[:, None], h[:, :-1]], 1)
        da = A * before
        dC[:, :, n], dB[:, :, n] = group(dp * h), group(A * step * u)
        du = du + A * Bn * step
        dstep = dstep + A * Bn * u - da * a * lr * lr
        dlog[:, n] = (-2.0 * lr * da * a * step).reshape(B, H, L).sum((0, 2))
        dx0[:, n] = a[:, 0] * A[:, 0]
    back3 = lambda t: t.reshape(B, H) if flat else t.reshape(B, H, L)
    y = total if gate is None else total * gate
    ends = ends.reshape(B, H, N)
    if not train:
        return back3(y), ends
    ddelta = dstep * torch.where(alive, torch.sigmoid(delta), zero)
    sums = lambda t: t.reshape(B, H, L).sum((0, 2))
    return (back3(y), ends, back3(torch.where(alive, du, zero)), back3(ddelta), dB, dC,
            None if gate is None else back3(dy * total * slope), dlog,
            None if s["D"] is None else sums(dp * u),
            None if s["dt_bias"] is None else sums(ddelta), dx0.reshape(B, H, N))


def _exact_conv(case, s):
    """As a product with each step's window of inputs."""
    kind, K = case["kind"], case["K"]
    B, H, L = case["B"], case["H"], case["L"]
    u = s["u"].double().reshape(B, H, L)
    lens = torch.full((B,), L, device="cuda") if s["lens"] is None else s["lens"].long()
    alive = (torch.arange(L, device="cuda")[None] < lens[:, None])[:, None].double()
    u = torch.where(alive > 0, u, torch.zeros_like(u))
    past = torch.cat([s["x0"].double(), u], 2)
    windows = past.unfold(2, K, 1)  # [B, H, L, K]
    pre = (windows * s["w"].double()[None, :, None]).sum(-1) + s["bias"].double()[None, :, None]
    ex = torch.exp(-pre)
    y = alive * (pre / (1.0 + ex) if case["act"] else pre)
    end = torch.stack([past[b, :, int(n):int(n) + K - 1] for b, n in enumerate(lens.tolist())])
    if kind == "conv_step":
        return y[..., 0], end
    if kind == "conv":
        return y, end
    dp = alive * torch.where(alive > 0, s["dy"].double(), torch.zeros_like(u))
    if case["act"]:
        dp = dp * (1.0 + ex + pre * ex) / (1.0 + ex) ** 2
    # a past input k steps before step t met tap K - 1 - k
    later = torch.cat([dp.new_zeros(B, H, K - 1), dp, dp.new_zeros(B, H, K - 1)], 2)
    dpast = (later.unfold(2, K, 1) * s["w"].double().flip(1)[None, :, None]).sum(-1)
    for b, n in enumerate(lens.tolist()):
        dpast[b, :, int(n):int(n) + K - 1] += s["dx"][b].double()
    dw = (windows * dp[..., None]).sum((0, 2))
    return y, end, dpast[..., K - 1:] * alive, dw, dp.sum((0, 2)), dpast[..., :K - 1]


def _exact_norm8(case, s):
    """With the channels last."""
    dt, H = DTYPES[case["dtype"]], case["H"]
    flat = s["x"].dim() == 2
    last = (lambda t: t.double()) if flat else (lambda t: t.double().transpose(1, 2))

    def normed(t):
        c = t - t.sum(-1, keepdim=True) / H if case["layer"] else t
        return c * ((c * c).sum(-1, keepdim=True) / H + EPS).rsqrt()

    o, y = last(s["x"]), last(s["y"])
    if case["post"]:
        g = last(s["g"])
        y = normed(y) * s["w_post"].double() * s["scale"].double() * g / (1.0 + torch.exp(-g))
    o = o + y
    n = normed(o.to(dt).double()) * s["w_pre"].double()
    top = n.abs().max(-1, keepdim=True).values
    if case["form"] == "int8":
        v = torch.round(n * 127.0 / top) * top / 127.0
    else:
        # three bits behind the leading one, down to steps of 2^-9
        m = n * 448.0 / top
        exponent = torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6)))
        unit = torch.exp2(exponent - 3.0)
        v = torch.round(m / unit) * unit * top / 448.0
    return (o if flat else o.transpose(1, 2)), v


def exact(case, seed):
    s = _make(case, seed)
    kind = case["kind"]
    if kind.startswith("scan"):
        return _exact_scan(case, s)
    if kind.startswith("conv"):
        return _exact_conv(case, s)
    return _exact_norm8(case, s)
