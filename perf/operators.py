"""The operators around the gated linear recurrence, case by case, for timing and comparison.

Three operators over activations [B, H, L] (time fastest), as the layer forward takes them:

* the gated recurrence: h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) u_t,
  a_t = exp(-log_re^2 sigmoid(r_t)), in streaming (a state in and out), one-token and training form;
* activation checkpoints in 8 bits: groups of 64 steps as int8 times a power of two, by themselves
  and as what the gated recurrence's backward pass reads;
* the residual norm: o = x + scale norm(y) w_post silu(g), n = norm(o) w_pre, norms over H.

`own` false: plain torch operations in 32 bits.  `own` true: the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
GROUP = 64    # steps that share a power of two in an 8-bit checkpoint
CHUNK = 512   # steps between the states a checkpoint keeps
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token for a small batch: latency
        dict(name="step_small", kind="step", B=8, H=1024, L=1, dtype="bf16"),
        # one generated token for a server's batch of streams
        dict(name="step_server", kind="step", B=256, H=4096, L=1, dtype="f16"),
        # a million steps of few channels in float32, continued from a state
        dict(name="prefill_long", kind="prefill", B=1, H=4, L=1 << 20, dtype="f32", ragged=False),
        # prompts of different lengths in one padded batch, gates out of one joint projection
        dict(name="prefill_batch", kind="prefill", B=8, H=2048, L=2048, dtype="bf16", ragged=True),
        # training on the long-sequence workload's shape in float32
        dict(name="train_f32", kind="train", B=4, H=128, L=16384, dtype="f32", ragged=False,
             bits8=False),
        # odd sizes and a padded batch, small
        dict(name="train_odd", kind="train", B=3, H=131, L=1001, dtype="f16", ragged=True,
             bits8=False),
        # the largest: a wide layer's training step, kept activations in their own type
        dict(name="train_wide", kind="train", B=4, H=2048, L=8192, dtype="bf16", ragged=False,
             bits8=False),
        # the same layer with the kept activations in 8 bits
        dict(name="train_wide_8bit", kind="train", B=4, H=2048, L=8192, dtype="bf16",
             ragged=False, bits8=True),
        # any activation put away in 8 bits and taken out again
        dict(name="ckpt8", kind="ckpt8", B=4, H=256, L=16384, dtype="bf16"),
        # around one generated token of a server's batch
        dict(name="norm_token", kind="norm", B=64, H=4096, L=1, dtype="bf16", layer=False),
        # a wide layer's block in inference
        dict(name="norm_wide", kind="norm", B=4, H=1024, L=8192, dtype="bf16", layer=False),
        # training with layer norms on the multi-input workload's shape, odd length
        dict(name="norm_train", kind="normtrain", B=4, H=256, L=16383, dtype="f32", layer=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["step", "prefill", "train", "train", "ckpt8", "norm", "norm", "normtrain"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if kind == "step" or (kind == "norm" and rng.random() < 0.4):
        case = dict(kind=kind, B=_log_int(rng, 1, 256), H=_log_int(rng, 16, 4096), L=1, dtype=dtype)
    else:
        most = 1 << 25  # elements: at most half of the largest listed case
        L = _log_int(rng, 64, 1 << 20 if kind == "prefill" else 32768)
        H = _log_int(rng, 1 if kind == "prefill" else 16, min(4096, max(16, most // L)))
        B = _log_int(rng, 1, max(1, min(16, most // (L * H))))
        case = dict(kind=kind, B=B, H=H, L=L, dtype=dtype)
    if kind in ("prefill", "train"):
        case["ragged"] = rng.random() < 0.5
    if kind == "train":
        case["bits8"] = rng.random() < 0.5
    if kind in ("norm", "normtrain"):
        case["layer"] = rng.random() < 0.5
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

    def uniform(n, lo, hi):
        return torch.rand(n, generator=gen, device="cuda") * (hi - lo) + lo

    s = {}
    if kind in ("step", "prefill", "train"):
        # decays over the range of the layer's own initialisation, gate logits spread around 0
        s["log_re"] = torch.exp(uniform(H, math.log(0.015), math.log(1.0)))
        if kind == "step":
            s["u"], s["r"], s["i"] = (normal(B, H, sd=sd) for sd in (1.0, 1.5, 1.5))
        else:
            # one joint projection's output: the three inputs are slices of it
            p = torch.empty(B, 3 * H, L, dtype=dt, device="cuda")
            for k, sd in enumerate((1.0, 1.5, 1.5)):
                p[:, k * H:(k + 1) * H] = normal(B, H, L, sd=sd)
            s["u"], s["r"], s["i"] = p[:, :H], p[:, H:2 * H], p[:, 2 * H:]
        s["x0"] = normal(B, H, dtype=torch.float32)
        if case.get("ragged"):
            # the longest fills the batch, the others end anywhere
            lens = (uniform(B, 0.1, 1.0) * L).to(torch.int32)
            lens[0] = L
            s["lens"] = lens
        else:
            s["lens"] = None
        if kind == "train":
            s["dy"] = normal(B, H, L)
            s["dx"] = normal(B, H, dtype=torch.float32)
    elif kind == "ckpt8":
        # activations of channels of different scale, with a few outliers
        x = torch.randn(B, H, L, generator=gen, device="cuda")
        x = x * torch.exp(uniform(H, -3.0, 3.0))[None, :, None]
        far = torch.rand(B, H, L, generator=gen, device="cuda") < 1e-3
        s["x"] = torch.where(far, x * 12.0, x).to(dt)
    else:
        shape = (B, H) if L == 1 else (B, H, L)
        s["x"], s["y"] = normal(*shape, sd=2.0), normal(*shape, sd=0.7, mean=0.1)
        s["g"] = normal(*shape, sd=1.5)
        s["w_post"] = normal(H, sd=0.2, mean=1.0, dtype=torch.float32)
        s["w_pre"] = normal(H, sd=0.2, mean=1.0, dtype=torch.float32)
        s["scale"] = normal(H, sd=0.1, mean=0.3, dtype=torch.float32)
        if kind == "normtrain":
            s["do"], s["dn"] = normal(*shape), normal(*shape)
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
    if kind == "step":
        y = bd.gated_step(s["u"], s["r"], s["i"], s["log_re"], s["x0"], x_out=s["x"])
        return y, s["x"]
    if kind == "prefill":
        y = bd.gated_forward(s["u"], s["r"], s["i"], s["log_re"], x=s["x0"], x_out=s["x"],
                             lens=s["lens"])
        return y, s["x"]
    if kind == "train":
        ck = bd.CKPT_INT8 if case["bits8"] else bd.CKPT_STATE
        y, ckpt = bd.gated_forward_ckpt(s["u"], s["r"], s["i"], s["log_re"], ck, x=s["x0"],
                                        x_out=s["x"], lens=s["lens"])
        kept = {} if case["bits8"] else dict(u=s["u"], r=s["r"], i=s["i"])
        g = bd.gated_backward(s["dy"], ckpt, ck, s["log_re"], dx=s["dx"], lens=s["lens"], **kept)
        return y, s["x"], g["du"], g["dr"], g["di"], g["dlog_re"], g["dx0"]
    if kind == "ckpt8":
        blob = bd.ckpt8_pack(s["x"])
        return bd.ckpt8_unpack(blob, s["x"].shape, s["x"].dtype)
    norm = bd.NORM_LAYER if case["layer"] else bd.NORM_RMS
    prm = (s["w_post"], s["scale"], s["w_pre"])
    if kind == "norm":
        return bd.resnorm_forward(s["x"], s["y"], s["g"], *prm, norm=norm, eps=EPS)
    o, n, stats = bd.resnorm_forward_stats(s["x"], s["y"], s["g"], *prm, norm=norm, eps=EPS)
    g = bd.resnorm_backward(o, s["y"], s["g"], stats, *prm, s["do"], s["dn"], norm=norm)
    return o, n, g["dx"], g["dy"], g["dg"], g["dw_post"], g["dscale"], g["dw_pre"]


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _gates(u, r, i, log_re):
    """Decay a, its complement beta, sigmoids and the driven input.  In 32 bits but for a: the
    slowest channels remember some ten thousand steps, and as many roundings next to 1 add up."""
    q, s = torch.sigmoid(r), torch.sigmoid(i)
    z = (log_re * log_re)[None, :, None] * q
    a = torch.exp(-z if r.shape[-1] == 1 else -z.double())
    beta = torch.sqrt(-torch.expm1(-2.0 * z))
    return a, beta, q, s, beta * s * u


def _scan(a, b, x0):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = x0, by doubling, in the type of a; 32 bits out."""
    b = b.to(a.dtype)
    b = torch.cat([b[..., :1] + a[..., :1] * x0[..., None], b[..., 1:]], -1)
    o = 1
    while o < b.shape[-1]:
        b = torch.cat([b[..., :o], b[..., o:] + a[..., o:] * b[..., :-o]], -1)
        a = torch.cat([a[..., :o], a[..., o:] * a[..., :-o]], -1)
        o *= 2
    return b.float()


def _valid(lens, B, L, device):
    if lens is None:
        return None
    return (torch.arange(L, device=device)[None, :] < lens[:, None])[:, None, :]


def _quantised(x, valid=None):
    """The values an 8-bit checkpoint stands for (32 bits: every step is exact)."""
    shape = x.shape
    x = x.float()
    if valid is not None:
        x = torch.where(valid, x, torch.zeros_like(x))
    pad = -shape[-1] % GROUP
    if pad:
        x = torch.cat([x, x.new_zeros(shape[:-1] + (pad,))], -1)
    v = x.reshape(shape[:-1] + (-1, GROUP))
    m, k = torch.frexp(v.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 127.0 / 128.0, k - 7, k - 6).clamp(min=-126)
    power = lambda n: ((n.int() + 127) << 23).view(torch.float32)  # 2^n, -127 < n < 128
    v = (torch.round(v * power(-e)) * power(e)).reshape(shape[:-1] + (-1,))
    return v[..., :shape[-1]]


def _run_gated_plain(s):
    case = s["case"]
    kind = case["kind"]
    dt = DTYPES[case["dtype"]]
    u, r, i = s["u"].float(), s["r"].float(), s["i"].float()
    if kind == "step":
        u, r, i = u[..., None], r[..., None], i[..., None]
    B, H, L = u.shape
    log_re = s["log_re"]
    valid = _valid(s["lens"], B, L, u.device)
    a, beta, q, sg, b = _gates(u, r, i, log_re)
    if valid is not None:  # past a row's end the state stays
        a = torch.where(valid, a, torch.ones_like(a))
        b = torch.where(valid, b, torch.zeros_like(b))
    h = _scan(a, b, s["x0"])
    y = h if valid is None else torch.where(valid, h, torch.zeros_like(h))
    y = y.to(dt)
    if kind == "step":
        return y[..., 0], h[..., -1]
    if kind == "prefill":
        return y, h[..., -1].contiguous()
    x0, xT = s["x0"], h[..., -1].contiguous()
    if case["bits8"]:
        # gradients at the decoded activations, the state restarted at every chunk
        u, r, i = _quantised(s["u"], valid), _quantised(s["r"], valid), _quantised(s["i"], valid)
        a, beta, q, sg, b = _gates(u, r, i, log_re)
        if valid is not None:
            a = torch.where(valid, a, torch.ones_like(a))
            b = torch.where(valid, b, torch.zeros_like(b))
        starts = torch.cat([x0[..., None], h[..., CHUNK - 1:L - 1:CHUNK]], -1)
        parts = [_scan(a[..., c * CHUNK:(c + 1) * CHUNK], b[..., c * CHUNK:(c + 1) * CHUNK],
                       starts[..., c]) for c in range(starts.shape[-1])]
        prev = [torch.cat([starts[..., c:c + 1], p[..., :-1]], -1) for c, p in enumerate(parts)]
        h_prev = torch.cat(prev, -1)
    else:
        h_prev = torch.cat([x0[..., None], h[..., :-1]], -1)
    dy = s["dy"].float()
    if valid is not None:
        dy = torch.where(valid, dy, torch.zeros_like(dy))
    nxt = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    last = torch.zeros_like(dy)
    last[..., -1] = s["dx"]
    G = _scan(nxt.flip(-1), (dy + last).flip(-1), torch.zeros_like(x0)).flip(-1)
    a = a.float()
    live = torch.ones_like(a) if valid is None else valid.float()
    du = G * beta * sg * live
    di = G * beta * u * sg * (1.0 - sg) * live
    dz = (-a * G * h_prev + torch.where(beta > 0, G * sg * u * a * a / beta,
                                        torch.zeros_like(G))) * live
    dr = dz * (log_re * log_re)[None, :, None] * q * (1.0 - q)
    dlog = 2.0 * log_re.double() * (dz * q).double().sum((0, 2))
    dx0 = a[..., 0] * G[..., 0]
    return y, xT, du.to(dt), dr.to(dt), di.to(dt), dlog.float(), dx0


def _norm_plain(y, layer):
    """Normalised values and the factor, over the channels."""
    m = y.mean(1, keepdim=True) if layer else torch.zeros_like(y[:, :1])
    d = y - m
    rs = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * rs, rs


def _norm_back(dv, vh, rs, layer):
    out = dv - vh * (dv * vh).mean(1, keepdim=True)
    if layer:
        out = out - dv.mean(1, keepdim=True)
    return out * rs


def _run_norm_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x, y, g = (s[k].float() for k in ("x", "y", "g"))
    flat = x.dim() == 2
    if flat:
        x, y, g = x[..., None], y[..., None], g[..., None]
    wo, sc, wr = (s[k][None, :, None] for k in ("w_post", "scale", "w_pre"))
    yh, ry = _norm_plain(y, case["layer"])
    sg = torch.sigmoid(g)
    o = (x + sc * (yh * wo) * (g * sg)).to(dt)
    of = o.float()  # what the next block sees is the stored stream
    oh, ro = _norm_plain(of, case["layer"])
    n = (oh * wr).to(dt)
    if case["kind"] == "norm":
        return (o[..., 0], n[..., 0]) if flat else (o, n)
    do, dn = s["do"].float(), s["dn"].float()
    if flat:
        do, dn = do[..., None], dn[..., None]
    t = do + _norm_back(dn * wr, oh, ro, case["layer"])
    dv = t * sc * (g * sg)
    dy = _norm_back(dv * wo, yh, ry, case["layer"])
    dg = t * sc * yh * wo * sg * (1.0 + g * (1.0 - sg))
    total = lambda v: v.double().sum((0, 2)).float()
    out = [o, n, t.to(dt), dy.to(dt), dg.to(dt)]
    if flat:
        out = [v[..., 0] for v in out]
    return tuple(out) + (total(dv * yh), total(t * yh * wo * g * sg), total(dn * oh))


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind in ("step", "prefill", "train"):
        return _run_gated_plain(state)
    if kind == "ckpt8":
        return _quantised(state["x"]).to(state["x"].dtype)
    return _run_norm_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B, H, L, kind = case["B"], case["H"], case["L"], case["kind"]
    n, e = B * H * L, BYTES[case["dtype"]]
    row = 4 * H
    if kind == "step":
        return dict(bytes=n * (4 * e + 8) + row, flops=30 * n)
    if kind == "prefill":
        return dict(bytes=n * 4 * e + 8 * B * H + row, flops=30 * n)
    eight = 1 + 1 / GROUP
    if kind == "train":
        # forward: u, r, i -> y; backward: u, r, i (or their 8 bits), dy -> du, dr, di
        kept = 2 * 3 * eight if case["bits8"] else 3 * e
        return dict(bytes=int(n * (4 * e + kept + 4 * e + 8 / CHUNK)) + 20 * B * H + 3 * row,
                    flops=110 * n)
    if kind == "ckpt8":
        return dict(bytes=int(n * (2 * e + 2 * eight)), flops=6 * n)
    if kind == "norm":
        return dict(bytes=n * 5 * e + 3 * row, flops=20 * n)
    return dict(bytes=n * 13 * e + 9 * row, flops=70 * n)


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
    h = torch.empty_like(b)
    p = torch.empty_like(a)
    hs, ps = torch.zeros_like(b[..., 0]), torch.ones_like(a[..., 0])
    for t in range(T):
        hs = hs * a[..., t] + b[..., t]
        ps = ps * a[..., t]
        h[..., t], p[..., t] = hs, ps
    carry = torch.empty_like(hs)
    c = start
    for k in range(nb):
        carry[:, k] = c
        c = ps[:, k] * c + hs[:, k]
    return (h + p * carry[..., None]).reshape(R, nb * T)[:, :L]


def _decode64(x):
    """Groups of 64 steps as whole multiples, at most 127, of the smallest power of two that
    reaches their largest value."""
    L = x.shape[-1]
    out = torch.zeros_like(x)
    full = L // GROUP * GROUP
    for lo, hi, width in ((0, full, GROUP), (full, L, L - full)):
        if hi == lo:
            continue
        v = x[..., lo:hi].reshape(x.shape[:-1] + (-1, width))
        top = v.abs().max(-1, keepdim=True).values
        n = torch.ceil(torch.log2(top.clamp(min=1e-300) / 127.0)).clamp(min=-126.0)
        scale = ((n.long() + 1023) << 52).view(torch.float64)
        # log2's own rounding may miss by one power; put both sides right
        scale = torch.where(top > 127.0 * scale, scale * 2.0, scale)
        scale = torch.where((top <= 127.0 * scale * 0.5) & (scale > 2.0 ** -126), scale * 0.5, scale)
        out[..., lo:hi] = (torch.round(v / scale) * scale).reshape(x.shape[:-1] + (-1,))
    return out


def _exact_gated(case, s):
    kind = case["kind"]
    B, H, L = case["B"], case["H"], case["L"]
    lr = s["log_re"].double().repeat(B)[:, None]
    rows = lambda t: t.double().reshape(B * H, L)
    x0 = s["x0"].double().reshape(B * H)
    lens = torch.full((B,), L, device="cuda") if s["lens"] is None else s["lens"].long()
    alive = torch.arange(L, device="cuda")[None] < lens.repeat_interleave(H)[:, None]

    def parts(u, r, i):
        z = lr.square() / (1.0 + torch.exp(-r))
        w = torch.where(alive, -torch.expm1(-2.0 * z), torch.zeros_like(z))  # 1 - a^2
        return torch.where(alive, torch.exp(-z), torch.ones_like(z)), w.sqrt()

    u, r, i = rows(s["u"]), rows(s["r"]), rows(s["i"])
    a, beta = parts(u, r, i)
    u0 = torch.where(alive, u, torch.zeros_like(u))
    h = _walk(a, beta * u0 / (1.0 + torch.exp(-i)), x0)
    y = torch.where(alive, h, torch.zeros_like(h))
    end = h[:, -1].reshape(B, H)
    if kind == "step":
        return y.reshape(B, H), end
    if kind == "prefill":
        return y.reshape(B, H, L), end
    before = torch.cat([x0[:, None], h[:, :-1]], 1)
    if case["bits8"]:
        zero = torch.zeros_like(u)
        u, r, i = (_decode64(torch.where(alive, t, zero)) for t in (u, r, i))
        a, beta = parts(u, r, i)
        bb = beta * u / (1.0 + torch.exp(-i))
        again = torch.empty_like(h)
        for lo in range(0, L, CHUNK):
            st = before[:, lo].clone()
            hh = _walk(a[:, lo:lo + CHUNK], bb[:, lo:lo + CHUNK], st)
            again[:, lo] = st
            again[:, lo + 1:lo + CHUNK] = hh[:, :-1]
        before = again
    del h
    # the adjoint runs the other way: G_t = dy_t + a_{t+1} G_{t+1}
    dy = torch.where(alive, rows(s["dy"]), torch.zeros_like(u))
    dy[:, -1] += s["dx"].double().reshape(-1)
    back = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    G = _walk(back.flip(1), dy.flip(1), torch.zeros_like(x0)).flip(1)
    q, sg = torch.sigmoid(r), torch.sigmoid(i)
    Ga = torch.where(alive, G, torch.zeros_like(G))
    u = torch.where(alive, u, torch.zeros_like(u))
    db = Ga * sg * u
    ratio = torch.where(beta > 0, a * a / beta, torch.zeros_like(beta))
    dz = db * ratio - Ga * a * before
    back3 = lambda t: t.reshape(B, H, L)
    dlog = 2.0 * s["log_re"].double() * (dz * q).reshape(B, H, L).sum((0, 2))
    return (back3(y), end, back3(Ga * beta * sg), back3(dz * lr.square() * q * (1 - q)),
            back3(Ga * beta * u * sg * (1 - sg)), dlog, (a[:, 0] * G[:, 0]).reshape(B, H))


def _exact_norm(case, s):
    """With the channels last, and the norms' gradients as products with their Jacobian."""
    layer, dt, H = case["layer"], DTYPES[case["dtype"]], case["H"]
    flat = s["x"].dim() == 2
    last = (lambda t: t.double()) if flat else (lambda t: t.double().transpose(1, 2).contiguous())
    first = (lambda t: t) if flat else (lambda t: t.transpose(1, 2).contiguous())
    x, y, g = last(s["x"]), last(s["y"]), last(s["g"])
    wo, sc, wr = s["w_post"].double(), s["scale"].double(), s["w_pre"].double()

    def centred(t):
        return t - t.sum(-1, keepdim=True) / H if layer else t

    def factor(c):
        return ((c * c).sum(-1, keepdim=True) / H + EPS).rsqrt()

    yc = centred(y)
    fy = factor(yc)
    silu = g / (1.0 + torch.exp(-g))
    v = yc * fy * wo
    o = x + sc * v * silu
    # the second norm is of the stream as it is stored
    oc = centred(o.to(dt).double())
    fo = factor(oc)
    n = oc * fo * wr
    if case["kind"] == "norm":
        return first(o), first(n)

    def through(grad, c, f):
        # d(c f)/dt applied to grad, f = (mean c^2 + eps)^(-1/2)
        d = grad * f - c * f ** 3 * ((grad * c).sum(-1, keepdim=True) / H)
        return centred(d)

    do, dn = last(s["do"]), last(s["dn"])
    t = do + through(dn * wr, oc, fo)
    dvs = t * sc
    dy = through(dvs * silu * wo, yc, fy)
    e = torch.exp(-g)
    dg = dvs * v * (1.0 + e + g * e) / (1.0 + e) ** 2
    axes = tuple(range(t.dim() - 1))
    return (first(o), first(n), first(t), first(dy), first(dg), (dvs * silu * yc * fy).sum(axes),
            (t * v * silu).sum(axes), (dn * oc * fo).sum(axes))


def exact(case, seed):
    s = _make(case, seed)
    kind = case["kind"]
    if kind in ("step", "prefill", "train"):
        return _exact_gated(case, s)
    if kind == "ckpt8":
        return _decode64(s["x"].double())
    return _exact_norm(case, s)
