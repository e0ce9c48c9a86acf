"""A selective block put together from the library's calls, as a model would run it: the residual
sum and norm in 8 bits, the joint projection, the short convolution, the projections of the step
sizes, read-in and read-out, the scan with its gate.  Training against float64 autograd on the
CPU, and a prompt followed by tokens against the prompt in one call.

In float32 every stage is off by some 2^-23 times the absolute values of its terms, a few tens of
them at worst (selective_cases.py) and a few on average; the 2-norms of results after seven stages
are asked to agree to 2^-23 * 64 = 8e-6 forward and twice that backward.
"""
import numpy as np
import pytest

from long_convolution_sequence_amd import binding as bd

from seq_cases import np64, say, torch_

pytestmark = pytest.mark.gpu

B, H, N, G, K, R = 2, 48, 6, 2, 4, 5
EPS = 1e-5


def parameters(seed):
    torch = torch_()
    g = np.random.default_rng(seed)
    up = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    return dict(w=up(1 + 0.2 * g.normal(size=H)), w_in=up(g.normal(size=(2 * H, H)) / H ** 0.5),
                taps=up(g.normal(size=(H, K)) / K ** 0.5), bias=up(0.1 * g.normal(size=H)),
                w_x=up(g.normal(size=(R + 2 * G * N, H)) / H ** 0.5),
                w_dt=up(g.normal(size=(H, R)) / R ** 0.5), dt_bias=up(g.uniform(-4, -1, H)),
                log_re=up(np.sqrt(np.arange(1, N + 1))[None] * g.uniform(0.8, 1.2, (H, N))),
                D=up(g.normal(size=H)))


def modes(p, lo):
    """G groups of N modes, as a slice of the projection's channels."""
    return p[:, lo:lo + G * N].unflatten(1, (G, N))


def forward(prm, x, y, states=None, keep=False):
    """The block over [B, H, L] from and to its states (conv, scan), updated in place."""
    torch = torch_()
    conv, scan = states if states else (None, None)
    o, q, qs, st = bd.resnorm8_forward_stats(x, y, None, None, None, prm["w"], eps=EPS)
    n = q.float() * qs[..., None]                      # [B, L, H], as the product reads it
    p = prm["w_in"] @ n.transpose(1, 2)
    c = bd.shortconv_forward(p[:, :H], prm["taps"], prm["bias"], x=conv)
    e = prm["w_x"] @ c
    delta = prm["w_dt"] @ e[:, :R]
    a = (c, delta, modes(e, R), modes(e, R + G * N), prm["log_re"])
    kw = dict(D=prm["D"], dt_bias=prm["dt_bias"], z=p[:, H:])
    if not keep:
        return o, bd.selective_forward(*a, x=scan, **kw)
    out, ckpt = bd.selective_forward_ckpt(*a, x=scan, **kw)
    return o, out, (n, st, p, c, e, a, kw, ckpt)


def token(prm, x, y, states):
    conv, scan = states
    o, q, qs = bd.resnorm8_forward(x, y, None, None, None, prm["w"], eps=EPS)
    p = (q.float() * qs[:, None]) @ prm["w_in"].T
    c = bd.shortconv_step(p[:, :H], prm["taps"], prm["bias"], conv)
    e = c @ prm["w_x"].T
    delta = e[:, :R] @ prm["w_dt"].T
    return o, bd.selective_step(c, delta, modes(e, R), modes(e, R + G * N), prm["log_re"], scan,
                                D=prm["D"], dt_bias=prm["dt_bias"], z=p[:, H:])


def relative(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("L", [33, 400])
def test_training(L):
    torch = torch_()
    prm = parameters(1)
    g = np.random.default_rng(L)
    up = lambda *s: torch.from_numpy(g.normal(size=s).astype(np.float32)).cuda()
    x, y, do, dout = (up(B, H, L) for _ in range(4))
    o, out, (n, st, p, c, e, a, kw, ckpt) = forward(prm, x, y, keep=True)
    # back, each gradient into its place in the projections'
    dp, de = torch.empty_like(p), torch.empty_like(e)
    s = bd.selective_backward(dout, ckpt, *a, dz=dp[:, H:], dB=modes(de, R), dC=modes(de, R + G * N),
                              **kw)
    de[:, :R] = prm["w_dt"].T @ s["ddelta"]
    dc = s["du"] + prm["w_x"].T @ de
    k = bd.shortconv_backward(dc, p[:, :H], prm["taps"], prm["bias"], du=dp[:, :H])
    dn = prm["w_in"].T @ dp
    r = bd.resnorm_backward(o, None, None, st, None, None, prm["w"], do, dn)
    got = dict(x=r["dx"], w=r["dw_pre"], w_in=torch.matmul(dp, n).sum(0), taps=k["dw"],
               bias=k["dbias"], w_x=torch.matmul(de, c.transpose(1, 2).contiguous()).sum(0),
               w_dt=torch.matmul(s["ddelta"], e[:, :R].transpose(1, 2).contiguous()).sum(0),
               dt_bias=s["ddt_bias"], log_re=s["dlog_re"], D=s["dD"])

    # the same in float64 on the CPU, by autograd, the rounding to 8 bits taken for the identity
    t = {kk: v.double().cpu().requires_grad_() for kk, v in prm.items()}
    xd = x.double().cpu().requires_grad_()
    od = xd + y.double().cpu()
    nd = od / torch.sqrt((od ** 2).mean(1, keepdim=True) + EPS) * t["w"][None, :, None]
    nd = nd + (n.transpose(1, 2).double().cpu() - nd).detach()
    pd = t["w_in"] @ nd
    ext = torch.nn.functional.pad(pd[:, :H], (K - 1, 0))
    pre = t["bias"][None, :, None] + sum(t["taps"][None, :, j, None] * ext[..., j:j + L]
                                         for j in range(K))
    cd = pre * torch.sigmoid(pre)
    ed = t["w_x"] @ cd
    dt = torch.nn.functional.softplus(t["w_dt"] @ ed[:, :R] + t["dt_bias"][None, :, None])
    spread = lambda v: v.repeat_interleave(H // G, 1)
    Bd, Cd = spread(modes(ed, R)), spread(modes(ed, R + G * N))
    h = torch.zeros(B, H, N, dtype=torch.float64)
    ys = []
    for i in range(L):
        step = dt[..., i, None]
        h = torch.exp(-t["log_re"][None] ** 2 * step) * h + step * Bd[..., i] * cd[..., i, None]
        ys.append((Cd[..., i] * h).sum(-1))
    yd = torch.stack(ys, -1) + t["D"][None, :, None] * cd
    z = pd[:, H:]
    outd = yd * z * torch.sigmoid(z)
    ((od * do.double().cpu()).sum() + (outd * dout.double().cpu()).sum()).backward()
    rel = relative(np64(out), outd.detach().numpy())
    say("  out %.2e" % rel)
    assert rel < 8e-6
    for name, v in got.items():
        ref = (xd if name == "x" else t[name]).grad.numpy()
        rel = relative(np64(v), ref)
        say("  d%s %.2e" % (name, rel))
        assert rel < 1.6e-5, name


def test_prompt_and_tokens():
    torch = torch_()
    prm = parameters(2)
    g = np.random.default_rng(3)
    L, cut = 200, 193
    x, y = (torch.from_numpy(g.normal(size=(B, H, L)).astype(np.float32)).cuda() for _ in range(2))
    fresh = lambda: (torch.zeros(B, H, K - 1, device="cuda"), torch.zeros(B, H, N, device="cuda"))
    whole_states, states = fresh(), fresh()
    o, out = forward(prm, x, y, whole_states)
    part = lambda t: t[..., :cut].contiguous()
    o1, out1 = forward(prm, part(x), part(y), states)
    os, outs = [o1], [out1]
    for i in range(cut, L):
        a, b = token(prm, x[..., i].contiguous(), y[..., i].contiguous(), states)
        os.append(a[..., None])
        outs.append(b[..., None])
    assert torch.equal(torch.cat(os, -1), o)
    rel = relative(np64(torch.cat(outs, -1)), np64(out))
    say("  out %.2e" % rel)
    # the projections of a token and of a prompt add up in another order; a value next to a border
    # of its 8 bits may fall on its other side: one step of 127 in one of 48 channels
    assert rel < 1e-3
    for a, b in zip(states, whole_states):
        assert relative(np64(a), np64(b)) < 1e-3
