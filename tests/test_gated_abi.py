"""What the gated recurrence, the 8-bit checkpoints and the residual norm refuse
(C ABI, host side; no kernel is launched), and the sizes they report."""
import ctypes

import pytest

from long_convolution_sequence_amd import binding as bd

FAKE = 1 << 20  # an aligned, never-dereferenced device address
INV, UNS, WS = bd.DSSM_ERR_INVALID_ARG, bd.DSSM_ERR_UNSUPPORTED, bd.DSSM_ERR_WORKSPACE


def at(k):
    return FAKE * (k + 1)


def gshape(B=2, H=3, L=40, dtype=bd.BF16):
    return bd.GatedShape(B, H, L, dtype)


def size(fn, *args):
    out = ctypes.c_size_t(123)
    rc = fn(*(list(args) + [ctypes.byref(out)]))
    return rc, out.value


def inputs(**bad):
    v = dict(u=at(0), r=at(1), i=at(2), stride_b=120, log_re=at(3), lens=None)
    v.update(bad)
    return bd.GatedInputs(*[v[k] for k in ("u", "r", "i", "stride_b", "log_re", "lens")])


BAD_SHAPES = [(dict(B=-1), INV), (dict(H=-1), INV), (dict(L=-1), INV), (dict(dtype=3), INV),
              (dict(dtype=-1), INV), (dict(H=65536), UNS), (dict(L=(1 << 24) + 1), UNS),
              (dict(B=1 << 16, H=1 << 10), UNS), (dict(B=1 << 10, H=1 << 10, L=1 << 21), UNS),
              (dict(B=(1 << 31) - 1, H=65535, L=1 << 24), UNS)]


@pytest.mark.parametrize("bad,rc", BAD_SHAPES)
def test_gated_sizes_refuse(bad, rc):
    L = bd.lib()
    s = ctypes.byref(gshape(**bad))
    assert size(L.dssm_gated_workspace_size, s)[0] == rc and L.dssm_last_error()
    assert size(L.dssm_gated_ckpt_size, s, bd.CKPT_STATE)[0] == rc


def test_gated_sizes():
    L = bd.lib()
    s = ctypes.byref(gshape())
    assert L.dssm_gated_workspace_size(s, None) == INV
    assert L.dssm_gated_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INV
    assert size(L.dssm_gated_ckpt_size, s, 3)[0] == INV
    assert size(L.dssm_gated_ckpt_size, s, -1)[0] == INV
    assert size(L.dssm_gated_ckpt_size, s, bd.CKPT_NONE) == (0, 0)
    assert size(L.dssm_gated_ckpt_size, s, bd.CKPT_STATE) == (0, 256)
    # 6 states; three blobs of 6 rows of 48 bytes (-> 512) and 6 exponents (-> 256)
    assert size(L.dssm_gated_ckpt_size, s, bd.CKPT_INT8) == (0, 256 + 3 * 768)
    for empty in (gshape(B=0), gshape(H=0), gshape(L=0)):
        assert size(L.dssm_gated_ckpt_size, ctypes.byref(empty), bd.CKPT_INT8) == (0, 0)
    # the longest row: states every 512 steps
    s = ctypes.byref(gshape(B=1, H=1, L=1 << 24))
    assert size(L.dssm_gated_ckpt_size, s, bd.CKPT_STATE) == (0, 4 << 15)
    assert L.dssm_ckpt8_size(6, 40, None) == INV
    assert size(L.dssm_ckpt8_size, 6, 40) == (0, 768)
    assert size(L.dssm_ckpt8_size, 0, 40) == (0, 0) and size(L.dssm_ckpt8_size, 6, 0) == (0, 0)
    assert size(L.dssm_ckpt8_size, -1, 4)[0] == INV and size(L.dssm_ckpt8_size, 1, -4)[0] == INV
    assert size(L.dssm_ckpt8_size, 1, (1 << 24) + 1)[0] == UNS
    assert size(L.dssm_ckpt8_size, 1 << 62, 1 << 24)[0] == UNS


def test_gated_forward_refuses():
    L = bd.lib()

    def call(s=None, inp=None, x0=at(5), xe=at(6), y=at(7), kind=bd.CKPT_STATE, ckpt=at(8),
             ws=at(9), n=1 << 30):
        s = gshape() if s is None else s
        inp = inputs() if inp is None else inp
        return L.dssm_gated_forward(ctypes.byref(inp), ctypes.byref(s), x0, xe, y, kind, ckpt, ws,
                                    n, None)

    for bad, rc in BAD_SHAPES:
        assert call(s=gshape(**bad)) == rc, bad
    assert L.dssm_gated_forward(None, ctypes.byref(gshape()), None, None, at(7), 0, None, at(9),
                                1 << 30, None) == INV
    for k in ("u", "r", "i", "log_re"):
        assert call(inp=inputs(**{k: None})) == INV and k.encode() in L.dssm_last_error()
        assert call(inp=inputs(**{k: at(0) + 1})) == INV
    assert call(inp=inputs(lens=at(4) + 2)) == INV
    assert call(inp=inputs(stride_b=119)) == INV and b"stride_b" in L.dssm_last_error()
    assert call(inp=inputs(stride_b=(1 << 40) + 1)) == UNS
    assert call(y=None) == INV
    assert call(y=at(0)) == INV and call(y=at(2)) == INV and call(y=at(5)) == INV
    assert call(y=at(6)) == INV  # the end state's own memory
    assert call(xe=at(0)) == INV and call(xe=at(3)) == INV
    assert call(x0=at(5) + 2) == INV and call(xe=at(6) + 2) == INV
    assert call(kind=3) == INV and call(kind=-1) == INV
    assert call(ckpt=None) == INV and call(ckpt=at(8) + 16) == INV
    assert call(n=16) == WS and call(ws=None) == INV and call(ws=at(9) + 16) == INV
    # nothing to do: B or H is 0
    assert call(s=gshape(B=0), inp=inputs(u=None)) == 0 and call(s=gshape(H=0), y=None) == 0
    assert L.dssm_last_error() == b""


def test_gated_step_refuses():
    L = bd.lib()

    def call(s=None, inp=None, x0=at(5), xe=at(5), y=at(7)):
        s = gshape(L=1) if s is None else s
        inp = inputs() if inp is None else inp
        return L.dssm_gated_step(ctypes.byref(inp), ctypes.byref(s), x0, xe, y, None)

    assert call(s=gshape(L=2)) == INV and b"L must be 1" in L.dssm_last_error()
    assert call(s=gshape(L=0)) == INV
    assert call(s=gshape(L=1, dtype=7)) == INV
    assert call(s=gshape(B=1 << 16, H=1 << 15, L=1)) == UNS
    assert call(inp=inputs(stride_b=2)) == INV
    assert call(inp=inputs(u=None)) == INV and call(y=None) == INV
    assert call(y=at(1)) == INV and call(y=at(5)) == INV
    assert call(s=gshape(B=0, L=1), inp=inputs(u=None)) == 0


def test_gated_backward_refuses():
    L = bd.lib()

    def grads(**bad):
        v = dict(du=at(10), dr=at(11), di=at(12), stride_b=120, dlog_re=at(13), dx0=at(14))
        v.update(bad)
        return bd.GatedGrads(*[v[k] for k in ("du", "dr", "di", "stride_b", "dlog_re", "dx0")])

    def call(s=None, inp=None, kind=bd.CKPT_STATE, ckpt=at(8), dy=at(7), dx=at(6), g=None,
             ws=at(9), n=1 << 30):
        s = gshape() if s is None else s
        inp = inputs() if inp is None else inp
        g = grads() if g is None else g
        return L.dssm_gated_backward(ctypes.byref(inp), ctypes.byref(s), kind, ckpt, dy, dx,
                                     ctypes.byref(g), ws, n, None)

    for bad, rc in BAD_SHAPES:
        assert call(s=gshape(**bad)) == rc, bad
    assert call(kind=bd.CKPT_NONE) == INV and call(kind=3) == INV
    for k in ("u", "r", "i"):
        assert call(inp=inputs(**{k: None})) == INV
    assert call(inp=inputs(log_re=None)) == INV and call(inp=inputs(stride_b=7)) == INV
    for k in ("du", "dr", "di", "dlog_re"):
        assert call(g=grads(**{k: None})) == INV
        assert call(g=grads(**{k: at(7)})) == INV  # dy's memory
    assert call(g=grads(dr=at(10))) == INV and call(g=grads(stride_b=100)) == INV
    assert call(g=grads(dx0=at(6))) == INV and call(g=grads(du=at(0))) == INV
    assert call(dy=None) == INV and call(ckpt=None) == INV and call(ckpt=at(8) + 8) == INV
    assert call(n=16) == WS and call(ws=None) == INV
    # 8 bits: the inputs are not looked at, the gradients still are
    none = inputs(u=None, r=None, i=None, stride_b=0)
    assert call(inp=none, kind=bd.CKPT_INT8, n=16) == WS
    assert call(inp=none, kind=bd.CKPT_INT8, g=grads(du=None)) == INV
    assert call(s=gshape(H=0), inp=none) == 0


def test_ckpt8_refuses():
    L = bd.lib()
    for fn, args in ((L.dssm_ckpt8_pack, lambda x, b: (x, 6, 40, bd.F16, b, None)),
                     (L.dssm_ckpt8_unpack, lambda x, b: (b, 6, 40, bd.F16, x, None))):
        assert fn(*args(None, at(1))) == INV and fn(*args(at(0), None)) == INV
        assert fn(*args(at(0) + 1, at(1))) == INV and fn(*args(at(0), at(1) + 16)) == INV
        assert fn(*args(at(0), at(0))) == INV
    assert L.dssm_ckpt8_pack(at(0), 6, 40, 5, at(1), None) == INV
    assert L.dssm_ckpt8_pack(at(0), -6, 40, 0, at(1), None) == INV
    assert L.dssm_ckpt8_pack(None, 0, 40, 0, None, None) == 0
    assert L.dssm_ckpt8_unpack(None, 6, 0, 0, None, None) == 0


def rshape(B=2, H=3, L=40, dtype=bd.F32, norm=0, eps=1e-6):
    return bd.ResnormShape(B, H, L, dtype, norm, eps)


def rparams(**bad):
    v = dict(w_post=at(3), scale=at(4), w_pre=at(5))
    v.update(bad)
    return bd.ResnormParams(v["w_post"], v["scale"], v["w_pre"])


RBAD = [(dict(B=-1), INV), (dict(dtype=3), INV), (dict(norm=2), INV), (dict(eps=-1.0), INV),
        (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(H=8193), UNS),
        (dict(L=(1 << 24) + 1), UNS), (dict(B=5000, L=4000), UNS),
        (dict(B=(1 << 22) + 1, L=1), UNS)]


def test_resnorm_forward_refuses():
    L = bd.lib()

    def call(s=None, p=None, x=at(0), y=at(1), g=at(2), sg=120, lens=None, o=at(6), n=at(7),
             st=at(8)):
        return L.dssm_resnorm_forward(x, y, g, sg, ctypes.byref(p or rparams()),
                                      ctypes.byref(s or rshape()), lens, o, n, st, None)

    for bad, rc in RBAD:
        assert call(s=rshape(**bad)) == rc, bad
    assert call(x=None) == INV and call(x=at(0) + 2) == INV and call(y=at(1) + 2) == INV
    assert call(g=at(2) + 2) == INV and call(sg=119) == INV and call(lens=at(9) + 1) == INV
    assert call(o=None) == INV and call(y=None) == INV  # a gate (and o) without y
    assert call(y=None, g=None) == INV and call(y=None, g=None, o=None, n=None) == INV
    for k in ("w_post", "scale", "w_pre"):
        assert call(p=rparams(**{k: None})) == INV
    for out in ("o", "n", "st"):
        assert call(**{out: at(0)}) == INV
    assert call(o=at(7)) == INV and call(st=at(8) + 2) == INV
    assert call(s=rshape(B=0), x=None) == 0 and call(s=rshape(L=0), o=None) == 0


def test_resnorm_backward_refuses():
    L = bd.lib()

    def grads(**bad):
        v = dict(dx=at(10), dy=at(11), dg=at(12), stride_dg=120, dw_post=at(13), dscale=at(14),
                 dw_pre=at(15))
        v.update(bad)
        return bd.ResnormGrads(*[v[k] for k in ("dx", "dy", "dg", "stride_dg", "dw_post", "dscale",
                                                "dw_pre")])

    def call(s=None, p=None, o=at(0), y=at(1), g=at(2), sg=120, st=at(6), do=at(7), dn=at(8),
             gr=None, ws=at(9), n=1 << 30):
        return L.dssm_resnorm_backward(o, y, g, sg, st, ctypes.byref(p or rparams()),
                                       ctypes.byref(s or rshape()), None, do, dn,
                                       ctypes.byref(gr or grads()), ws, n, None)

    for bad, rc in RBAD:
        assert call(s=rshape(**bad)) == rc, bad
    assert call(do=None, dn=None) == INV and call(y=None, g=None, dn=None) == INV
    assert call(o=None) == INV and call(st=None) == INV and call(sg=100) == INV
    for k in ("dx", "dy", "dg", "dw_post", "dscale", "dw_pre"):
        assert call(gr=grads(**{k: None})) == INV, k
        assert call(gr=grads(**{k: at(7)})) == INV, k
    assert call(gr=grads(stride_dg=100)) == INV and call(gr=grads(dx=at(11))) == INV
    assert call(n=16) == WS and call(ws=at(9) + 64) == INV
    # without y its gradients may be left out
    assert call(y=None, g=None, n=16,
                gr=grads(dy=None, dg=None, dw_post=None, dscale=None)) == WS
    assert call(s=rshape(H=0), o=None) == 0
    assert size(L.dssm_resnorm_workspace_size, ctypes.byref(rshape(B=0))) == (0, 0)
    rc, n = size(L.dssm_resnorm_workspace_size, ctypes.byref(rshape()))
    assert rc == 0 and n >= 3 * 3 * 4 and n % 256 == 0


def test_binding_needs_a_checkpoint():
    """A backward pass reads what a forward pass kept: None is refused, and no
    buffer made in its place (host side; nothing is launched)."""
    import torch
    dy = torch.zeros(1, 2, 3)
    for kind in (bd.CKPT_STATE, bd.CKPT_INT8):
        for ckpt in (None, 1 << 20):
            with pytest.raises(TypeError, match="ckpt"):
                bd.gated_backward(dy, ckpt, kind, torch.ones(2), u=dy, r=dy, i=dy)
    with pytest.raises(ValueError, match="blob"):
        bd.ckpt8_unpack(None, (2, 3), torch.float32)


def test_scratch_memory_is_its_own():
    """A checkpoint or workspace that is another buffer of the call would be
    written over while it is read: refused."""
    L = bd.lib()
    inp, s = inputs(lens=at(4)), gshape()

    def forward(ckpt, ws, kind=bd.CKPT_INT8):
        rc = L.dssm_gated_forward(ctypes.byref(inp), ctypes.byref(s), at(5), at(6), at(7), kind,
                                  ckpt, ws, 1 << 30, None)
        return rc, L.dssm_last_error()

    for k in list(range(8)) + [9]:
        rc, text = forward(at(k), at(9))
        assert rc == INV and b"alias" in text, k
    for k in range(9):
        rc, text = forward(at(8), at(k))
        assert rc == INV and b"alias" in text, k
    g = bd.GatedGrads(at(10), at(11), at(12), 120, at(13), at(14))
    for kind in (bd.CKPT_STATE, bd.CKPT_INT8):
        for k in ([0, 1, 2] if kind == bd.CKPT_STATE else []) + [3, 4, 6, 7, 8, 10, 11, 12, 13, 14]:
            assert L.dssm_gated_backward(ctypes.byref(inp), ctypes.byref(s), kind, at(8), at(7), at(6),
                                         ctypes.byref(g), at(k), 1 << 30, None) == INV, (kind, k)
            assert b"alias" in L.dssm_last_error()
    gr = bd.ResnormGrads(at(10), at(11), at(12), 120, at(13), at(14), at(15))
    for k in (0, 1, 2, 6, 7, 8, 10, 11, 12, 13, 14, 15):
        assert L.dssm_resnorm_backward(at(0), at(1), at(2), 120, at(6), ctypes.byref(rparams()),
                                       ctypes.byref(rshape()), None, at(7), at(8), ctypes.byref(gr),
                                       at(k), 1 << 30, None) == INV, k
        assert b"alias" in L.dssm_last_error()
