"""What the short convolution, the selective scan and the norm in 8 bits refuse
(C ABI, host side; no kernel is launched), and the sizes they report."""
import ctypes

import pytest

from long_convolution_sequence_amd import binding as bd

FAKE = 1 << 20  # an aligned, never-dereferenced device address
INV, UNS, WS = bd.DSSM_ERR_INVALID_ARG, bd.DSSM_ERR_UNSUPPORTED, bd.DSSM_ERR_WORKSPACE


def at(k):
    return FAKE * (k + 1)


def size(fn, *args):
    out = ctypes.c_size_t(123)
    rc = fn(*(list(args) + [ctypes.byref(out)]))
    return rc, out.value


def cshape(B=2, H=3, L=40, K=4, dtype=bd.BF16, act=bd.ACT_SILU):
    return bd.ShortconvShape(B, H, L, K, dtype, act)


def sshape(B=2, H=6, L=40, N=5, G=2, dtype=bd.BF16):
    return bd.SelectiveShape(B, H, L, N, G, dtype)


DIMS = [(dict(B=-1), INV), (dict(H=-1), INV), (dict(L=-1), INV), (dict(dtype=3), INV),
        (dict(dtype=-1), INV), (dict(H=65536), UNS), (dict(L=(1 << 24) + 1), UNS),
        (dict(B=1 << 16, H=1 << 10), UNS), (dict(B=1 << 10, H=1 << 10, L=1 << 21), UNS)]
CBAD = DIMS + [(dict(K=0), INV), (dict(K=-3), INV), (dict(K=9), UNS), (dict(act=2), INV)]
SBAD = DIMS + [(dict(N=0), INV), (dict(N=129), UNS), (dict(G=0), INV), (dict(G=4), INV),
               (dict(G=-1), INV), (dict(B=1 << 13, H=1 << 11, N=128, L=4097, G=1), UNS),
               (dict(B=1 << 23, H=1, G=1, N=65, L=1), UNS)]


def test_shortconv_sizes():
    L = bd.lib()
    for bad, rc in CBAD:
        assert size(L.dssm_shortconv_workspace_size, ctypes.byref(cshape(**bad)))[0] == rc, bad
        assert L.dssm_last_error()
    assert L.dssm_shortconv_workspace_size(ctypes.byref(cshape()), None) == INV
    assert L.dssm_shortconv_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INV
    # 6 rows of 5 sums
    assert size(L.dssm_shortconv_workspace_size, ctypes.byref(cshape())) == (0, 256)
    assert size(L.dssm_shortconv_workspace_size, ctypes.byref(cshape(B=0))) == (0, 0)


@pytest.mark.parametrize("step", [False, True])
def test_shortconv_forward_refuses(step):
    L = bd.lib()
    fn = L.dssm_shortconv_step if step else L.dssm_shortconv_forward
    length = 1 if step else 40

    def call(s=None, u=at(0), sb=120, w=at(1), bias=at(2), lens=None, x0=at(3), xe=at(4), y=at(5)):
        return fn(u, sb, w, bias, ctypes.byref(s or cshape(L=length)), lens, x0, xe, y, None)

    for bad, rc in CBAD:
        got = call(s=cshape(**{**dict(L=length), **bad}))
        assert got == rc or (step and got == INV), bad
    if step:
        assert call(s=cshape(L=2)) == INV and b"L must be 1" in L.dssm_last_error()
        assert call(s=cshape(L=0)) == INV
    assert fn(at(0), 120, at(1), None, None, None, None, None, at(5), None) == INV
    assert call(u=None) == INV and call(u=at(0) + 1) == INV and call(w=None) == INV
    assert call(w=at(1) + 2) == INV and call(bias=at(2) + 2) == INV and call(lens=at(6) + 2) == INV
    assert call(sb=2) == INV and call(sb=(1 << 40) + 1) == UNS
    assert call(y=None) == INV and call(y=at(5) + 1) == INV and call(x0=at(3) + 1) == INV
    assert call(xe=at(4) + 1) == INV
    for k in (0, 1, 2, 3, 4):  # an output in another buffer's place
        assert call(y=at(k)) == INV, k
    assert call(xe=at(0)) == INV and call(xe=at(1)) == INV
    assert call(s=cshape(B=0, L=length), u=None) == 0
    assert call(s=cshape(H=0, L=length), y=None) == 0
    assert L.dssm_last_error() == b""


def test_shortconv_backward_refuses():
    L = bd.lib()

    def grads(**bad):
        v = dict(du=at(10), stride_b=120, dw=at(11), dbias=at(12), dx0=at(13))
        v.update(bad)
        return bd.ShortconvGrads(*[v[k] for k in ("du", "stride_b", "dw", "dbias", "dx0")])

    def call(s=None, u=at(0), sb=120, w=at(1), bias=at(2), lens=None, x0=at(3), dy=at(5), dx=at(6),
             g=None, ws=at(9), n=1 << 30):
        return L.dssm_shortconv_backward(u, sb, w, bias, ctypes.byref(s or cshape()), lens, x0, dy,
                                         dx, ctypes.byref(g or grads()), ws, n, None)

    for bad, rc in CBAD:
        assert call(s=cshape(**bad)) == rc, bad
    assert call(u=None) == INV and call(w=None) == INV and call(dy=None) == INV
    assert call(dy=at(5) + 1) == INV and call(dx=at(6) + 1) == INV and call(sb=7) == INV
    assert call(g=grads(du=None)) == INV and call(g=grads(dw=None)) == INV
    assert call(g=grads(stride_b=7)) == INV and call(g=grads(dx0=at(13) + 2)) == INV
    for k in ("du", "dw", "dbias", "dx0"):
        for other in (at(0), at(1), at(3), at(5), at(6), at(9)):
            assert call(g=grads(**{k: other})) == INV, (k, other)
    assert call(n=16) == WS and call(ws=None) == INV and call(ws=at(9) + 16) == INV
    assert call(s=cshape(H=0), u=None, dy=None) == 0


def sinputs(**bad):
    v = dict(u=at(0), delta=at(1), z=at(2), Bm=at(3), Cm=at(4), stride_u=240, stride_delta=240,
             stride_z=240, stride_B=400, stride_C=400, log_re=at(5), D=at(6), dt_bias=at(7),
             lens=None)
    v.update(bad)
    return bd.SelectiveInputs(*[v[k] for k, _ in bd.SelectiveInputs._fields_])


def sgrads(**bad):
    v = dict(du=at(20), ddelta=at(21), dz=at(22), dB=at(23), dC=at(24), stride_u=240,
             stride_delta=240, stride_z=240, stride_B=400, stride_C=400, dlog_re=at(25), dD=at(26),
             ddt_bias=at(27), dx0=at(28))
    v.update(bad)
    return bd.SelectiveGrads(*[v[k] for k, _ in bd.SelectiveGrads._fields_])


def test_selective_sizes():
    L = bd.lib()
    for bad, rc in SBAD:
        s = ctypes.byref(sshape(**bad))
        for back in (0, 1):
            assert size(L.dssm_selective_workspace_size, s, back)[0] == rc, bad
        assert size(L.dssm_selective_ckpt_size, s)[0] == rc, bad
    s = ctypes.byref(sshape())
    assert L.dssm_selective_workspace_size(s, 0, None) == INV
    assert L.dssm_selective_ckpt_size(s, None) == INV
    assert size(L.dssm_selective_workspace_size, s, 0) == (0, 0)
    # 2 2 2 5 rows of 128 steps; 12 rows of 5 modes (-> 256); 12 rows of 2 (-> 256)
    assert size(L.dssm_selective_workspace_size, s, 1) == (0, 4 * 40 * 128 + 512)
    assert size(L.dssm_selective_ckpt_size, s) == (0, 256)
    assert size(L.dssm_selective_ckpt_size, ctypes.byref(sshape(L=300))) == (0, 768)
    for empty in (sshape(B=0), sshape(H=0)):
        assert size(L.dssm_selective_workspace_size, ctypes.byref(empty), 1) == (0, 0)
        assert size(L.dssm_selective_ckpt_size, ctypes.byref(empty)) == (0, 0)
    # few long rows are cut into segments, which are joined in the workspace
    long_rows = ctypes.byref(sshape(B=1, H=4, G=1, L=1 << 16))
    assert size(L.dssm_selective_workspace_size, long_rows, 0)[1] > 0


def check_selective_inputs(L, call, strides):
    for k in ("u", "delta", "Bm", "Cm", "log_re"):
        assert call(inp=sinputs(**{k: None})) == INV and k.encode() in L.dssm_last_error()
        assert call(inp=sinputs(**{k: at(0) + 1})) == INV
    assert call(inp=sinputs(z=at(2) + 1)) == INV
    for k in ("D", "dt_bias", "lens"):
        assert call(inp=sinputs(**{k: at(9) + 2})) == INV
    for k, least in strides.items():
        assert call(inp=sinputs(**{k: least - 1})) == INV and k.encode() in L.dssm_last_error()
        assert call(inp=sinputs(**{k: (1 << 40) + 1})) == UNS


def test_selective_forward_refuses():
    L = bd.lib()

    def call(s=None, inp=None, x0=at(10), xe=at(11), y=at(12), ckpt=at(13), ws=at(14), n=1 << 30):
        return L.dssm_selective_forward(ctypes.byref(inp or sinputs()), ctypes.byref(s or sshape()),
                                        x0, xe, y, ckpt, ws, n, None)

    for bad, rc in SBAD:
        assert call(s=sshape(**bad)) == rc, bad
    check_selective_inputs(L, call, dict(stride_u=240, stride_delta=240, stride_z=240,
                                         stride_B=400, stride_C=400))
    assert call(y=None) == INV and call(y=at(12) + 1) == INV
    assert call(x0=at(10) + 2) == INV and call(xe=at(11) + 2) == INV
    for k in list(range(8)) + [10, 11]:
        assert call(y=at(k)) == INV, k
    for k in range(8):
        assert call(xe=at(k)) == INV, k
    assert call(ckpt=at(13) + 16) == INV
    for k in list(range(8)) + [10, 11, 12]:
        assert call(ckpt=at(k)) == INV, k
    long_rows = sshape(B=1, H=6, L=1 << 16)
    assert call(s=long_rows, n=16) == WS and call(s=long_rows, ws=None) == INV
    assert call(s=long_rows, ws=at(14) + 16) == INV and call(s=long_rows, ws=at(12)) == INV
    assert call(s=sshape(B=0), inp=sinputs(u=None)) == 0 and call(s=sshape(H=0, G=1), y=None) == 0
    assert L.dssm_last_error() == b""


def test_selective_step_refuses():
    L = bd.lib()

    def call(s=None, inp=None, x0=at(10), xe=at(10), y=at(12)):
        return L.dssm_selective_step(ctypes.byref(inp or sinputs()),
                                     ctypes.byref(s or sshape(L=1)), x0, xe, y, None)

    assert call(s=sshape(L=2)) == INV and b"L must be 1" in L.dssm_last_error()
    assert call(s=sshape(L=0)) == INV and call(s=sshape(L=1, N=129)) == UNS
    check_selective_inputs(L, call, dict(stride_u=6, stride_delta=6, stride_z=6, stride_B=10,
                                         stride_C=10))
    assert call(y=None) == INV and call(y=at(1)) == INV and call(y=at(10)) == INV
    assert call(xe=at(3)) == INV
    assert call(s=sshape(B=0, L=1), inp=sinputs(u=None)) == 0


def test_selective_backward_refuses():
    L = bd.lib()

    def call(s=None, inp=None, ckpt=at(13), dy=at(15), dx=at(16), g=None, ws=at(14), n=1 << 30):
        return L.dssm_selective_backward(ctypes.byref(inp or sinputs()),
                                         ctypes.byref(s or sshape()), ckpt, dy, dx,
                                         ctypes.byref(g or sgrads()), ws, n, None)

    for bad, rc in SBAD:
        assert call(s=sshape(**bad)) == rc, bad
    check_selective_inputs(L, call, dict(stride_u=240, stride_delta=240, stride_z=240,
                                         stride_B=400, stride_C=400))
    for k in ("du", "ddelta", "dz", "dB", "dC", "dlog_re", "dD", "ddt_bias"):
        assert call(g=sgrads(**{k: None})) == INV, k
    for k in ("du", "ddelta", "dz", "dB", "dC", "dlog_re", "dD", "ddt_bias", "dx0"):
        for other in [at(i) for i in list(range(8)) + [13, 14, 15, 16]]:
            assert call(g=sgrads(**{k: other})) == INV, (k, other)
    for k in ("stride_u", "stride_delta", "stride_z", "stride_B", "stride_C"):
        assert call(g=sgrads(**{k: 7})) == INV
    # gradients of inputs that are not there
    for k, d in (("z", "dz"), ("D", "dD"), ("dt_bias", "ddt_bias")):
        assert call(inp=sinputs(**{k: None})) == INV and d.encode() in L.dssm_last_error()
    assert call(ckpt=None) == INV and call(ckpt=at(13) + 8) == INV
    assert call(dy=None) == INV and call(dx=at(16) + 2) == INV
    assert call(n=16) == WS and call(ws=None) == INV and call(ws=at(14) + 16) == INV
    assert call(s=sshape(H=0, G=1), inp=sinputs(u=None)) == 0


def test_launches_of_2_to_the_32_lanes():
    """Calls within the other limits that one launch cannot hold are refused before any."""
    L = bd.lib()
    rows = ctypes.byref(cshape(B=1 << 7, H=1 << 10, L=1 << 18))  # 2^35 steps, 8 to a lane
    assert L.dssm_shortconv_forward(at(0), 1 << 28, at(1), at(2), rows, None, None, None, at(5),
                                    None) == UNS
    assert b"2^32 lanes" in L.dssm_last_error()
    # a channel to a group: a workgroup of 512 lanes to each of 2^23 rows
    for length in (1, 65):
        s = sshape(B=1 << 12, H=1 << 11, G=1 << 11, N=1, L=length)
        t = length << 11
        inp = sinputs(stride_u=t, stride_delta=t, stride_z=t, stride_B=t, stride_C=t)
        assert L.dssm_selective_forward(ctypes.byref(inp), ctypes.byref(s), None, None, at(12),
                                        None, at(14), 1 << 40, None) == UNS
        g = sgrads(stride_u=t, stride_delta=t, stride_z=t, stride_B=t, stride_C=t)
        assert L.dssm_selective_backward(ctypes.byref(inp), ctypes.byref(s), at(13), at(15), None,
                                         ctypes.byref(g), at(14), 1 << 50, None) == UNS
        assert b"2^32 lanes" in L.dssm_last_error()


def test_resnorm8_refuses():
    L = bd.lib()

    def call(s=None, p=None, x=at(0), y=at(1), g=at(2), sg=120, lens=None, form=bd.Q8_INT8,
             o=at(6), q=at(7), qs=at(8), st=at(9)):
        s = s or bd.ResnormShape(2, 3, 40, bd.F32, 0, 1e-6)
        p = bd.ResnormParams(at(3), at(4), at(5)) if p is None else p
        return L.dssm_resnorm8_forward(x, y, g, sg, ctypes.byref(p), ctypes.byref(s), lens, form, o,
                                       q, qs, st, None)

    for bad, rc in ((dict(B=-1), INV), (dict(dtype=3), INV), (dict(norm=2), INV),
                    (dict(eps=-1.0), INV), (dict(H=8193), UNS), (dict(L=(1 << 20) + 1), UNS),
                    (dict(B=(1 << 22) + 1, L=1), UNS)):
        v = {**dict(B=2, H=3, L=40, dtype=0, norm=0, eps=1e-6), **bad}
        s = bd.ResnormShape(*[v[k] for k in ("B", "H", "L", "dtype", "norm", "eps")])
        assert call(s=s) == rc, bad
    assert call(form=2) == INV and call(form=-1) == INV
    assert call(x=None) == INV and call(x=at(0) + 2) == INV and call(y=at(1) + 2) == INV
    assert call(sg=119) == INV and call(lens=at(9) + 1) == INV
    assert call(o=None) == INV and call(q=None) == INV and call(qs=None) == INV
    assert call(qs=at(8) + 2) == INV and call(st=at(9) + 2) == INV
    assert call(y=None) == INV and call(y=None, g=None) == INV  # o without y
    none = ctypes.c_void_p(None).value
    # without w_post y is only added: neither scale nor gate
    assert call(p=bd.ResnormParams(none, at(4), at(5)), g=None) == INV
    assert call(p=bd.ResnormParams(none, none, at(5))) == INV
    assert call(p=bd.ResnormParams(at(3), none, at(5))) == INV
    assert call(p=bd.ResnormParams(at(3), at(4), none)) == INV
    for k in ("o", "q", "qs", "st"):
        for other in (at(0), at(1), at(2), at(3), at(5)):
            assert call(**{k: other}) == INV, (k, other)
    assert call(q=at(6)) == INV and call(qs=at(7)) == INV
    empty = bd.ResnormShape(0, 3, 40, bd.F32, 0, 1e-6)
    assert call(s=empty, x=None) == 0
