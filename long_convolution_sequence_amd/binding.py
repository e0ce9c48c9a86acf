"""ctypes binding of libdssm.so (C ABI in include/dssm.h).

Argument marshalling only: every step of the forward map runs in the library's
HIP kernels.  Torch supplies device memory and the current stream.  If the
library is missing or a call fails, an exception is raised -- there is no
fallback path.
"""
import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdssm.so")

DSSM_OK = 0
DSSM_ERR_INVALID_ARG = -1
DSSM_ERR_UNSUPPORTED = -2
DSSM_ERR_WORKSPACE = -3
DSSM_ERR_HIP = -4

OP_GEN, OP_FFT, OP_SCAN, OP_BWD, OP_S5_SCAN, OP_S5_FFT, OP_S5_FUSED = 0, 1, 2, 3, 4, 5, 6
# how the S5 state recurrence runs: scan between the projections, per-state FFT
# convolution, or fused with both projections (v and x on chip)
S5_SCAN, S5_FFT, S5_FUSED = 0, 1, 2
CAST_RE, CAST_RE_IM = 0, 1  # Re K, or Re K * Im K (DLR-prod)
F32, BF16, F16 = 0, 1, 2  # activation types of the gated recurrence and the block around it
# what a gated forward keeps: nothing, the states entering its chunks, or these
# and u, r, i in 8 bits
CKPT_NONE, CKPT_STATE, CKPT_INT8 = 0, 1, 2
GATED_CHUNK, CKPT8_GROUP = 512, 64
NORM_RMS, NORM_LAYER = 0, 1

# Every function the header declares (checked by the ABI tests).
EXPORTS = [
    "dssm_version", "dssm_status_string", "dssm_last_error", "dssm_workspace_size",
    "dssm_gen_kernel", "dssm_gen_kernel_cast", "dssm_forward_fft", "dssm_forward_fft_noalloc",
    "dssm_forward_fft_cast",
    "dssm_forward_scan", "dssm_backward",
    "dssm_forward_fft_timed", "dssm_forward_scan_timed",
    "dssm_forward_scan_state", "dssm_step",
    "dssm_s5_workspace_size", "dssm_s5_tv_workspace_size", "dssm_s5_forward",
    "dssm_s5_forward_timed", "dssm_s5_forward_tv",
    "dssm_gated_workspace_size", "dssm_gated_ckpt_size", "dssm_gated_forward", "dssm_gated_step",
    "dssm_gated_backward", "dssm_ckpt8_size", "dssm_ckpt8_pack", "dssm_ckpt8_unpack",
    "dssm_resnorm_forward", "dssm_resnorm_workspace_size", "dssm_resnorm_backward",
]


class Grads(ctypes.Structure):
    _fields_ = [("dlog_re", ctypes.c_void_p), ("dlog_im", ctypes.c_void_p),
                ("dW", ctypes.c_void_p), ("dD", ctypes.c_void_p)]


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("L", ctypes.c_int), ("bidirectional", ctypes.c_int)]


class DLRParams(ctypes.Structure):
    _fields_ = [("log_re", ctypes.c_void_p), ("log_im", ctypes.c_void_p),
                ("W", ctypes.c_void_p), ("D", ctypes.c_void_p)]


class S5Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("P", ctypes.c_int),
                ("L", ctypes.c_int), ("bidirectional", ctypes.c_int)]


class S5Params(ctypes.Structure):
    _fields_ = [("lam", ctypes.c_void_p), ("Bbar", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("D", ctypes.c_void_p)]


class S5TVParams(ctypes.Structure):
    _fields_ = [("lam_c", ctypes.c_void_p), ("Bt", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("D", ctypes.c_void_p), ("delta", ctypes.c_void_p)]


class GatedShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class GatedInputs(ctypes.Structure):
    _fields_ = [("u", ctypes.c_void_p), ("r", ctypes.c_void_p), ("i", ctypes.c_void_p),
                ("stride_b", ctypes.c_longlong), ("log_re", ctypes.c_void_p),
                ("lens", ctypes.c_void_p)]


class GatedGrads(ctypes.Structure):
    _fields_ = [("du", ctypes.c_void_p), ("dr", ctypes.c_void_p), ("di", ctypes.c_void_p),
                ("stride_b", ctypes.c_longlong), ("dlog_re", ctypes.c_void_p),
                ("dx0", ctypes.c_void_p)]


class ResnormShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int),
                ("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float)]


class ResnormParams(ctypes.Structure):
    _fields_ = [("w_post", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p)]


class ResnormGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("dg", ctypes.c_void_p),
                ("stride_dg", ctypes.c_longlong), ("dw_post", ctypes.c_void_p),
                ("dscale", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p)]


class DSSMError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("dssm status %d: %s" % (status, message))
        self.status = status


_lib = None


def lib():
    """Load libdssm.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libdssm.so is not built; run `python -m long_convolution_sequence_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    L.dssm_version.restype = ctypes.c_int
    L.dssm_version.argtypes = []
    L.dssm_status_string.restype = ctypes.c_char_p
    L.dssm_status_string.argtypes = [ctypes.c_int]
    L.dssm_last_error.restype = ctypes.c_char_p
    L.dssm_last_error.argtypes = []
    L.dssm_workspace_size.restype = ctypes.c_int
    L.dssm_workspace_size.argtypes = [ctypes.c_int, ctypes.POINTER(Shape), ctypes.POINTER(sz)]
    L.dssm_gen_kernel.restype = ctypes.c_int
    L.dssm_gen_kernel.argtypes = [ctypes.POINTER(DLRParams), ctypes.POINTER(Shape), ctypes.c_int,
                                  vp, vp, sz, vp]
    L.dssm_gen_kernel_cast.restype = ctypes.c_int
    L.dssm_gen_kernel_cast.argtypes = [ctypes.POINTER(DLRParams), ctypes.POINTER(Shape),
                                       ctypes.c_int, vp, vp, sz, vp]
    L.dssm_backward.restype = ctypes.c_int
    L.dssm_backward.argtypes = [vp, vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape), vp,
                                ctypes.POINTER(Grads), vp, sz, vp]
    L.dssm_forward_fft_cast.restype = ctypes.c_int
    L.dssm_forward_fft_cast.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape),
                                        ctypes.c_int, vp, vp, sz, vp]
    for name in ("dssm_forward_fft", "dssm_forward_scan"):
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape), vp, vp, sz, vp]
    for name in ("dssm_forward_fft_timed", "dssm_forward_scan_timed"):
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape), vp, vp, sz, vp,
                      ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    L.dssm_forward_fft_noalloc.restype = ctypes.c_int
    L.dssm_forward_fft_noalloc.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape),
                                           vp, vp]
    L.dssm_forward_scan_state.restype = ctypes.c_int
    L.dssm_forward_scan_state.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape),
                                          vp, vp, vp, sz, vp]
    L.dssm_step.restype = ctypes.c_int
    L.dssm_step.argtypes = [vp, ctypes.POINTER(DLRParams), ctypes.POINTER(Shape), vp, vp, vp]
    L.dssm_s5_tv_workspace_size.restype = ctypes.c_int
    L.dssm_s5_tv_workspace_size.argtypes = [ctypes.POINTER(S5Shape), ctypes.POINTER(ctypes.c_size_t)]
    L.dssm_s5_workspace_size.restype = ctypes.c_int
    L.dssm_s5_workspace_size.argtypes = [ctypes.POINTER(S5Shape), ctypes.c_int,
                                         ctypes.POINTER(sz)]
    L.dssm_s5_forward.restype = ctypes.c_int
    L.dssm_s5_forward.argtypes = [vp, ctypes.POINTER(S5Params), ctypes.POINTER(S5Shape),
                                  ctypes.c_int, vp, vp, sz, vp]
    L.dssm_s5_forward_timed.restype = ctypes.c_int
    L.dssm_s5_forward_timed.argtypes = [vp, ctypes.POINTER(S5Params), ctypes.POINTER(S5Shape),
                                        ctypes.c_int, vp, vp, sz, vp,
                                        ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    L.dssm_s5_forward_tv.restype = ctypes.c_int
    L.dssm_s5_forward_tv.argtypes = [vp, ctypes.POINTER(S5TVParams), ctypes.POINTER(S5Shape), vp,
                                     vp, vp, sz, vp]
    P = ctypes.POINTER
    gi, gs, gg = P(GatedInputs), P(GatedShape), P(GatedGrads)
    rp, rs, rg = P(ResnormParams), P(ResnormShape), P(ResnormGrads)
    for name, args in (
            ("dssm_gated_workspace_size", [gs, P(sz)]),
            ("dssm_gated_ckpt_size", [gs, ctypes.c_int, P(sz)]),
            ("dssm_gated_forward", [gi, gs, vp, vp, vp, ctypes.c_int, vp, vp, sz, vp]),
            ("dssm_gated_step", [gi, gs, vp, vp, vp, vp]),
            ("dssm_gated_backward", [gi, gs, ctypes.c_int, vp, vp, vp, gg, vp, sz, vp]),
            ("dssm_ckpt8_size", [ctypes.c_longlong, ctypes.c_int, P(sz)]),
            ("dssm_ckpt8_pack", [vp, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, vp, vp]),
            ("dssm_ckpt8_unpack", [vp, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, vp, vp]),
            ("dssm_resnorm_forward", [vp, vp, vp, ctypes.c_longlong, rp, rs, vp, vp, vp, vp, vp]),
            ("dssm_resnorm_workspace_size", [rs, P(sz)]),
            ("dssm_resnorm_backward", [vp, vp, vp, ctypes.c_longlong, vp, rp, rs, vp, vp, vp, rg,
                                       vp, sz, vp])):
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    _lib = L
    return L


def check(status):
    if status != DSSM_OK:
        raise DSSMError(status, lib().dssm_last_error().decode())


def workspace_size(op, B, H, N, L, bidirectional=False):
    shape = Shape(B, H, N, L, int(bool(bidirectional)))
    out = ctypes.c_size_t(0)
    check(lib().dssm_workspace_size(op, ctypes.byref(shape), ctypes.byref(out)))
    return out.value


# ----------------------------------------------------------------------------
# torch-facing wrappers
# ----------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _dev_f32(t, name, numel=None, device=None):
    """t as a contiguous float32 device tensor (complex64 viewed as pairs),
    with `numel` float32 elements and on `device` when those are given."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype == torch.complex64:
        t = torch.view_as_real(t)
    if t.dtype != torch.float32:
        raise TypeError("%s must be float32 (or complex64), got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s has %d float32 elements, expected %d" % (name, t.numel(), numel))
    return t


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(stream):
    """Context for the binding's own allocations (workspace, default outputs):
    made on the stream the kernels run on, so the caching allocator does not
    hand their memory to another stream's allocation while those kernels may
    still use it."""
    import contextlib

    torch = _torch()
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _workspace(op, shape, workspace, device, stream=None):
    torch = _torch()
    need = ctypes.c_size_t(0)
    check(lib().dssm_workspace_size(op, ctypes.byref(shape), ctypes.byref(need)))
    if workspace is None:
        with _on_stream(stream):
            workspace = torch.empty(max(need.value, 256), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


def _empty(shape, dtype, device, stream):
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _params(log_re, log_im, W, D, ndir, H, N, device):
    n = ndir * H * N
    lr = _dev_f32(log_re, "log_re", n, device)
    li = _dev_f32(log_im, "log_im", n, device)
    w = _dev_f32(W, "W", 2 * n, device)
    if D is None:  # generator only
        return DLRParams(lr.data_ptr(), li.data_ptr(), w.data_ptr(), None), (lr, li, w)
    d = _dev_f32(D, "D", ndir * H, device)
    keep = (lr, li, w, d)
    return DLRParams(lr.data_ptr(), li.data_ptr(), w.data_ptr(), d.data_ptr()), keep


def gen_kernel(log_re, log_im, W, L, complex_out=False, out=None, workspace=None, stream=None):
    """K[d,h,j] = sum_n W lambda^j for j < L.  log_re/log_im [ndir,H,N] f32,
    W [ndir,H,N] c64.  Returns Re K [ndir,H,L] f32 or K [ndir,H,L] c64."""
    torch = _torch()
    ndir, H, N = log_re.shape
    dev = log_re.device
    shape = Shape(1, H, N, L, ndir - 1)
    p, keep = _params(log_re, log_im, W, None, ndir, H, N, dev)
    if out is None:
        out = _empty((ndir, H, L), torch.complex64 if complex_out else torch.float32, dev, stream)
    o = _dev_f32(out, "out", ndir * H * L * (2 if complex_out else 1), dev)
    ws, nbytes = _workspace(OP_GEN, shape, workspace, dev, stream)
    check(lib().dssm_gen_kernel(ctypes.byref(p), ctypes.byref(shape), int(bool(complex_out)),
                                o.data_ptr(), ws.data_ptr(), nbytes, _stream(stream)))
    del keep
    return out


def gen_kernel_cast(log_re, log_im, W, L, cast=CAST_RE, out=None, workspace=None, stream=None):
    """The real kernel of a cast: Re K (CAST_RE) or Re K * Im K (CAST_RE_IM,
    DLR-prod), [ndir,H,L] f32."""
    torch = _torch()
    ndir, H, N = log_re.shape
    dev = log_re.device
    shape = Shape(1, H, N, L, ndir - 1)
    p, keep = _params(log_re, log_im, W, None, ndir, H, N, dev)
    if out is None:
        out = _empty((ndir, H, L), torch.float32, dev, stream)
    o = _dev_f32(out, "out", ndir * H * L, dev)
    ws, nbytes = _workspace(OP_GEN, shape, workspace, dev, stream)
    check(lib().dssm_gen_kernel_cast(ctypes.byref(p), ctypes.byref(shape), int(cast),
                                     o.data_ptr(), ws.data_ptr(), nbytes, _stream(stream)))
    del keep
    return out


def _rows(u, name="u"):
    uu = _dev_f32(u, name)
    if uu.dim() != 3:
        raise ValueError("%s must be [B, H, L]" % name)
    return uu


def _forward(fn, op, u, log_re, log_im, W, D, bidirectional, y, workspace, stream, events=None,
             cast=None):
    torch = _torch()
    uu = _rows(u)
    B, H, L = uu.shape
    dev = uu.device
    ndir = 2 if bidirectional else 1
    N = log_re.shape[-1]
    shape = Shape(B, H, N, L, int(bool(bidirectional)))
    p, keep = _params(log_re, log_im, W, D, ndir, H, N, dev)
    if y is None:
        y = _empty(uu.shape, torch.float32, dev, stream)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    ws, nbytes = _workspace(op, shape, workspace, dev, stream)
    args = [uu.data_ptr(), ctypes.byref(p), ctypes.byref(shape)]
    if cast is not None:
        args.append(int(cast))
    args += [yy.data_ptr(), ws.data_ptr(), nbytes, _stream(stream)]
    if events is not None:
        arr = (ctypes.c_void_p * len(events))(*events)
        args += [arr, len(events)]
    check(fn(*args))
    del keep
    return y


def forward_fft(u, log_re, log_im, W, D, bidirectional=False, y=None, workspace=None, stream=None):
    """Layer forward by the FFT convolution view.  u [B,H,L] f32 -> y [B,H,L]."""
    return _forward(lib().dssm_forward_fft, OP_FFT, u, log_re, log_im, W, D, bidirectional, y,
                    workspace, stream)


def forward_fft_noalloc(u, log_re, log_im, W, D, y, bidirectional=False, stream=None):
    """forward_fft into the caller's y with the library's fixed per-device
    scratch array as workspace: nothing is allocated, here or in the library.
    Calls that overlap in time on one device race on that array."""
    uu = _rows(u)
    B, H, L = uu.shape
    dev = uu.device
    ndir = 2 if bidirectional else 1
    N = log_re.shape[-1]
    shape = Shape(B, H, N, L, int(bool(bidirectional)))
    p, keep = _params(log_re, log_im, W, D, ndir, H, N, dev)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    check(lib().dssm_forward_fft_noalloc(uu.data_ptr(), ctypes.byref(p), ctypes.byref(shape),
                                         yy.data_ptr(), _stream(stream)))
    del keep
    return y


def forward_fft_cast(u, log_re, log_im, W, D, cast, bidirectional=False, y=None, workspace=None,
                     stream=None):
    """Layer forward by the FFT convolution view with the kernel cast `cast`
    (CAST_RE: as forward_fft; CAST_RE_IM: DLR-prod)."""
    return _forward(lib().dssm_forward_fft_cast, OP_FFT, u, log_re, log_im, W, D, bidirectional, y,
                    workspace, stream, cast=cast)


def backward(u, dy, log_re, log_im, W, D, bidirectional=False, du=None, workspace=None,
             stream=None):
    """Gradients of f = sum(dy * y) for the layer map: returns du [B,H,L] f32
    and a dict dlog_re, dlog_im [ndir,H,N] f32, dW [ndir,H,N] c64
    (d/d Re W + i d/d Im W), dD [ndir,H] f32."""
    torch = _torch()
    uu = _rows(u)
    dev = uu.device
    gg = _dev_f32(dy, "dy", uu.numel(), dev)
    B, H, L = uu.shape
    ndir = 2 if bidirectional else 1
    N = log_re.shape[-1]
    shape = Shape(B, H, N, L, int(bool(bidirectional)))
    p, keep = _params(log_re, log_im, W, D, ndir, H, N, dev)
    if du is None:
        du = _empty(uu.shape, torch.float32, dev, stream)
    dd = _dev_f32(du, "du", uu.numel(), dev)
    out = dict(dlog_re=_empty((ndir, H, N), torch.float32, dev, stream),
               dlog_im=_empty((ndir, H, N), torch.float32, dev, stream),
               dW=_empty((ndir, H, N), torch.complex64, dev, stream),
               dD=_empty((ndir, H), torch.float32, dev, stream))
    g = Grads(out["dlog_re"].data_ptr(), out["dlog_im"].data_ptr(), out["dW"].data_ptr(),
              out["dD"].data_ptr())
    ws, nbytes = _workspace(OP_BWD, shape, workspace, dev, stream)
    check(lib().dssm_backward(uu.data_ptr(), gg.data_ptr(), ctypes.byref(p), ctypes.byref(shape),
                              dd.data_ptr(), ctypes.byref(g), ws.data_ptr(), nbytes,
                              _stream(stream)))
    del keep
    return du, out


def forward_scan(u, log_re, log_im, W, D, bidirectional=False, y=None, workspace=None, stream=None):
    """Layer forward by the recurrence (scan) view.  u [B,H,L] f32 -> y [B,H,L]."""
    return _forward(lib().dssm_forward_scan, OP_SCAN, u, log_re, log_im, W, D, bidirectional, y,
                    workspace, stream)


def forward_scan_state(u, log_re, log_im, W, D, x, y=None, workspace=None, stream=None):
    """Streaming forward, one direction: continues the recurrence from the
    state x [B,H,N] c64 (updated in place to the state after the last step).
    u [B,H,L] f32 -> y [B,H,L]."""
    torch = _torch()
    uu = _rows(u)
    B, H, L = uu.shape
    dev = uu.device
    N = log_re.shape[-1]
    shape = Shape(B, H, N, L, 0)
    p, keep = _params(log_re, log_im, W, D, 1, H, N, dev)
    xx = _dev_f32(x, "x", 2 * B * H * N, dev)
    if y is None:
        y = _empty(uu.shape, torch.float32, dev, stream)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    ws, nbytes = _workspace(OP_SCAN, shape, workspace, dev, stream)
    check(lib().dssm_forward_scan_state(uu.data_ptr(), ctypes.byref(p), ctypes.byref(shape),
                                        xx.data_ptr(), yy.data_ptr(), ws.data_ptr(), nbytes,
                                        _stream(stream)))
    del keep
    return y


def step(u_t, log_re, log_im, W, D, x, y=None, stream=None):
    """One decode step: u_t [B,H] f32 -> y_t [B,H]; x [B,H,N] c64 updated in
    place."""
    torch = _torch()
    uu = _dev_f32(u_t, "u_t")
    if uu.dim() != 2:
        raise ValueError("u_t must be [B, H]")
    B, H = uu.shape
    dev = uu.device
    N = log_re.shape[-1]
    shape = Shape(B, H, N, 1, 0)
    p, keep = _params(log_re, log_im, W, D, 1, H, N, dev)
    xx = _dev_f32(x, "x", 2 * B * H * N, dev)
    if y is None:
        y = _empty(uu.shape, torch.float32, dev, stream)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    check(lib().dssm_step(uu.data_ptr(), ctypes.byref(p), ctypes.byref(shape), xx.data_ptr(),
                          yy.data_ptr(), _stream(stream)))
    del keep
    return y


def forward_timed(path, u, log_re, log_im, W, D, events, bidirectional=False, y=None,
                  workspace=None, stream=None):
    """forward_fft / forward_scan whose stages the GPU brackets with the given
    raw hipEvent_t handles (ints, None for an untimed stage): a start/stop pair
    per stage, 4 in all -- fft: kernel spectrum (from the parameters),
    convolution; scan: constants, scan."""
    if path == "fft":
        fn, op = lib().dssm_forward_fft_timed, OP_FFT
    else:
        fn, op = lib().dssm_forward_scan_timed, OP_SCAN
    return _forward(fn, op, u, log_re, log_im, W, D, bidirectional, y, workspace, stream,
                    events=list(events))


def s5_workspace_size(B, H, P, L, method=S5_SCAN):
    shape = S5Shape(B, H, P, L, 0)
    out = ctypes.c_size_t(0)
    check(lib().dssm_s5_workspace_size(ctypes.byref(shape), int(method), ctypes.byref(out)))
    return out.value


def s5_tv_workspace_size(B, H, P, L):
    shape = S5Shape(B, H, P, L, 0)
    out = ctypes.c_size_t(0)
    check(lib().dssm_s5_tv_workspace_size(ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def _s5_workspace(shape, workspace, device, stream, method=S5_SCAN):
    """method None: the size dssm_s5_forward_tv needs."""
    torch = _torch()
    need = ctypes.c_size_t(0)
    if method is None:
        check(lib().dssm_s5_tv_workspace_size(ctypes.byref(shape), ctypes.byref(need)))
    else:
        check(lib().dssm_s5_workspace_size(ctypes.byref(shape), int(method), ctypes.byref(need)))
    if workspace is None:
        with _on_stream(stream):
            workspace = torch.empty(max(need.value, 256), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


def s5_forward(u, lam, Bbar, C, D, y=None, workspace=None, stream=None, events=None,
               method=S5_SCAN):
    """S5 layer forward.  u [B,H,L] f32, lam [P] c64, Bbar [P,H] c64,
    C [H,P] c64, D [H] f32 -> y [B,H,L] f32.  method: S5_SCAN (the
    recurrence as a scan between the projections), S5_FFT (per state, the
    convolution with lambda^j by FFT) or S5_FUSED (projections and
    recurrence in one pass, v and x on chip).  events: optional 8 raw
    hipEvent_t handles, a start/stop pair per stage (pack, proj_in,
    recurrence, proj_out; for S5_FUSED: pack, state-only pass, powers of
    lambda, output pass)."""
    torch = _torch()
    uu = _rows(u)
    B, H, L = uu.shape
    dev = uu.device
    lm = _dev_f32(lam, "lam", device=dev)
    P = lm.numel() // 2
    bb = _dev_f32(Bbar, "Bbar", 2 * P * H, dev)
    cc = _dev_f32(C, "C", 2 * H * P, dev)
    dd = _dev_f32(D, "D", H, dev)
    shape = S5Shape(B, H, P, L, 0)
    prm = S5Params(lm.data_ptr(), bb.data_ptr(), cc.data_ptr(), dd.data_ptr())
    if y is None:
        y = _empty(uu.shape, torch.float32, dev, stream)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    ws, nbytes = _s5_workspace(shape, workspace, dev, stream, method)
    args = [uu.data_ptr(), ctypes.byref(prm), ctypes.byref(shape), int(method), yy.data_ptr(),
            ws.data_ptr(), nbytes, _stream(stream)]
    if events is None:
        check(lib().dssm_s5_forward(*args))
    else:
        arr = (ctypes.c_void_p * len(events))(*events)
        check(lib().dssm_s5_forward_timed(*(args + [arr, len(events)])))
    return y


def s5_forward_tv(u, lam_c, Bt, C, D, delta, step, y=None, workspace=None, stream=None):
    """Continuous-time S5 layer forward with a step size per (b, k).  u [B,H,L]
    f32, lam_c [P] c64, Bt [P,H] c64, C [H,P] c64, D [H] f32, delta [P] f32,
    step [B,L] f32 -> y [B,H,L] f32."""
    torch = _torch()
    uu = _rows(u)
    B, H, L = uu.shape
    dev = uu.device
    lm = _dev_f32(lam_c, "lam_c", device=dev)
    P = lm.numel() // 2
    bb = _dev_f32(Bt, "Bt", 2 * P * H, dev)
    cc = _dev_f32(C, "C", 2 * H * P, dev)
    dd = _dev_f32(D, "D", H, dev)
    dl = _dev_f32(delta, "delta", P, dev)
    ss = _dev_f32(step, "step", B * L, dev)
    shape = S5Shape(B, H, P, L, 0)
    prm = S5TVParams(lm.data_ptr(), bb.data_ptr(), cc.data_ptr(), dd.data_ptr(), dl.data_ptr())
    if y is None:
        y = _empty(uu.shape, torch.float32, dev, stream)
    yy = _dev_f32(y, "y", uu.numel(), dev)
    ws, nbytes = _s5_workspace(shape, workspace, dev, stream, None)
    check(lib().dssm_s5_forward_tv(uu.data_ptr(), ctypes.byref(prm), ctypes.byref(shape),
                                   ss.data_ptr(), yy.data_ptr(), ws.data_ptr(), nbytes,
                                   _stream(stream)))
    return y


# ----------------------------------------------------------------------------
# the gated recurrence, 8-bit checkpoints, the residual norm
# ----------------------------------------------------------------------------

# The checks below pass a good tensor in a few attribute reads (a single token's
# call costs about as much on the host as on the device); what is wrong with a
# bad one is found out only then.

def _dtype_code(t, name):
    torch = _torch()
    if isinstance(t, torch.Tensor) and t.is_cuda:
        dt = t.dtype
        if dt is torch.bfloat16:
            return BF16
        if dt is torch.float32:
            return F32
        if dt is torch.float16:
            return F16
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    raise ValueError("%s must be a device tensor" % name)


def _like(t, name, ref, refname):
    """t has ref's shape, type and device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype is not ref.dtype:
        raise TypeError("%s is %s, %s is %s" % (name, t.dtype, refname, ref.dtype))
    if t.device != ref.device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, ref.device))
    if t.shape != ref.shape:
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), tuple(ref.shape)))
    return t


def _plain(t, name, ref, refname):
    """_like, and contiguous."""
    _like(t, name, ref, refname)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _vec(t, name, numel, device):
    """Address of a contiguous float32 device tensor of `numel` elements."""
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.numel() == numel
            and t.device == device and t.is_contiguous()):
        t = _dev_f32(t, name, numel, device)
    return t.data_ptr()


def _opt_vec(t, name, numel, device):
    return None if t is None else _vec(t, name, numel, device)


def _batch_stride(t, name):
    """Elements between the batch rows of t [B, H, L] (or [B, H]), whose H L
    elements are contiguous."""
    shape = t.shape
    if t.is_contiguous():
        return shape[1] * shape[2] if len(shape) == 3 else shape[1]
    st = t.stride()
    inner = 1
    for d in range(len(shape) - 1, 0, -1):
        if st[d] != inner and shape[d] > 1:
            raise ValueError("%s must be contiguous within each batch row" % name)
        inner *= shape[d]
    if shape[0] == 1:
        return inner
    if st[0] < inner:
        raise ValueError("%s has overlapping batch rows" % name)
    return st[0]


def _one_stride(a, b, c, names):
    s = _batch_stride(a, names[0])
    st = a.stride()  # tensors of one shape and one set of strides are alike
    if ((b.stride() != st and _batch_stride(b, names[1]) != s)
            or (c.stride() != st and _batch_stride(c, names[2]) != s)):
        raise ValueError("%s, %s and %s must have the same batch stride" % names)
    return s


def _lens_ptr(lens, B, device):
    if lens is None:
        return None
    torch = _torch()
    if not isinstance(lens, torch.Tensor) or lens.dtype != torch.int32:
        raise TypeError("lens must be an int32 tensor")
    if lens.device != device or not lens.is_contiguous() or lens.numel() != B:
        raise ValueError("lens must be a contiguous tensor of %d on %s" % (B, device))
    return lens.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new(t, stream):
    """An uninitialised contiguous tensor of t's shape and type, on `stream`."""
    if stream is None and t.is_contiguous():
        return _torch().empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _current_stream(device):
    """Handle of the device's current stream, without a Stream object where
    torch offers that (1.8 us of a 10 us call)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream


def _launch(fn, device, stream, *args):
    """fn(*args, stream) with `device` current, on the caller's stream or the
    device's current one; a failure raises."""
    torch = _torch()
    if stream is None:
        handle = _current_stream(device)
    elif stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != DSSM_OK:
        check(status)


@functools.lru_cache(maxsize=256)
def _gated_bytes(B, H, L, code, kind):
    """Bytes of a checkpoint of `kind`, or (kind None) of the workspace."""
    need = ctypes.c_size_t(0)
    shape = GatedShape(B, H, L, code)
    if kind is None:
        check(lib().dssm_gated_workspace_size(ctypes.byref(shape), ctypes.byref(need)))
    else:
        check(lib().dssm_gated_ckpt_size(ctypes.byref(shape), kind, ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=256)
def _resnorm_bytes(B, H, L, code, norm):
    """Bytes of workspace of the residual norm's backward pass."""
    need = ctypes.c_size_t(0)
    shape = ResnormShape(B, H, L, code, norm, 0.0)
    check(lib().dssm_resnorm_workspace_size(ctypes.byref(shape), ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=256)
def _ckpt8_bytes(rows, L):
    need = ctypes.c_size_t(0)
    check(lib().dssm_ckpt8_size(rows, L, ctypes.byref(need)))
    return need.value


def _buffer(need, given, name, device, stream):
    """A workspace or checkpoint of `need` bytes: the caller's, or new."""
    torch = _torch()
    if given is None:
        need = max(need, 256)
        return _empty((need,), torch.uint8, device, stream), need
    if not isinstance(given, torch.Tensor) or given.device != device or not given.is_contiguous():
        raise ValueError("%s must be a contiguous tensor on %s" % (name, device))
    n = given.numel() * given.element_size()
    if n < need and name != "workspace":  # a workspace's size the library checks itself
        raise ValueError("%s has %d bytes, needs %d" % (name, n, need))
    return given, n


def _gated_rows(u, r, i, dims):
    code = _dtype_code(u, "u")
    if u.dim() != dims:
        raise ValueError("u must be %s" % ("[B, H, L]" if dims == 3 else "[B, H]"))
    _like(r, "r", u, "u")
    _like(i, "i", u, "u")
    return code, _one_stride(u, r, i, ("u", "r", "i"))


def _gated_forward(u, r, i, log_re, kind, x, x_out, lens, y, ckpt, workspace, stream):
    code, sb = _gated_rows(u, r, i, 3)
    B, H, L = u.shape
    dev = u.device
    inp = GatedInputs(u.data_ptr(), r.data_ptr(), i.data_ptr(), sb, _vec(log_re, "log_re", H, dev),
                      _lens_ptr(lens, B, dev))
    xp = _opt_vec(x, "x", B * H, dev)
    xo = xp if x_out is None else _vec(x_out, "x_out", B * H, dev)
    y = _new(u, stream) if y is None else _plain(y, "y", u, "u")
    sp = ctypes.byref(GatedShape(B, H, L, code))
    ws, nbytes = _buffer(_gated_bytes(B, H, L, code, None), workspace, "workspace", dev, stream)
    if kind != CKPT_NONE:
        ckpt, _ = _buffer(_gated_bytes(B, H, L, code, kind), ckpt, "ckpt", dev, stream)
    _launch(lib().dssm_gated_forward, dev, stream, ctypes.byref(inp), sp, xp, xo, y.data_ptr(),
            kind, _ptr(ckpt), ws.data_ptr(), nbytes)
    return y, ckpt


def gated_forward(u, r, i, log_re, x=None, x_out=None, lens=None, y=None, workspace=None,
                  stream=None):
    """The gated recurrence: x_t = a_t x_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) u_t,
    a_t = exp(-log_re^2 sigmoid(r_t)), y_t = x_t.  u, r, i [B,H,L] f32, bf16 or
    f16 (slices of a joint [B,3H,L] projection are taken as they are), log_re
    [H] f32 -> y [B,H,L].  x [B,H] f32: the state before the first step, None
    for zero; the state after the last goes to x_out, or back to x.  lens [B]
    int32: live steps per batch row (y is 0 behind them)."""
    return _gated_forward(u, r, i, log_re, CKPT_NONE, x, x_out, lens, y, None, workspace,
                          stream)[0]


def gated_forward_ckpt(u, r, i, log_re, kind=CKPT_STATE, x=None, x_out=None, lens=None, y=None,
                       ckpt=None, workspace=None, stream=None):
    """gated_forward that keeps what gated_backward needs: returns (y, ckpt).
    kind CKPT_STATE: the states entering every 512 steps (the backward pass
    takes u, r, i again); CKPT_INT8: also u, r, i in 8 bits (it does not)."""
    if kind not in (CKPT_STATE, CKPT_INT8):
        raise ValueError("kind must be CKPT_STATE or CKPT_INT8")
    return _gated_forward(u, r, i, log_re, kind, x, x_out, lens, y, ckpt, workspace, stream)


def gated_step(u_t, r_t, i_t, log_re, x, x_out=None, lens=None, y=None, stream=None):
    """One token of the gated recurrence: u_t, r_t, i_t [B,H] -> y_t [B,H]; the
    state x [B,H] f32 is updated in place, or left and written to x_out.
    lens [B] int32: rows with 0 are idle (state kept, y 0)."""
    code, sb = _gated_rows(u_t, r_t, i_t, 2)
    B, H = u_t.shape
    dev = u_t.device
    inp = GatedInputs(u_t.data_ptr(), r_t.data_ptr(), i_t.data_ptr(), sb,
                      _vec(log_re, "log_re", H, dev), _lens_ptr(lens, B, dev))
    xp = _vec(x, "x", B * H, dev)
    xo = xp if x_out is None else _vec(x_out, "x_out", B * H, dev)
    y = _new(u_t, stream) if y is None else _plain(y, "y", u_t, "u_t")
    _launch(lib().dssm_gated_step, dev, stream, ctypes.byref(inp),
            ctypes.byref(GatedShape(B, H, 1, code)), xp, xo, y.data_ptr())
    return y


def gated_backward(dy, ckpt, kind, log_re, u=None, r=None, i=None, dx=None, lens=None, du=None,
                   dr=None, di=None, workspace=None, stream=None):
    """Gradients of f = sum(dy y) + sum(dx x_end) for the forward call that kept
    `ckpt` (gated_forward_ckpt of the same kind, shape and lens).  dy [B,H,L];
    u, r, i as there for CKPT_STATE, None for CKPT_INT8; dx [B,H] f32 or None.
    Returns a dict du, dr, di [B,H,L], dlog_re [H] f32, dx0 [B,H] f32 (du, dr,
    di given: slices of one [B,3H,L] buffer are written as they are)."""
    torch = _torch()
    # _buffer() below makes a buffer that is not given: this one is read
    if not isinstance(ckpt, torch.Tensor):
        raise TypeError("ckpt must be a torch tensor")
    code = _dtype_code(dy, "dy")
    if dy.dim() != 3:
        raise ValueError("dy must be [B, H, L]")
    if kind not in (CKPT_STATE, CKPT_INT8):
        raise ValueError("kind must be CKPT_STATE or CKPT_INT8")
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    B, H, L = dy.shape
    dev = dy.device
    sb = H * L
    if kind == CKPT_STATE:
        if u is None or r is None or i is None:
            raise ValueError("CKPT_STATE keeps states only: u, r and i are needed")
        for t, name in ((u, "u"), (r, "r"), (i, "i")):
            _like(t, name, dy, "dy")
        sb = _one_stride(u, r, i, ("u", "r", "i"))
    elif u is not None or r is not None or i is not None:
        raise ValueError("CKPT_INT8 holds u, r and i itself: pass none")
    out = {}
    for name, t in (("du", du), ("dr", dr), ("di", di)):
        out[name] = _new(dy, stream) if t is None else _like(t, name, dy, "dy")
    gsb = _one_stride(out["du"], out["dr"], out["di"], ("du", "dr", "di"))
    lp = _vec(log_re, "log_re", H, dev)
    out["dlog_re"] = (_new(log_re, stream) if log_re.dim() == 1
                      else _empty((H,), torch.float32, dev, stream))
    out["dx0"] = _empty((B, H), torch.float32, dev, stream)
    sp = ctypes.byref(GatedShape(B, H, L, code))
    ws, nbytes = _buffer(_gated_bytes(B, H, L, code, None), workspace, "workspace", dev, stream)
    ckpt, _ = _buffer(_gated_bytes(B, H, L, code, kind), ckpt, "ckpt", dev, stream)
    inp = GatedInputs(_ptr(u), _ptr(r), _ptr(i), sb, lp, _lens_ptr(lens, B, dev))
    g = GatedGrads(out["du"].data_ptr(), out["dr"].data_ptr(), out["di"].data_ptr(), gsb,
                   out["dlog_re"].data_ptr(), out["dx0"].data_ptr())
    _launch(lib().dssm_gated_backward, dev, stream, ctypes.byref(inp), sp, kind, ckpt.data_ptr(),
            dy.data_ptr(), _opt_vec(dx, "dx", B * H, dev), ctypes.byref(g), ws.data_ptr(), nbytes)
    return out


def _rows_of(shape):
    if len(shape) == 0:
        raise ValueError("at least one dimension is needed")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return rows, shape[-1]


def ckpt8_size(shape):
    """Bytes of a tensor of this shape in 8 bits."""
    return _ckpt8_bytes(*_rows_of(tuple(shape)))


def ckpt8_pack(x, blob=None, stream=None):
    """x [..., L] f32, bf16 or f16 in 8 bits: groups of 64 along L as int8 times
    a power of two.  Returns a uint8 tensor (the layout is dssm_ckpt8_pack's)."""
    code = _dtype_code(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    rows, L = _rows_of(x.shape)
    dev = x.device
    blob, _ = _buffer(_ckpt8_bytes(rows, L), blob, "blob", dev, stream)
    _launch(lib().dssm_ckpt8_pack, dev, stream, x.data_ptr(), rows, L, code, blob.data_ptr())
    return blob


def ckpt8_unpack(blob, shape, dtype, x=None, stream=None):
    """The values a ckpt8_pack blob stands for, in `dtype`."""
    torch = _torch()
    if not isinstance(blob, torch.Tensor) or not blob.is_cuda:
        raise ValueError("blob must be a device tensor")
    shape = tuple(shape)
    rows, L = _rows_of(shape)
    dev = blob.device
    _buffer(_ckpt8_bytes(rows, L), blob, "blob", dev, stream)
    if x is None:
        x = _empty(shape, dtype, dev, stream)
    code = _dtype_code(x, "x")
    if tuple(x.shape) != shape or x.dtype != dtype or x.device != dev or not x.is_contiguous():
        raise ValueError("x must be a contiguous %s tensor of %s on %s" % (dtype, shape, dev))
    _launch(lib().dssm_ckpt8_unpack, dev, stream, blob.data_ptr(), rows, L, code, x.data_ptr())
    return x


def _resnorm_dims(x, name):
    """B, H, L of [B, H, L], or of [B, H] as one step."""
    if x.dim() not in (2, 3):
        raise ValueError("%s must be [B, H, L] or [B, H]" % name)
    return x.shape[0], x.shape[1], (x.shape[2] if x.dim() == 3 else 1)


def _resnorm_params(w_post, scale, w_pre, H, dev, y, n):
    def vec(t, name, used):
        return _vec(t, name, H, dev) if used or t is not None else None

    return ctypes.byref(ResnormParams(vec(w_post, "w_post", y), vec(scale, "scale", y),
                                      vec(w_pre, "w_pre", n)))


def _resnorm_forward(x, y, g, w_post, scale, w_pre, norm, eps, lens, o, n, stats, stream):
    code = _dtype_code(x, "x")
    B, H, L = _resnorm_dims(x, "x")
    dev = x.device
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if y is None and (g is not None or o is not None):
        raise ValueError("a gate or a stream output needs y")
    if y is None and w_pre is None:
        raise ValueError("without y there is only n: w_pre is needed")
    sg = 0
    if y is not None:
        _plain(y, "y", x, "x")
        o = _new(x, stream) if o is None else _plain(o, "o", x, "x")
        if g is not None:
            sg = _batch_stride(_like(g, "g", x, "x"), "g")
    if w_pre is not None:
        n = _new(x, stream) if n is None else _plain(n, "n", x, "x")
    elif n is not None:
        raise ValueError("n needs w_pre")
    if stats is True:
        stats = _empty((4 if norm == NORM_LAYER else 2, B, L), _torch().float32, dev, stream)
    _launch(lib().dssm_resnorm_forward, dev, stream, x.data_ptr(), _ptr(y), _ptr(g), sg,
            _resnorm_params(w_post, scale, w_pre, H, dev, y is not None, n is not None),
            ctypes.byref(ResnormShape(B, H, L, code, int(norm), float(eps))),
            _lens_ptr(lens, B, dev), _ptr(o), _ptr(n), _ptr(stats))
    return o, n, stats


def resnorm_forward(x, y, g, w_post, scale, w_pre, norm=NORM_RMS, eps=1e-6, lens=None, o=None,
                    n=None, stream=None):
    """Around a layer: o = x + scale norm(y) w_post silu(g), n = norm(o) w_pre,
    the norms over the H channels.  x, y, g [B,H,L] (or [B,H]: one token; g may
    be a slice of a joint projection), w_post, scale, w_pre [H] f32.  Returns
    (o, n).  g None: no gate; y None: n = norm(x) w_pre and o is None; w_pre
    None: n is None."""
    return _resnorm_forward(x, y, g, w_post, scale, w_pre, norm, eps, lens, o, n, None,
                            stream)[:2]


def resnorm_forward_stats(x, y, g, w_post, scale, w_pre, norm=NORM_RMS, eps=1e-6, lens=None,
                          o=None, n=None, stream=None):
    """resnorm_forward that also returns what resnorm_backward needs: (o, n, stats)."""
    return _resnorm_forward(x, y, g, w_post, scale, w_pre, norm, eps, lens, o, n, True, stream)


def resnorm_backward(o, y, g, stats, w_post, scale, w_pre, do, dn, norm=NORM_RMS, lens=None,
                     dg=None, workspace=None, stream=None):
    """Gradients of f = sum(do o) + sum(dn n) at resnorm_forward_stats's o (its
    x, if that call had no y) and stats.  do or dn may be None.  Returns a dict
    dx, dy, dg, dw_post, dscale, dw_pre (None where the call has no such
    input)."""
    torch = _torch()
    code = _dtype_code(o, "o")
    B, H, L = _resnorm_dims(o, "o")
    dev = o.device
    if not o.is_contiguous():
        raise ValueError("o must be contiguous")
    if y is None and g is not None:
        raise ValueError("a gate needs y")
    if dn is not None and w_pre is None:
        raise ValueError("dn needs w_pre")
    for t, name in ((y, "y"), (do, "do"), (dn, "dn")):
        if t is not None:
            _plain(t, name, o, "o")
    sg = 0 if g is None else _batch_stride(_like(g, "g", o, "o"), "g")
    vec = lambda: _empty((H,), torch.float32, dev, stream)
    out = dict(dx=_new(o, stream), dy=None if y is None else _new(o, stream), dg=None,
               dw_post=None, dscale=None, dw_pre=vec())
    sdg = 0
    if y is not None:
        out["dw_post"], out["dscale"] = vec(), vec()
    if g is not None:
        out["dg"] = _new(o, stream) if dg is None else _like(dg, "dg", o, "o")
        sdg = _batch_stride(out["dg"], "dg")
    elif dg is not None:
        raise ValueError("dg needs g")
    sp = ctypes.byref(ResnormShape(B, H, L, code, int(norm), 0.0))
    ws, nbytes = _buffer(_resnorm_bytes(B, H, L, code, int(norm)), workspace, "workspace", dev,
                         stream)
    gr = ResnormGrads(_ptr(out["dx"]), _ptr(out["dy"]), _ptr(out["dg"]), sdg,
                      _ptr(out["dw_post"]), _ptr(out["dscale"]), _ptr(out["dw_pre"]))
    _launch(lib().dssm_resnorm_backward, dev, stream, o.data_ptr(), _ptr(y), _ptr(g), sg,
            _vec(stats, "stats", (4 if norm == NORM_LAYER else 2) * B * L, dev),
            _resnorm_params(w_post, scale, w_pre, H, dev, y is not None, dn is not None), sp,
            _lens_ptr(lens, B, dev), _ptr(do), _ptr(dn), ctypes.byref(gr), ws.data_ptr(), nbytes)
    return out


class HipEvents:
    """Raw hipEvent_t handles through libamdhip64, for the timing variants
    (plumbing only: create, elapsed time, destroy)."""

    def __init__(self):
        self.h = ctypes.CDLL("libamdhip64.so")
        self.h.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        self.h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                               ctypes.c_void_p]
        self.h.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self.h.hipEventRecord.argtypes = [ctypes.c_void_p, ctypes.c_void_p]

    def create(self, n):
        out = []
        for _ in range(n):
            e = ctypes.c_void_p()
            rc = self.h.hipEventCreate(ctypes.byref(e))
            if rc != 0:
                raise RuntimeError("hipEventCreate failed: %d" % rc)
            out.append(e.value)
        return out

    def ms(self, a, b):
        t = ctypes.c_float()
        rc = self.h.hipEventElapsedTime(ctypes.byref(t), ctypes.c_void_p(a), ctypes.c_void_p(b))
        if rc != 0:
            raise RuntimeError("hipEventElapsedTime failed: %d" % rc)
        return t.value

    def record(self, e, stream):
        rc = self.h.hipEventRecord(ctypes.c_void_p(e), ctypes.c_void_p(stream))
        if rc != 0:
            raise RuntimeError("hipEventRecord failed: %d" % rc)

    def destroy(self, evs):
        for e in evs:
            self.h.hipEventDestroy(ctypes.c_void_p(e))
