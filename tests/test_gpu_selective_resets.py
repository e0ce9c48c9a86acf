"""Resets in the selective scan: steps of up to 2^127, which forget what was before them, side by
side, so that their sum is past float32."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from selective_cases import c_selective, c_selective_back, selective_inputs
from seq_cases import close, np64, say, torch_

pytestmark = pytest.mark.gpu

GRADS = ("du", "ddelta", "dz", "dB", "dC", "dlog_re", "dD", "ddt_bias", "dx0")


# modes that fill a wave's pairs and that do not; channels that fill a workgroup's rows and that do
# not; lanes of 4 and of 8 steps, rows in segments, rows enough to stay whole
@pytest.mark.parametrize("B,H,N,G,L,dtype", [
    (2, 17, 5, 1, 40, "f32"), (2, 32, 16, 1, 64, "bf16"), (2, 17, 5, 1, 300, "bf16"),
    (2, 16, 16, 1, 300, "f32"), (3, 10, 3, 2, 257, "f32"), (2, 17, 5, 1, 5000, "f32"),
    (1, 16, 8, 1, 5000, "bf16"), (140, 17, 2, 1, 600, "bf16")])
@pytest.mark.parametrize("keeps", [False, True])
def test_resets_side_by_side(B, H, N, G, L, dtype, keeps):
    """keeps: one mode's log_re is 0, which no step makes forget."""
    torch = torch_()
    say("case: B=%d H=%d N=%d G=%d L=%d %s keeps=%d" % (B, H, N, G, L, dtype, keeps))
    s = selective_inputs(B, H, N, G, L, dtype, seed=B + H + N + L)
    s["log_re"].copy_(torch.where(s["log_re"].abs() < 0.1, 0.1, s["log_re"]))
    if keeps:
        s["log_re"][:, N // 2] = 0.0
    for t in (4, 5, 16, 17, 18, L // 16 * 8, L // 16 * 8 + 1, L - 1):
        s["delta"][..., t] = 2.0 ** 127
        s["u"][..., t] = 0.0   # no drive: dt B u of such a step is past every type
        s["Bm"][..., t] = 0.0  # nor a gradient of its input, dt sum G B
    five = [s[k] for k in ("u", "delta", "Bm", "Cm", "log_re")]
    o = {k: s[k] for k in ("D", "dt_bias", "z")}
    xo = torch.empty_like(s["x0"])
    y, ckpt = bd.selective_forward_ckpt(*five, x=s["x0"], x_out=xo, **o)
    a, kw = [np64(t) for t in five], {k: np64(t) for k, t in o.items()}
    kw["x0"] = np64(s["x0"])
    ref, end = oracle.selective_scan(*a, **kw)
    mag, mend = oracle.selective_scan(*a, magnitude=True, **kw)
    close(y, ref, mag, c_selective(N, L), dtype, "y")
    close(xo, end, mend, c_selective(N, L), "f32", "state")
    got = bd.selective_backward(s["dy"], ckpt, *five, dx=s["dx"], **o)
    ref = oracle.selective_backward(*a, np64(s["dy"]), dx=np64(s["dx"]), **kw)
    mag = oracle.selective_backward(*a, np64(s["dy"]), dx=np64(s["dx"]), magnitude=True, **kw)
    for n in GRADS:
        t = "f32" if n in ("dlog_re", "dD", "ddt_bias", "dx0") else dtype
        close(got[n], ref[n], mag[n], c_selective_back(H, N, L), t, n)
