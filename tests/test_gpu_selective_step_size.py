"""The step sizes of the selective scan against float64: from no state, with unit drive and
read-out and modes that forget, an output is the step's size."""
import numpy as np
import pytest

from long_convolution_sequence_amd import binding as bd

from seq_cases import np64, say, torch_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lo,hi", [(-1.0, 0.0), (-8.0, -1.0), (-15.0, -8.0), (-30.0, -15.0),
                                   (-80.0, -30.0), (0.0, 8.0), (8.0, 80.0)])
@pytest.mark.parametrize("form", ["short", "tiles", "token"])
def test_step_sizes(lo, hi, form):
    torch = torch_()
    B, H, L = {"short": (60, 1000, 3), "tiles": (4, 200, 300), "token": (180, 1000, 1)}[form]
    say("case: %s v in [%g, %g]" % (form, lo, hi))
    gen = torch.Generator("cuda").manual_seed(7)
    v = torch.rand(B, H, L, device="cuda", generator=gen) * (hi - lo) + lo
    one, bc = torch.ones_like(v), torch.ones(B, 1, 1, L, device="cuda")
    # log_re^2 dt is 2^126 e^-80 > 1500 at least (the square stops at 2^126): every decay is 0, as
    # the reference below takes it to be (at 1e18 it would be e^-18)
    log_re = torch.full((H, 1), 1e19, device="cuda")
    if form == "token":
        x = torch.zeros(B, H, 1, device="cuda")
        y = bd.selective_step(one[..., 0], v[..., 0], bc[..., 0], bc[..., 0], log_re, x)[..., None]
    else:
        y = bd.selective_forward(one, v, bc, bc, log_re)
    x = np64(v)
    ref = np.logaddexp(0.0, x)
    # t = exp(-|v|): the product |v| log2(e) rounded (|v| 2^-24 of t), log2(e) itself (0.23 |v|
    # 2^-24), exp2 (2^-23); the polynomial 2^-24, its last two sums and the last product 3 2^-24.
    # A step above log 2 is v and at most as much again.  Products, sums by 1 and 0 are exact.
    tol = (1.25 * np.abs(x) + 6.0) * 2.0 ** -24
    tol = np.where(x > 0, tol * np.log1p(np.exp(-np.abs(x))) / ref + 2.0 ** -24, tol)
    err = np.abs(np64(y) - ref) / ref
    say("  worst %.2e, of its tolerance %.3f" % (err.max(), (err / tol).max()))
    assert (err <= tol).all()
