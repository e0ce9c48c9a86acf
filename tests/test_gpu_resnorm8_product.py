"""The norm in 8 bits feeding the product that reads it: q [B, L, H] as it is, as the left operand."""
import numpy as np
import pytest

import oracle
from long_convolution_sequence_amd import binding as bd

from seq_cases import np64, say, torch_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("B,H,L", [(2, 256, 72), (3, 1040, 33), (64, 512, 1)])
def test_product_of_the_norm(B, H, L, form):
    """norm(x + y) w_pre times a matrix in 8 bits: what the bytes stand for times the matrix, and
    within the two roundings to 8 bits of the product itself."""
    torch = torch_()
    say("case: B=%d H=%d L=%d %s" % (B, H, L, form))
    N = 128
    gen = torch.Generator("cuda").manual_seed(H + L)
    shape = (B, H) if L == 1 else (B, H, L)
    x, y = (torch.randn(*shape, device="cuda", generator=gen).bfloat16() for _ in range(2))
    w_pre = 1.0 + 0.2 * torch.randn(H, device="cuda", generator=gen)
    w = torch.randn(N, H, device="cuda", generator=gen) / H ** 0.5
    top = 127.0 if form == "int8" else 448.0
    unit = w.abs().amax(1, keepdim=True) / top
    o, q, qs = bd.resnorm8_forward(x, y, None, None, None, w_pre,
                                   form=bd.Q8_INT8 if form == "int8" else bd.Q8_E4M3)
    rows = q.reshape(-1, H)  # no copy: channels are fastest
    assert rows.data_ptr() == q.data_ptr()
    if form == "int8":
        wq = torch.round(w / unit).to(torch.int8)
        acc = torch._int_mm(rows, wq.t())
        values = np64(rows) @ np64(wq).T
        assert np.array_equal(np64(acc), values)  # whole numbers below 2^24
        got = acc.float() * (qs.reshape(-1, 1) * unit.reshape(1, -1))
    else:
        wq = (w / unit).to(torch.float8_e4m3fn)
        got = torch._scaled_mm(rows, wq.t(), scale_a=qs.reshape(-1, 1), scale_b=unit.reshape(1, -1),
                               out_dtype=torch.bfloat16)
        a, b = np64(rows.float()), np64(wq.float())
        scale = np64(qs).reshape(-1, 1) * np64(unit).reshape(1, -1)
        values, size = (a @ b.T) * scale, (np.abs(a) @ np.abs(b).T) * scale
        # sums of H terms in float32, the result rounded to bfloat16
        tol = H * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(values) * (1 + 2.0 ** -8)
        assert (np.abs(np64(got) - values) <= tol + H * 2.0 ** -24 * size).all()
    n = oracle.resnorm_out(np64(o).reshape(B, H, L), np64(w_pre), False, 1e-6)
    n = n.transpose(0, 2, 1).reshape(-1, H)
    ref = n @ np64(w).T
    # each operand off by half a step: of its row's largest (whole numbers), or of itself and of
    # 2^-9 of a unit (e4m3's smallest step is 2^-9 of its unit)
    if form == "int8":
        da = 0.5 * np64(qs).reshape(-1, 1) * np.ones_like(n)
        db = 0.5 * np64(unit) * np.ones((N, H))
    else:
        da = np.abs(n) * 2.0 ** -4 + 2.0 ** -10 * np64(qs).reshape(-1, 1)
        db = np.abs(np64(w)) * 2.0 ** -4 + 2.0 ** -10 * np64(unit)
    bound = da @ np.abs(np64(w)).T + (np.abs(n) + da) @ db.T
    err = np.abs(np64(got) - ref)
    say("  error / bound %.3f, relative error %.1e" % ((err / bound).max(),
                                                       np.linalg.norm(err) / np.linalg.norm(ref)))
    assert (err <= bound + 2.0 ** -8 * np.abs(ref) + (H + 40) * 2.0 ** -23 * (np.abs(n) @ np.abs(np64(w)).T)).all()
