"""One token of the selective scan for so many rows that a lane takes two batch rows."""
import numpy as np
import pytest

from long_convolution_sequence_amd import binding as bd

import oracle
from selective_cases import c_selective, selective_inputs
from seq_cases import close, np64, say, torch_

pytestmark = pytest.mark.gpu


# at least 2^20 lanes of four modes: odd batches, whose last lane has one row; channels that end
# inside a workgroup; modes that end inside a lane's four (states not aligned); 32 lanes to a row
@pytest.mark.parametrize("B,H,N,G,dtype,what", [
    (257, 1024, 16, 1, "f32", "gsbr"), (257, 1030, 15, 2, "bf16", "gsbr"),
    (301, 111, 128, 3, "f16", "gbr"), (2049, 130, 13, 2, "bf16", "gsb"),
    (1025, 1025, 3, 1, "f16", "sr"), (133, 4001, 5, 1, "f32", "gr"),
    (66000, 17, 1, 17, "bf16", "gsbr")])
@pytest.mark.parametrize("in_place", [True, False])
def test_two_batch_rows_to_a_lane(B, H, N, G, dtype, what, in_place):
    torch = torch_()
    say("case: B=%d H=%d N=%d G=%d %s %s in_place=%d" % (B, H, N, G, dtype, what, in_place))
    lanes = 1
    while 4 * lanes < N:
        lanes *= 2
    assert B * H * lanes >= 1 << 20
    s = selective_inputs(B, H, N, G, 1, dtype, seed=B + H + N, gate="g" in what, skip="s" in what,
                         bias="b" in what)
    if "r" in what:  # pairs with both rows live, one of them and none
        s["lens"] = torch.from_numpy(np.random.default_rng(B).integers(-1, 3, B).astype(np.int32)).cuda()
        s["lens"][:6] = torch.tensor([1, 0, 0, 1, 0, -1], dtype=torch.int32)
        s["lens"][-1] = 1
        idle = s["lens"] <= 0
        for k in ("u", "delta", "z", "Bm", "Cm"):
            if s[k] is not None:
                s[k][idle] = float("nan")
    flat = [s[k][..., 0].contiguous() for k in ("u", "delta", "Bm", "Cm")]
    prm = dict(D=s["D"], dt_bias=s["dt_bias"], lens=s["lens"],
               z=None if s["z"] is None else s["z"][..., 0].contiguous())
    x = s["x0"].clone()
    xo = x if in_place else torch.full_like(x, float("nan"))
    y = bd.selective_step(*flat, s["log_re"], x, x_out=None if in_place else xo, **prm)
    if not in_place:
        assert torch.equal(x, s["x0"])
    live = np.ones(B, bool) if s["lens"] is None else (s["lens"] > 0).cpu().numpy()
    # a few hundred rows against the oracle, pairs' both sides and the last one among them
    pick = sorted(set(range(min(B, 120))) | {B - 2, B - 1} | set(range(B // 2, B // 2 + 60)))
    a = [np.nan_to_num(np64(s[k][pick])) for k in ("u", "delta", "Bm", "Cm")] + [np64(s["log_re"])]
    kw = {k: None if s[k] is None else np64(s[k]) for k in ("D", "dt_bias")}
    kw.update(x0=np64(s["x0"][pick]), z=None if s["z"] is None else np.nan_to_num(np64(s["z"][pick])),
              lens=live[pick].astype(np.int32))
    ref, end = oracle.selective_scan(*a, **kw)
    mag, mend = oracle.selective_scan(*a, magnitude=True, **kw)
    close(y[pick], ref[..., 0], mag[..., 0], c_selective(N, 1), dtype, "y")
    close(xo[pick], end, mend, c_selective(N, 1), "f32", "state")
    idle = torch.from_numpy(~live).cuda()
    assert torch.equal(xo[idle], s["x0"][idle]) and not y[idle].any()
    # every row against the kernel of one row to a lane, on parts of the batch
    part = max(1, ((1 << 20) - 1) // (H * lanes))
    cut = lambda t, lo: None if t is None else t[lo:lo + part].contiguous()
    for lo in range(0, B, part):
        xs = cut(s["x0"], lo)
        ys = bd.selective_step(*[cut(t, lo) for t in flat], s["log_re"], xs, D=prm["D"],
                               dt_bias=prm["dt_bias"], z=cut(prm["z"], lo), lens=cut(prm["lens"], lo))
        assert torch.equal(ys, y[lo:lo + part]) and torch.equal(xs, xo[lo:lo + part]), lo
