"""The sums over steps of the selective scan's parameter gradients: rows of many steps whose last
ones are large and whose others a float32 sum of those would drop."""
import pytest

from long_convolution_sequence_amd import binding as bd

from seq_cases import say, torch_

pytestmark = pytest.mark.gpu

# 130 workgroups: whole rows, a tile of 128 steps after the other from the end
B, H, L, LAST = 2, 1040, 24576, 128


def ones(*n):
    return torch_().ones(*n, device="cuda")


def test_skip_and_bias():
    """dD = sum dy u and ddt_bias = sum of the steps' gradients, of one mode that forgets all."""
    torch = torch_()
    small = 2e-7
    dy = torch.full((B, H, L), small, device="cuda")
    dy[..., L - LAST:] = 1.0
    u, bc = ones(B, H, L), ones(B, 1, 1, L)
    five = [u, torch.zeros_like(u), bc, bc, torch.full((H, 1), 1e19, device="cuda")]
    prm = dict(D=torch.zeros(H, device="cuda"), dt_bias=torch.zeros(H, device="cuda"))
    y, ckpt = bd.selective_forward_ckpt(*five, **prm)
    g = bd.selective_backward(dy, ckpt, *five, **prm)
    ref = B * (LAST + (L - LAST) * float(dy[0, 0, 0]))
    # a step's gradient: C dy B u sigmoid(0); four steps, 16 tiles and five joins in float32, the
    # part and the result rounded, the sigmoid two more
    for name, r in (("dD", ref), ("ddt_bias", ref / 2)):
        err = float((g[name].double() - r).abs().max()) / r
        say("  %-8s error %.2e" % (name, err))
        assert err <= (3 + 16 + 5 + 2 + 2) * 2.0 ** -24, name


def test_decays():
    """dlog_re = -2 log_re sum w dt, w = dx exp(-log_re^2 sum dt) x0 at every step without drive."""
    torch = torch_()
    delta = torch.full((B, H, L), -17.4, device="cuda")
    delta[..., L - LAST:] = 0.5
    zero, bc = torch.zeros(B, H, L, device="cuda"), torch.zeros(B, 1, 1, L, device="cuda")
    five = [zero, delta, bc, bc, torch.full((H, 1), 1e-3, device="cuda")]
    x0 = ones(B, H, 1)
    y, ckpt = bd.selective_forward_ckpt(*five, x=x0, x_out=torch.empty_like(x0))
    g = bd.selective_backward(zero, ckpt, *five, dx=x0)
    lr = float(five[4][0, 0])
    dt = torch.nn.functional.softplus(delta[0, 0].double(), threshold=100.0)
    total = float(dt.sum())
    ref = -2.0 * lr * B * total * float(torch.exp(torch.tensor(-lr * lr * total).double()))
    err = float((g["dlog_re"].double() - ref).abs().max()) / abs(ref)
    say("  dlog_re  error %.2e" % err)
    # the large steps' size (1.25 / 2 + 6), their decays (next to 1: half a step each, of which the
    # tiles' joins use none and the 8 of a lane all, in both directions 16), products 3, the lane's
    # eight, four joins and 16 tiles, the part and the result
    assert err <= (7 + 16 + 3 + 8 + 4 + 16 + 2) * 2.0 ** -24
