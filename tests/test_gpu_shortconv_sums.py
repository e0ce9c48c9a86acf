"""The sums over steps of the short convolution's weight gradients."""
import pytest

from long_convolution_sequence_amd import binding as bd

from seq_cases import say, torch_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,L,dtype", [(8, 1024, 8191, "bf16"), (2, 128, 1 << 18, "bf16"),
                                         (4, 2048, 4096, "f32")])
def test_small_terms_are_not_lost_in_long_rows(B, H, L, dtype):
    """A few hundred steps of size 1, then thousands that a float32 sum of those would drop."""
    torch = torch_()
    say("case: B=%d H=%d L=%d %s" % (B, H, L, dtype))
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    dy = torch.full((B, H, L), 4e-7, device="cuda").to(dt)
    dy[:, :, :504] = 1.0
    u = torch.ones(B, H, L, dtype=dt, device="cuda")
    g = bd.shortconv_backward(dy, u, torch.ones(H, 4, device="cuda"), torch.zeros(H, device="cuda"),
                              act=bd.ACT_NONE)
    small = float(dy[0, 0, -1])
    # tap 3 - k meets all steps but the first k
    for got, k in [(g["dw"][:, 3 - k], k) for k in range(4)] + [(g["dbias"], 0)]:
        ref = B * (504 - k + (L - 504) * small)
        err = float((got.double() - ref).abs().max()) / ref
        say("  k=%d error %.2e" % (k, err))
        # eight terms added up in float32, a row's sum and the result rounded to it
        assert err <= 10 * 2.0 ** -24
