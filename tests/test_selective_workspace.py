"""How the selective scan's workspace grows (host side; no kernel is launched)."""
import ctypes

import pytest

from long_convolution_sequence_amd import binding as bd


def size(fn, *args):
    out = ctypes.c_size_t(0)
    assert fn(*args, ctypes.byref(out)) == bd.DSSM_OK, bd.lib().dssm_last_error()
    return out.value


# few modes and many, one tile and many, split rows and whole ones, groups of one channel
@pytest.mark.parametrize("B,H,G,N,L", [
    (1, 1, 1, 1, 1), (3, 130, 2, 13, 1001), (4, 2048, 1, 16, 4096), (8, 4096, 1, 128, 8192),
    (8, 8192, 1, 128, 4096), (1, 128, 1, 128, 1 << 20), (1, 16, 1, 1, 1 << 24),
    (2, 1040, 1, 128, 16513), (1, 1024, 1, 128, 33000), (5600, 48, 1, 128, 129),
    (8400, 40, 2, 127, 40),
    (2, 16400, 16400, 128, 1), (1, 65535, 65535, 128, 300), (1 << 17, 128, 1, 128, 128)])
def test_bounded_by_two_gibibytes_and_the_checkpoint(B, H, G, N, L):
    L_ = bd.lib()
    s = ctypes.byref(bd.SelectiveShape(B, H, L, N, G, bd.BF16))
    keep = size(L_.dssm_selective_ckpt_size, s)
    assert size(L_.dssm_selective_workspace_size, s, 0) <= 2 * keep
    assert size(L_.dssm_selective_workspace_size, s, 1) <= (1 << 31) + 6 * keep
