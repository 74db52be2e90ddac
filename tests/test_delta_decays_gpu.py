"""The gated delta rule where decays are strong and uneven (GPU): the sum of a
chunk's decays is in the thousands, while the tokens behind a strong one differ
by little.  The decay between two tokens keeps its digits all the same; the
tolerances are test_delta_gpu's.  A result below the smallest normal fp32 number
(the gradient of an initial state that has decayed to nothing) has no digits to
compare: it is below that number here too."""
import numpy as np
import pytest
import torch

from tests.test_delta_gpu import TOL, close, device, draw, reference

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16


def check(d):
    dev = device(d)
    dev.fwd()
    dev.bwd()
    assert dev.device_status() == 0
    got, ref = dev.results(), reference(d, d["q"].shape[-1] ** -0.5)
    for n in ref:
        if np.abs(ref[n]).max() < 2.0 ** -126:
            assert np.abs(got[n].numpy()).max() < 2.0 ** -126, n
        else:
            close(got[n].numpy(), ref[n], TOL[d["v"].dtype], n)


def decays(kind, L):
    """(L,) log decays, none of them below the -100 that forgets."""
    t = torch.arange(L)
    if kind == "bursts":            # 24 of every 32 tokens strong
        return torch.where(t % 32 < 24, -16.0, -0.01)
    if kind == "every other":
        return torch.where(t % 2 == 0, -20.0, -0.003)
    if kind == "first":             # a strong run before a long gentle one
        return torch.where(t % 64 < 20, -99.0, -1e-3)
    return torch.where(t % 32 < 31, -99.0, -0.5)    # nearly all


@pytest.mark.parametrize("kind", ["bursts", "every other", "first", "nearly all"])
@pytest.mark.parametrize("P,N,dtype", [(16, 16, F), (40, 56, F), (24, 40, B), (64, 64, B),
                                       (64, 128, B)])
def test_strong_and_uneven_decays(kind, P, N, dtype):
    d = draw(1, 200, 4, P, N, 2, dtype, init=True, dfinal=True)
    d["g"] = decays(kind, 200)[None, :, None].expand(1, 200, 4).contiguous().to(dtype)
    check(d)


@pytest.mark.parametrize("dtype,P,N", [(F, 24, 32), (B, 64, 64)])
def test_strong_decays_in_packed_rows(dtype, P, N):
    d = draw(1, 190, 4, P, N, 2, dtype, nseq=4, init=True, dfinal=True)
    d["g"] = decays("first", 190)[None, :, None].expand(1, 190, 4).contiguous().to(dtype)
    check(d)
