"""The recurrent step and decays that forget (GPU): -inf, or below -100, hides
what a slot holds, as in the chunked forms, also where that is not finite."""
import pytest
import torch

from oracle import delta as od
from tests.test_delta_gpu import TOL, close, draw, f64

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T", [1, 2, 4, 7])
@pytest.mark.parametrize("dtype,P,N", [(F, 40, 57), (B, 64, 128), (F, 16, 256)])
@pytest.mark.parametrize("g", [-float("inf"), -101.0, -3e38])
def test_a_slot_of_nan_is_forgotten(T, dtype, P, N, g):
    from mamba_selective_state_gb300 import runner
    b, H = 3, 2
    d = draw(b, T, H, P, N, 1, dtype, seed=T, init=True, state_dtype=F)
    d["g"][1, 0] = g                                # the first token of sequence 1
    if T > 4:
        d["g"][2, 4] = g                            # in the second stage of tokens
    x = [d[n].cuda() for n in ("q", "k", "v", "g", "beta")]
    pool = d["init"].cuda()
    pool[1] = float("nan")
    pool[1, :, 0] = float("inf")
    dev = runner.DeltaStepDevice(pool)
    y = dev.step(*x)
    args = [f64(d[n]) for n in ("q", "k", "v", "g", "beta")]
    want, fin = od.delta_fwd(*args, N ** -0.5, f64(d["init"]))
    close(y.double().cpu().numpy(), want, TOL[dtype], "y")
    close(dev.states.double().cpu().numpy(), fin, TOL[F], "states")


def test_the_strongest_decay_that_does_not_forget():
    """At -100 the state still counts: an infinite one stays, as by definition."""
    from mamba_selective_state_gb300 import runner
    d = draw(1, 1, 1, 8, 16, 1, F, init=True)
    d["g"][:] = -100.0
    pool = torch.full_like(d["init"], float("inf")).cuda()
    dev = runner.DeltaStepDevice(pool)
    y = dev.step(*[d[n].cuda() for n in ("q", "k", "v", "g", "beta")])
    assert not torch.isfinite(y).any() and not torch.isfinite(dev.states).any()
