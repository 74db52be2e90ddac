"""The gradient of a given token whose own logit is -inf."""
import math

import numpy as np
import pytest
import torch

from oracle import readout as ro

F32, BF16 = torch.float32, torch.bfloat16


def test_oracle_of_an_excluded_token():
    """Its gradient is the limit of that of an ever less likely one."""
    x = np.array([[0.3, -1.0, -80.0, 2.0]])
    near = ro.token_logprobs_bwd(x, [2], 1.5, [0.7], [-0.2])
    x[0, 2] = -np.inf
    at = ro.token_logprobs_bwd(x, [2], 1.5, [0.7], [-0.2])
    assert np.allclose(near, at, rtol=0, atol=1e-30) and at[0, 2] == 1.5 * 0.7


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [5, 5003])
def test_a_given_token_that_is_excluded(dt, V):
    """Its log probability is -inf; its gradient is the formula's scale * dlogprob,
    every other excluded word's 0."""
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn(4, V, generator=g, device="cuda").to(dt)
    logits[:, ::2] = -math.inf
    at = [0, V // 4 * 2, V - 1, 2]
    tok = torch.tensor(at, dtype=torch.int32, device="cuda")
    dl, dH = torch.randn(4, generator=g, device="cuda"), torch.randn(4, generator=g, device="cuda")
    dev = runner.LogProbsDevice(logits, tok, scale=1.5, dlogprobs=dl, dentropy=dH)
    dev.fwd()
    dev.bwd()
    assert (dev.logprobs == -math.inf).all()
    got = dev.dlogits.double().cpu().numpy()
    want = ro.token_logprobs_bwd(logits.double().cpu().numpy(), tok.cpu().numpy(), 1.5, dl.double().cpu().numpy(),
                                 dH.double().cpu().numpy())
    own = got[range(4), at]
    assert np.allclose(own, 1.5 * dl.double().cpu().numpy(), rtol=2.0 ** -8 if dt is BF16 else 2.0 ** -23)
    got[range(4), at] = 0
    assert not got[:, ::2].any()
    want[range(4), at] = 0
    assert (np.abs(got - want) <= 2.0 ** -16 * (1 + np.abs(want)) + 2.0 ** -8 * np.abs(want)).all()
