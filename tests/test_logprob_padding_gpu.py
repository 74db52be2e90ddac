"""Rows into which no gradient comes (padding without a gradient of the entropy)
send none back, whatever their logits hold."""
import math

import numpy as np
import pytest
import torch

from oracle import readout as ro

F32, BF16 = torch.float32, torch.bfloat16


def test_oracle_of_padding():
    x = np.array([[0.3, np.nan, 1.0], [np.inf, 0.0, 1.0], [-np.inf] * 3, [0.3, 0.2, 0.1]])
    for dH in (None, np.zeros(4)):
        assert not ro.token_logprobs_bwd(x, [-1, 3, -1, 7], 1.0, np.ones(4), dH).any()
    assert np.isnan(ro.token_logprobs_bwd(x, [-1, 3, -1, 7], 1.0, np.ones(4), np.ones(4))[:2]).all()
    assert np.isnan(ro.token_logprobs_bwd(x, [0, 1, 0, 0], 1.0, np.zeros(4))[:2]).all()


# a row by one CTA and by several; rows that are whole vectors and not, in place too
@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [7, 1000, 5003, 40001])
@pytest.mark.parametrize("entropy", [None, 0.0])
@pytest.mark.parametrize("inplace", [False, True])
def test_padding_sends_nothing_back(dt, V, entropy, inplace):
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn(9, V, generator=g, device="cuda").to(dt)
    tok = torch.randint(0, V, (9,), generator=g, device="cuda", dtype=torch.int32)
    tok[2:6] = torch.tensor([-1, V, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    logits[2] = math.nan
    logits[3, V // 2] = math.inf
    logits[4] = -math.inf
    logits[5, V - 1] = math.nan
    logits[6, 0] = math.nan                     # not padding: it has to show
    dl = torch.randn(9, generator=g, device="cuda")
    dl[2] = math.nan                            # (nothing reads it)
    dH = None
    if entropy is not None:
        dH = torch.randn(9, generator=g, device="cuda")
        dH[2:6] = entropy
    kept = logits.double().cpu().numpy()
    dev = runner.LogProbsDevice(logits, tok, dlogprobs=dl, dentropy=dH, dlogits=logits if inplace else None)
    dev.fwd()
    dev.bwd()
    got = dev.dlogits.double().cpu().numpy()
    want = ro.token_logprobs_bwd(kept, tok.cpu().numpy(), 1.0, dl.double().cpu().numpy(),
                                 None if dH is None else dH.double().cpu().numpy())
    assert not got[2:6].any() and np.isnan(got[6]).all()
    rest = [0, 1, 7, 8]
    # (within the rounding to bf16, and 2^-16 of what a row's gradients are made of)
    assert (np.abs(got - want)[rest] <= 2.0 ** -16 * (1 + np.abs(want[rest])) + 2.0 ** -8 * np.abs(want[rest])).all()


@pytest.mark.gpu
def test_entropy_alone_sends_nothing_back_from_rows_without_it():
    from mamba_selective_state_gb300 import runner
    logits = torch.randn(3, 300, device="cuda")
    logits[1, 5] = math.nan
    tok = torch.tensor([1, -1, 2], dtype=torch.int32, device="cuda")
    dev = runner.LogProbsDevice(logits, tok, dentropy=torch.tensor([1.0, 0.0, 1.0], device="cuda"))
    dev.fwd()
    dev.bwd()
    assert not dev.dlogits[1].any() and torch.isfinite(dev.dlogits).all() and dev.dlogits[[0, 2]].any(1).all()
