"""Logits farther apart than fp32's largest value (GPU), and the scales below which
such words would still weigh in the sums (refused, CPU)."""
import numpy as np
import pytest
import torch

from oracle import readout as ro

FAKE = 1 << 20
LEAST = 2.0 ** -120


def test_too_small_scales_are_refused():
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import _lib

    def both(scale):
        p = _lib.make_logprob_problem(4, 100, scale, 0, torch.float32)
        return {_lib.ssd_token_logprobs(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0, check=False),
                _lib.ssd_token_logprobs_bwd(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, stream=0, check=False)}
    for scale in (LEAST * (1 - 2.0 ** -24), 1e-38, 2.0 ** -149):
        assert both(scale) == {_lib.SSD_ERR_UNSUPPORTED}, scale


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 700, 20003])
@pytest.mark.parametrize("scale", [0.25, 2.0 ** -30, LEAST])
def test_far_apart(dt, V, scale):
    from mamba_selective_state_gb300 import runner
    big = torch.finfo(dt).max
    x = torch.full((4, V), -big, dtype=dt)
    x[:, V // 2] = big
    x[1, 3] = 0.75 * big
    x[2, [0, V - 1]] = big
    x[3] = torch.linspace(-big / 2, big / 2, V, dtype=torch.float64).to(dt) * 2
    tok = torch.tensor([1, 3, 4, 0], dtype=torch.int32)
    dl, dH = torch.tensor([1.0, -2.0, 0.5, 1.0]), torch.tensor([0.5, 1.0, -1.0, 0.25])
    dev = runner.LogProbsDevice(x.cuda(), tok.cuda(), scale=scale, ntop=3, dlogprobs=dl.cuda(), dentropy=dH.cuda())
    dev.fwd()
    dev.bwd()
    xs = x.double().numpy()
    want = ro.token_logprobs(xs, tok.numpy(), scale, 3)
    assert np.array_equal(dev.top_tokens.cpu().numpy(), want["top_tokens"])
    with np.errstate(over="ignore"):
        for name in ("logprobs", "lse", "entropy", "top_logprobs"):
            got, w = getattr(dev, name).cpu().numpy(), want[name].astype(np.float32)
            # the difference, its product, the sum's logarithm (V / 256 + 96 roundings of it) and its subtraction
            assert np.array_equal(np.isinf(got), np.isinf(w)), name
            fine = np.isfinite(w)
            tol = (V / 256 + 96) * 2.0 ** -24 + 6 * 2.0 ** -24 * np.abs(w[fine].astype(np.float64))
            # a word a few hundred below the largest: its exponent's roundings weigh it by 2^-24 of that each
            assert (np.abs(got[fine].astype(np.float64) - w[fine]) <= tol + 2.0 ** -24 * 600).all(), name
    assert np.isfinite(dev.logprobs.cpu().numpy()).all()
    assert torch.isfinite(dev.dlogits).all()
