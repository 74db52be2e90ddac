"""The largest scales of the log probabilities: where scale log2(e) is no longer
finite the call is refused (CPU), up to there the answers are the oracle's (GPU)."""
import numpy as np
import pytest
import torch

from oracle import readout as ro

FAKE = 1 << 20
LARGEST = float(np.nextafter(np.float32(float(np.finfo(np.float32).max) / np.log2(np.e)), np.float32(0)))


def test_too_large_scales_are_refused():
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import _lib

    def both(scale):
        p = _lib.make_logprob_problem(4, 100, scale, 0, torch.float32)
        return {_lib.ssd_token_logprobs(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0, check=False),
                _lib.ssd_token_logprobs_bwd(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, stream=0, check=False)}
    for scale in (2.4e38, float(np.finfo(np.float32).max)):
        assert both(scale) == {_lib.SSD_ERR_UNSUPPORTED}, scale
    assert both(float("inf")) == both(0.0) == {_lib.SSD_ERR_INVALID_ARGUMENT}


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_the_largest_scale(dt):
    from mamba_selective_state_gb300 import runner
    x = torch.tensor([[0.0, -1.0, 0.0, -2.0 ** -100], [-2.0 ** -127, -2.0 ** -126, -2.0 ** -125, -1.0],
                      [0.5, 0.25, -4.0, 0.5]]).to(dt).cuda()
    tok = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    dl = torch.ones(3, device="cuda")
    dev = runner.LogProbsDevice(x, tok, scale=LARGEST, ntop=3, dlogprobs=dl, dentropy=dl)
    dev.fwd()
    dev.bwd()
    scale, xs = float(np.float32(LARGEST)), x.double().cpu().numpy()
    want = ro.token_logprobs(xs, tok.cpu().numpy(), scale, 3)
    for name in ("logprobs", "entropy", "lse", "top_logprobs"):
        got = getattr(dev, name).double().cpu().numpy()
        # (a few roundings of sums of four words and of exponents below 8)
        assert np.allclose(got, want[name], rtol=2.0 ** -18, atol=2.0 ** -18), name
    assert np.array_equal(dev.top_tokens.cpu().numpy(), want["top_tokens"])
    # a gradient is scale times at most 2 for each of the two, here below 1.1 in all
    # (a row's gradient does not see what all its logits have in common; the oracle's lse would round the row's sum away)
    grad = ro.token_logprobs_bwd(xs - xs.max(1, keepdims=True), tok.cpu().numpy(), scale, np.ones(3), np.ones(3)) / scale
    got = dev.dlogits.double().cpu().numpy() / scale
    assert np.allclose(got, grad, atol=2.0 ** -7 if dt is torch.bfloat16 else 2.0 ** -18)
