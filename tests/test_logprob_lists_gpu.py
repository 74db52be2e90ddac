"""Alternatives from lists of 97 to 512 words, which are shortened before they are
sorted (GPU): many rows, many times, so that the CTAs' warps meet in many orders."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def tops(logits, ntop):
    """The largest first, equal ones by their index."""
    return (logits.float() + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :ntop].int()


# few words to a row: fewer than ntop of the groups of threads have any, so that all are listed (one CTA to a row, of 64
# threads; of 128; clusters); and rows with 97 to 512 words that are equal and the largest
LISTS = [(4096, 130, 32, 0), (4096, 200, 32, 0), (4096, 300, 32, 0), (2000, 5003, 20, 97), (2000, 5003, 20, 300),
         (1000, 40001, 20, 511), (60, 5003, 32, 300), (3, 100003, 5, 2000)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,V,ntop,equal", LISTS)
def test_lists_that_are_shortened(rows, V, ntop, equal, dt):
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(rows + V + equal)
    logits = (3 * torch.randn(rows, V, generator=g, device="cuda")).to(dt)
    if equal:
        at = torch.rand(rows, V, generator=g, device="cuda").argsort(1)[:, :equal]
        logits.scatter_(1, at, 20.0)
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    want = tops(logits, ntop)
    dev = runner.LogProbsDevice(logits, tok, ntop=ntop)
    first = None
    for _ in range(30):
        dev.top_tokens.fill_(-7)
        dev.fwd()
        assert torch.equal(dev.top_tokens, want)
        got = [t.clone() for t in (dev.logprobs, dev.entropy, dev.lse, dev.top_logprobs)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    lp = torch.log_softmax(logits.double(), -1).gather(1, want.long())
    # lse and the difference in fp32: V / 256 + 100 roundings of the sum, 4 of values below 64
    assert float((dev.top_logprobs.double() - lp).abs().max()) <= (V / 256 + 100 + 4 * 64) * 2.0 ** -24
