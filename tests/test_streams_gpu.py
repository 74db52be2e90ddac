"""Calls on a stream that is not the current one (GPU): what they allocate for
their results belongs to the stream that fills it, not to the current one,
whose earlier work may still use a block that it has given back."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def given_back(nbytes):
    """The address of a block that the current stream has just given back: the
    one its allocator hands out next for that size."""
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == at
    del again
    return at


@pytest.mark.parametrize("raw", [False, True])
def test_step_output_is_the_launching_streams(raw):
    from mamba_selective_state_gb300 import runner
    b, T, H, P, N = 3, 2, 4, 64, 32
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda") * 0.3  # noqa: E731
    x = [r(b, T, H, N), r(b, T, H, N), r(b, T, H, P), -r(b, T, H).abs(), r(b, T, H).abs()]
    dev = runner.DeltaStepDevice(r(b, H, P, N))
    want = dev.step(*x, update=False)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    at = given_back(want.numel() * 4)
    y = dev.step(*x, update=False, stream=s.cuda_stream if raw else s)
    s.synchronize()
    assert y.data_ptr() != at
    assert torch.equal(y, want)


@pytest.mark.parametrize("raw", [False, True])
def test_verified_tokens_are_the_launching_streams(raw):
    from mamba_selective_state_gb300 import runner
    b, V = 300, 40
    gen = torch.Generator(device="cuda").manual_seed(0)
    p = torch.softmax(torch.randn(b, 1, V, generator=gen, device="cuda"), -1)
    noise = torch.empty(b, V, device="cuda").exponential_(generator=gen)
    none = torch.empty(b, 0, device="cuda")
    args = (p, None, none.int(), none, noise)
    want, _ = runner.verify_draft(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    at = given_back(b * 4)
    tokens, kept = runner.verify_draft(*args, stream=s.cuda_stream if raw else s)
    s.synchronize()
    assert at not in (tokens.data_ptr(), kept.data_ptr())
    assert torch.equal(tokens, want) and not kept.any()


def test_the_default_stream_by_its_number():
    """0 is the default stream, also where another one is current."""
    from mamba_selective_state_gb300 import runner
    states = torch.ones(1, 1, 4, 8, device="cuda")
    x = [torch.ones(1, 1, 1, n, device="cuda") for n in (8, 8, 4)]
    g = torch.zeros(1, 1, 1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        y = runner.DeltaStepDevice(states).step(*x, g, g, 1.0, stream=0)
        torch.cuda.synchronize()
        assert bool((y == 8).all())
