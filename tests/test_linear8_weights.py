"""Linear8.from_weight takes weights however they lie in memory, and refuses what
is not a matrix (the rounding on the CPU, with the checks of the device passed over)."""
import pytest
import torch


@pytest.fixture
def linear8(monkeypatch):
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import runner
    monkeypatch.setattr(runner, "_on_gpu", lambda device, what: None)
    return runner.Linear8


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_weights_that_are_not_dense(linear8, form):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(20, 33, generator=g)
    want = linear8.from_weight(w, form)
    wide = torch.full((20, 50), 9.0)
    wide[:, 10:43] = w
    for other in (w.t().contiguous().t(), wide[:, 10:43], w.flip(0).flip(0), w.repeat_interleave(2, 1)[:, ::2],
                  torch.nn.Parameter(w.t().contiguous().t())):
        lin = linear8.from_weight(other, form)
        assert lin.codes.is_contiguous() and torch.equal(lin.codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(lin.scales, want.scales) and not lin.scales.requires_grad


def test_refusals(linear8):
    for bad in (torch.randn(4), torch.randn(2, 3, 4), torch.zeros(3, 0), torch.zeros(0, 3)):
        with pytest.raises(ValueError):
            linear8.from_weight(bad)
