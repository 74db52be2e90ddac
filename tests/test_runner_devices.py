"""The delta-rule, verification and state-cache wrappers take tensors of the
current CUDA device only (CPU: they refuse before any call into the library,
which would launch kernels on whatever address it gets)."""
import pytest
import torch

F = torch.float32


@pytest.fixture
def runner(monkeypatch):
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import _lib, runner

    def refuse(*a, **kw):
        raise AssertionError("reached the library")
    for name in ("ssd_delta_fwd", "ssd_delta_bwd", "ssd_delta_step", "ssd_verify_draft",
                 "ssd_state_cache_store", "ssd_state_cache_load"):
        monkeypatch.setattr(_lib, name, refuse)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return runner


def tokens(b=1, L=4, H=4, P=16, N=8, G=2, device="cpu"):
    z = lambda *s: torch.zeros(s, device=device)  # noqa: E731
    return z(b, L, G, N), z(b, L, G, N), z(b, L, H, P), z(b, L, H), z(b, L, H)


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_host_tensors_are_refused(runner, device):
    z = lambda *s, dtype=F: torch.zeros(s, dtype=dtype, device=device)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        runner.DeltaDevice(*tokens(device=device)).fwd()
    with pytest.raises(ValueError, match="CUDA"):
        runner.DeltaStepDevice(z(1, 4, 16, 8)).step(*tokens(device=device))
    with pytest.raises(ValueError, match="CUDA"):
        runner.verify_draft(z(1, 3, 9), z(1, 2, 9), z(1, 2, dtype=torch.int32), z(1, 2), z(1, 9))
    with pytest.raises(ValueError, match="CUDA"):
        runner.StateCache(1, 4, 16, 8, device=device).store(z(1, 4, 16, 8))


@pytest.mark.parametrize("device,fits", [("cuda:0", True), ("cuda:1", False), ("cpu", False)])
def test_only_the_current_device(runner, device, fits):
    if fits:
        runner._on_gpu(torch.device(device), "x")
    else:
        with pytest.raises(ValueError, match="current CUDA device"):
            runner._on_gpu(torch.device(device), "x")


def test_the_current_device_may_have_changed_since(runner, monkeypatch):
    """An object built on one device and called with another one current."""
    dev = runner.DeltaDevice.__new__(runner.DeltaDevice)
    dev.v, dev.saved = type("T", (), {"device": torch.device("cuda:0")}), True
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (dev.fwd, dev.bwd):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
