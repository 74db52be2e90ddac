"""The current stream's handle (CPU, fakes of torch's calls): with and without
torch's unofficial short way to it."""
import types

import pytest
import torch


@pytest.fixture
def lib():
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import _lib
    return _lib


@pytest.mark.parametrize("short", [True, False])
def test_current_stream(lib, monkeypatch, short):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(lib, "_raw_stream", (lambda d: 74 + d) if short else None)
    assert lib._stream(None) == 77


def test_given_streams(lib):
    assert lib._stream(5) == 5
    assert lib._stream(types.SimpleNamespace(cuda_stream=6)) == 6


def test_a_torch_without_the_short_way(monkeypatch):
    """The binding also loads where torch does not have that name."""
    import importlib.util

    from mamba_selective_state_gb300 import _lib
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=78))
    spec = importlib.util.spec_from_file_location(_lib.__name__ + "_again", _lib.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert again._stream(None) == 78
