"""The gated-MLP calls' way to the current stream and device (nothing is launched)."""
import contextlib
import types

import pytest
import torch

import fp8_fine_grained_x1_b200 as fg


@pytest.fixture
def no_short_forms(monkeypatch):
    """A torch without the private short forms."""
    monkeypatch.setattr(fg, "_queries", None)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    return entered


def test_public_functions_do_where_torch_lacks_the_short_ones(no_short_forms):
    calls = []

    def call(*a):
        calls.append(a)
        return fg.FP8_OK
    fg._call_on(0, None, call, "x", "a")
    assert calls == [("a", 1000)] and not no_short_forms
    fg._call_on(1, None, call, "x", "b")                       # not the current device: made so for the call
    assert calls[1:] == [("b", 1001)] and no_short_forms == [1]


def test_a_stream_of_another_device_is_refused(no_short_forms):
    stream = types.SimpleNamespace(device_index=1, cuda_stream=7)
    with pytest.raises(ValueError, match="cuda:1"):
        fg._call_on(0, stream, lambda *a: fg.FP8_OK, "x")
    with pytest.raises(fg.Fp8Error):
        fg._call_on(1, stream, lambda raw: fg.FP8_ERR_SHAPE, "x")
