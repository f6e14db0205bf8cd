"""GatedMlpStep on the host: which stream its gradient buffers belong to, and
when it counts as having run forward.  The library calls and torch's streams are
stand-ins; nothing is launched."""
import contextlib

import pytest
import torch

from fp8_fine_grained_x1_b200 import linear

CALLS = [n for n in dir(linear) if n.startswith("fp8_") and not n.endswith("_bytes")]


class _Fork:
    def __init__(self, device):
        pass

    def begin(self, stream):
        return stream, "side"

    def end(self, cur):
        pass


@pytest.fixture
def step(monkeypatch):
    """A step over CPU tensors, and a list of (shape, stream) of what it allocates."""
    for name in CALLS:
        monkeypatch.setattr(linear, name, lambda *a, **k: None)
    monkeypatch.setattr(linear, "_Fork", _Fork)
    now, seen, empty = ["caller's"], [], torch.empty

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    def allocate(shape, **k):
        seen.append((tuple(shape), now[-1]))
        return empty(shape, **k)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.cuda, "stream", use)
    step = linear.GatedMlpStep(torch.zeros((128, 256)), torch.zeros((512, 256)), torch.zeros((384, 256)))
    seen.clear()
    return step, seen


def test_gradient_buffers_belong_to_the_stream_that_first_uses_them(step):
    step, seen = step
    step("main")
    dy = torch.zeros((128, 384))
    step.backward(dy, "main")
    assert seen and all(stream == "main" for _, stream in seen)
    seen.clear()
    step.backward(dy, "main")
    assert not seen                    # kept from call to call


def test_a_forward_pass_that_failed_does_not_count(step, monkeypatch):
    step, _ = step

    def refuse(*a, **k):
        raise RuntimeError("refused")
    monkeypatch.setattr(linear, "fp8_quant_w_128x128", refuse)
    with pytest.raises(RuntimeError, match="refused"):
        step("main")
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(torch.zeros((128, 384)), "main")


def test_a_later_forward_pass_that_failed_takes_the_earlier_one_back(step, monkeypatch):
    """It may have overwritten a part of what backward needs."""
    step, _ = step
    step("main")

    def refuse(*a, **k):
        raise RuntimeError("refused")
    monkeypatch.setattr(linear, "fp8_swiglu_quant", refuse)
    with pytest.raises(RuntimeError, match="refused"):
        step("main")
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(torch.zeros((128, 384)), "main")
