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


def _bytes(*steps):
    """Bytes that the steps hold in tensors of their own (not their inputs), each storage counted once."""
    seen = {}
    for s in steps:
        own = [v for v in vars(s).values() if torch.is_tensor(v)] + [v for v in (s._grad or {}).values()]
        inputs = {t.data_ptr() for t in s.inputs}
        seen.update({t.data_ptr(): t.numel() * t.element_size() for t in own if t.data_ptr() not in inputs})
    return sum(seen.values())


def test_steps_share_their_scratch(step):
    """A further layer adds what it has to keep (FP8 checkpoints, FP8 weights) and hand out (Y and the gradients)."""
    first, _ = step
    M, K, I, N = 128, 256, 256, 384
    dy = torch.zeros((M, N))
    second = linear.GatedMlpStep(torch.zeros((M, K)), torch.zeros((2 * I, K)), torch.zeros((N, I)), share=first)
    third = linear.GatedMlpStep(torch.zeros((M, K)), torch.zeros((2 * I, K)), torch.zeros((N, I)), share=second)
    for s in (first, second, third):
        s("main")
    for s in (third, first, second):
        s.backward(dy, "main")
    keep = M * (K + 2 * I) + 4 * M * (K + 2 * I) // 128
    weights = (2 * I * K + N * I) + 4 * (2 * I * K + N * I) // 128 ** 2
    hand_out = 2 * M * N + 2 * M * K + 4 * (2 * I * K + N * I)
    assert _bytes(first, second, third) - _bytes(first, second) == keep + weights + hand_out
    for other in (torch.zeros((256, K)), None):
        with pytest.raises(ValueError, match="share"):
            if other is not None:
                linear.GatedMlpStep(other, torch.zeros((2 * I, K)), torch.zeros((N, I)), share=first)
            else:
                linear.GatedMlpStep(torch.zeros((M, K)), torch.zeros((2 * I, K)), torch.zeros((N + 128, I)), share=first)


@pytest.mark.gpu
def test_layers_that_share_give_the_bits_of_layers_that_do_not():
    from fp8_fine_grained_x1_b200 import synth
    d = torch.device("cuda", 0)
    M, K, I = 256, 256, 384
    w = [(synth.normal((2 * I, K), K ** -0.5, 2 + i).to(d), synth.normal((K, I), I ** -0.5, 7 + i).to(d)) for i in range(3)]
    dy = synth.normal((M, K), 1e-3, 4).to(d)
    results = []
    for shared in (False, True):
        x, steps = synth.activations(M, K, seed=1).to(d), []
        for w13, w2 in w:
            steps.append(linear.GatedMlpStep(x, w13, w2, share=steps[0] if shared and steps else None))
            x = steps[-1]()
        g, out = dy, [x.clone()]
        for s in reversed(steps):
            g, dw13, dw2 = s.backward(g)
            out += [g.clone(), dw13.clone(), dw2.clone()]
        results.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*results))
