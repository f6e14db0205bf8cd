"""The allocating forms with a `stream`: what they allocate has to belong to that
stream, or the allocator may hand a block to another stream that this one still
uses (a scratch block freed on return, an output whose memory the current
stream's earlier work still reads).

On the CPU the calls run against stand-ins for torch's allocator and streams
and for the library calls, and every allocation is looked at; on a GPU they run
on a side stream while the current stream allocates and fills blocks of the same
sizes at once, and have to give the bits of an undisturbed call.
"""
import contextlib

import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import build as fgbuild
from fp8_fine_grained_x1_b200 import synth

U8, F32, BF, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def _inputs(device, seed=0):
    """Operands of every allocating form (T = 40 tokens, or 128 where groups run along tokens)."""
    rng = np.random.default_rng(seed)

    def codes(*shape):
        return torch.from_numpy(synth.random_e4m3_codes(shape, seed)).to(device)

    def scales(*shape):
        return torch.from_numpy(synth.random_scales(shape, seed)).to(device)

    x = torch.from_numpy(rng.normal(0, 1, (128, 256)).astype(np.float32)).to(torch.bfloat16).to(device)
    topk = torch.from_numpy(rng.integers(0, 4, (40, 2)).astype(np.int32)).to(device)
    w = torch.from_numpy(rng.uniform(0.1, 1, (40, 2)).astype(np.float32)).to(device)
    offsets = torch.tensor([0, 128, 128, 256, 384], dtype=I32, device=device)
    q, s = codes(128, 256), scales(2, 128)
    return {
        "quant_act_1x128": (x,), "quant_act_128x1": (x,), "quant_w_128x128": (x,),
        "requant_1x128_to_128x1": (q, s),
        "gemm": (q, s, codes(128, 256), scales(1, 2)),
        "grouped_gemm": (codes(384, 256), scales(2, 384), codes(4, 128, 256), scales(4, 1, 2), offsets),
        "moe_dispatch": (q[:40].contiguous(), s[:, :40].contiguous(), topk, 4),
        "swiglu_quant": (x,),
        "swiglu_bwd": (q, s, x[:, :128].contiguous()),
        "moe_mlp_few": (x[:40].contiguous(), topk, w, codes(4, 256, 256), scales(4, 2, 2), codes(4, 256, 128),
                        scales(4, 2, 1)),
    }


FORMS = sorted(_inputs("cpu"))


def _tensors(r):
    return [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,)) if t is not None]


class _Streams:
    """Stand-ins: which stream is current, where each tensor was allocated, which streams it was marked for."""

    def __init__(self, monkeypatch):
        self.now, self.allocated, self.marked = "caller's", [], []
        empty = torch.empty

        @contextlib.contextmanager
        def use(s):
            before, self.now = self.now, s
            yield
            self.now = before

        def allocate(*a, **k):
            t = empty(*a, **k)
            self.allocated.append((t, self.now))
            return t
        monkeypatch.setattr(torch, "empty", allocate)
        monkeypatch.setattr(torch.cuda, "stream", use)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.marked.append((t, s)), raising=False)


@pytest.mark.parametrize("name", FORMS)
def test_allocations_belong_to_the_stream(name, monkeypatch):
    fgbuild.build()
    args = _inputs("cpu")[name]
    launched = []
    monkeypatch.setattr(fg, "fp8_" + name, lambda *a, **k: launched.append(k.get("stream", a[-1])), raising=False)
    if name in ("gemm", "grouped_gemm"):
        call = {"gemm": "fp8_blockscaled_gemm", "grouped_gemm": "fp8_grouped_gemm"}[name]
        monkeypatch.setattr(fg, call, lambda *a, **k: launched.append(k.get("stream", a[-1])))
    seen = _Streams(monkeypatch)
    out = _tensors(getattr(fg, name)(*args, stream="side"))
    assert launched == ["side"] and len(seen.allocated) >= len(out)
    assert all(where == "side" for _, where in seen.allocated)
    # the results are the caller's: freed by it, they wait for what it made of them on its own stream
    assert all(any(t is m and s == "caller's" for m, s in seen.marked) for t in out)
    # without a stream nothing is switched or marked
    seen.allocated.clear()
    seen.marked.clear()
    getattr(fg, name)(*args)
    assert launched[1:] == [None] and not seen.marked
    assert all(where == "caller's" for _, where in seen.allocated)


@pytest.mark.gpu
@pytest.mark.parametrize("name", FORMS)
def test_side_stream_beside_allocations_of_the_current_one(name):
    device = torch.device("cuda", 0)
    args = _inputs(device)[name]
    form = getattr(fg, name)
    ref = [t.clone() for t in _tensors(form(*args))]
    sizes = [t.numel() * t.element_size() for t in ref]
    if name == "moe_mlp_few":
        sizes.append(fg.fp8_moe_mlp_few_workspace_bytes(40, 2, 4, 256, 128, 256))
    if name == "moe_dispatch":
        sizes.append(fg.fp8_moe_dispatch_workspace_bytes(40, 2, 4))
        live = int(ref[2][-1])
        ref[0], ref[1], ref[4] = ref[0][:live], ref[1][:, :live], ref[4][:live]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)          # about a millisecond: the call's kernels start behind it
        got = _tensors(form(*args, stream=side))
        junk = [torch.full((max(n, 1),), 0x5A, dtype=U8, device=device) for n in sizes for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        if name == "moe_dispatch":
            got[0], got[1], got[4] = got[0][:live], got[1][:, :live], got[4][:live]
        for a, b in zip(got, ref):
            assert torch.equal(a.contiguous().view(U8), b.contiguous().view(U8))
        del got, junk
    assert fg.fp8_get_status() == fg.FP8_OK
