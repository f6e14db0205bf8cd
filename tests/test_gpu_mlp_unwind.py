"""The failure path of the gated-MLP kernels on the GPU, without a fault: a
self-test launch holds back one hand-over (SwiGLU backward) or the token rows of
every CTA's first unit (few-token MoE MLP, either phase), so that the waits run
into a short limit.  The launch has to end, with FP8_ERR_TIMEOUT reported once,
write nothing outside its outputs, and leave the context and its own workspace fit
for a normal call, whose bits are those of an undisturbed one.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
import oracle
from fp8_fine_grained_x1_b200 import synth

from gpu_util import dev, to_dev

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000          # ns


def _times_out(launch):
    assert fg.fp8_get_status() == fg.FP8_OK
    fg.fp8_set_wait_timeout_ns(LIMIT)
    try:
        launch()
        assert fg.fp8_get_status() == fg.FP8_ERR_TIMEOUT
        assert fg.fp8_get_status() == fg.FP8_OK
    finally:
        fg.fp8_set_wait_timeout_ns(0)


def _guarded(shape, dtype, before=4096):
    """A tensor of this shape between two stretches of a known byte, and a check that they are untouched."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    room = torch.full((n + 2 * before,), 0x5A, dtype=torch.uint8, device=dev())
    t = room[before:before + n].view(dtype).view(shape)

    def intact():
        return bool((room[:before] == 0x5A).all()) and bool((room[before + n:] == 0x5A).all())
    return t, intact


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,I", [(128, 128), (2560, 1152)])       # one tile; more tiles than CTAs
def test_swiglu_bwd(M, I, dtype):
    rng = np.random.default_rng(M)
    q, s = oracle.quant_act_1x128(rng.normal(0, 2, (M, 2 * I)).astype(np.float32))
    q, s = to_dev(q), to_dev(s)
    da = to_dev(rng.normal(0, 1e-3, (M, I)).astype(np.float32)).to(dtype)
    ref = fg.swiglu_bwd(q, s, da, ("qdhT",))
    (qdhT, ok1), (sdhT, ok2) = _guarded((2 * I, M), torch.uint8), _guarded((M // 128, 2 * I), torch.float32)
    _times_out(lambda: fg.fp8_selftest_swiglu_bwd_unwind(q, s, da, qdhT, sdhT))
    assert ok1() and ok2()
    fg.fp8_swiglu_bwd(q, s, da, qdhT=qdhT, sdhT=sdhT)
    assert torch.equal(qdhT, ref["qdhT"]) and torch.equal(sdhT, ref["sdhT"])
    assert ok1() and ok2() and fg.fp8_get_status() == fg.FP8_OK


@pytest.mark.parametrize("phase", [1, 2])
@pytest.mark.parametrize("T", [4, 20, 33, 128])                   # 16 and 32 columns; rows
def test_moe_mlp_few(T, phase):
    k, G, K, I, N = 2, 5, 512, 256, 640
    x = synth.activations(T, K, seed=T).to(dev())
    topk = synth.zipf_topk_routing(T, G, k, seed=1).to(torch.int32).to(dev())
    w = torch.full((T, k), 0.5, dtype=torch.float32, device=dev())
    args = [x, topk, w]
    for n, c, sd in ((2 * I, K, 2), (N, I, 3)):
        codes = torch.empty((G, n, c), dtype=torch.uint8, device=dev())
        scales = torch.empty((G, n // 128, c // 128), dtype=torch.float32, device=dev())
        fg.fp8_quant_w_128x128(synth.normal((G * n, c), c ** -0.5, sd).to(dev()), codes.view(G * n, c),
                               scales.view(G * n // 128, c // 128))
        args += [codes, scales]
    ref = fg.moe_mlp_few(*args)
    n = fg.fp8_moe_mlp_few_workspace_bytes(T, k, G, K, I, N)
    (out, ok1), (ws, ok2) = _guarded((T, N), torch.bfloat16), _guarded((n,), torch.uint8)
    _times_out(lambda: fg.fp8_selftest_moe_mlp_few_unwind(phase, *args, out, ws))
    assert ok1() and ok2()
    fg.fp8_moe_mlp_few(*args, out, ws)
    assert torch.equal(out, ref) and fg.fp8_get_status() == fg.FP8_OK
    assert ok1() and ok2()
