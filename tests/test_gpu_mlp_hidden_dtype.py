"""The steps of linear.py with H (and dA) kept in FP32 between the GEMMs and the
SwiGLU: every stage against FP64 on the operands the GPU itself handed it."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import linear, synth
from oracle import mlp

from gpu_util import assert_gemm_close, d2h, dev

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -20          # FP32 rounding of the SwiGLU's arithmetic


def _n(t):
    return t.cpu().numpy()


def _rows_ok(q, s, v, err):
    S = np.repeat(_n(s).astype(np.float64).T, 128, axis=1)
    assert mlp.code_excess(_n(q), S, v, err) <= 0.0


def test_gated_mlp_with_fp32_h_and_da():
    M, K, I, N = 256, 256, 128, 384
    x = synth.activations(M, K, seed=1).to(dev())
    w13, w2 = synth.normal((2 * I, K), K ** -0.5, 2).to(dev()), synth.normal((N, I), I ** -0.5, 3).to(dev())
    step = linear.GatedMlpStep(x, w13, w2, hidden_dtype=torch.float32)
    step()
    step.backward(synth.normal((M, N), 1e-3, 4).to(dev()))
    g = step._grad
    assert step.h.dtype == g["da"].dtype == torch.float32
    X, W13 = mlp.decode_1x128(_n(step.qx), _n(step.sx)), mlp.decode_128x128(_n(step.qw13), _n(step.sw13))
    assert_gemm_close(d2h(step.h), X @ W13.T, np.abs(X) @ np.abs(W13).T, False, "h")
    h = d2h(step.h).astype(np.float64)
    a = mlp.swiglu(h)
    _rows_ok(step.qa, step.sa, a, ERR * np.abs(a))
    DY, W2 = mlp.decode_1x128(_n(g["qdy"]), _n(g["sdy"])), mlp.decode_128x128(_n(step.qw2), _n(step.sw2))
    assert_gemm_close(d2h(g["da"]), DY @ W2, np.abs(DY) @ np.abs(W2), False, "da")
    dh, mag = mlp.swiglu_grads(mlp.decode_1x128(_n(step.qh), _n(step.sh)), d2h(g["da"]).astype(np.float64))
    _rows_ok(g["qdh"], g["sdh"], dh, ERR * mag)
    # the sums themselves, not sums rounded to BF16
    assert bool((step.h != step.h.bfloat16().float()).any())
    with pytest.raises(ValueError, match="share"):
        linear.GatedMlpStep(x, w13, w2, share=step)
    assert fg.fp8_get_status() == fg.FP8_OK


def test_dispatched_moe_mlp_with_fp32_h_agrees_better_with_the_few_token_form():
    """With H in FP32 in both forms only the order of its sums differs: 1e-4 of their sums of magnitudes at most
    (the GEMMs' bound), where BF16 rounds by 2^-9.  Few activations then round to another E4M3 code, so
    the two outputs (BF16 sums of BF16 products: 2^-9 each) are nearer than with BF16 H."""
    T, k, G, K, I, N = 96, 4, 8, 512, 256, 512
    x = synth.activations(T, K, seed=3).to(dev())
    topk = synth.zipf_topk_routing(T, G, k, seed=4).to(torch.int32).to(dev())
    w = torch.from_numpy(np.random.default_rng(5).uniform(0.1, 1.0, (T, k)).astype(np.float32)).to(dev())
    q = []
    for n, c, sd in ((2 * I, K, 6), (N, I, 7)):
        codes = torch.empty((G, n, c), dtype=torch.uint8, device=dev())
        scales = torch.empty((G, n // 128, c // 128), dtype=torch.float32, device=dev())
        fg.fp8_quant_w_128x128(synth.normal((G * n, c), c ** -0.5, sd).to(dev()), codes.view(G * n, c),
                               scales.view(G * n // 128, c // 128))
        q += [codes, scales]
    few = linear.MoeMlpStep(x, topk, w, *q)().double()
    off = []
    for dtype in (torch.bfloat16, torch.float32):
        step = linear.MoeMlpStep(x, topk, w, *q, few=False, hidden_dtype=dtype)
        assert step.h.dtype == dtype
        off.append(float((step().double() - few).norm() / few.norm()))
    assert off[1] < off[0] and off[1] <= 0.026       # (the bound that holds for BF16 H)
    assert fg.fp8_get_status() == fg.FP8_OK
