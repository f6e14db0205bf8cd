"""The SwiGLU's backward over the grouped rows of an MoE layer, as training
runs it: dispatch, grouped GEMM, forward and backward with the rows in use taken
from the dispatch's offsets, then each expert's Wgrads by the dense GEMM on its
columns of the operands along tokens.  Every stage against FP64 on the operands
the GPU itself handed it.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import synth
from oracle import mlp

from gpu_util import assert_gemm_close, d2h, dev

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -20          # FP32 rounding of the SwiGLU's arithmetic


def _n(t):
    return t.cpu().numpy()


def _cols(qT, s):
    """128x1 codes [C, T], scales [T/128, C] -> values [C, T]."""
    return mlp.decode(_n(qT)) * np.repeat(_n(s).astype(np.float64).T, 128, axis=1)


def _cols_ok(qT, s, v, err):
    S = np.repeat(_n(s).astype(np.float64), 128, axis=0)
    assert mlp.code_excess(_n(qT).T, S, v, err) <= 0.0


@pytest.mark.parametrize("T,k,G,K,I,N", [(300, 2, 5, 256, 128, 384), (64, 1, 6, 128, 256, 128)])
def test_grouped_forward_backward_and_wgrads(T, k, G, K, I, N):
    d = dev()
    x = synth.activations(T, K, seed=1).to(d)
    topk = synth.zipf_topk_routing(T, G, k, seed=2).to(torch.int32).to(d)
    w13, s13 = (torch.empty((G, 2 * I, K), dtype=torch.uint8, device=d),
                torch.empty((G, 2 * I // 128, K // 128), dtype=torch.float32, device=d))
    fg.fp8_quant_w_128x128(synth.normal((G * 2 * I, K), K ** -0.5, 3).to(d), w13.view(G * 2 * I, K),
                           s13.view(G * 2 * I // 128, K // 128))
    qx, sx = fg.quant_act_1x128(x)
    rows = fg.moe_dispatch(qx, sx, topk, G)
    off, n_rows = _n(rows["offsets"]), rows["offsets"][G:]
    live = int(off[-1])
    M = rows["q"].shape[0]
    assert live < M                                       # rows behind the last group: whatever they hold
    h = fg.grouped_gemm(rows["q"], rows["sA"], w13, s13, rows["offsets"])
    h[live:] = float("nan")
    u8, f32 = dict(dtype=torch.uint8, device=d), dict(dtype=torch.float32, device=d)
    qa, sa, qh, sh = (torch.zeros((M, I), **u8), torch.zeros((I // 128, M), **f32), torch.zeros((M, 2 * I), **u8),
                      torch.zeros((2 * I // 128, M), **f32))
    fg.fp8_swiglu_quant(h, qa, sa, qh, sh, n_rows=n_rows)
    # gradients of the second GEMM's input: rows that pad a group carry none
    da = synth.normal((M, I), 1e-3, 4).to(torch.bfloat16).to(d)
    da[rows["row_token"] < 0] = 0
    da[live:] = float("nan")
    dy = synth.normal((M, N), 1e-3, 5).to(torch.bfloat16).to(d)
    dy[rows["row_token"] < 0] = 0
    dy[live:] = 0
    g = dict(qdh=torch.zeros((M, 2 * I), **u8), sdh=torch.zeros((2 * I // 128, M), **f32),
             qdhT=torch.zeros((2 * I, M), **u8), sdhT=torch.zeros((M // 128, 2 * I), **f32),
             qaT=torch.zeros((I, M), **u8), saT=torch.zeros((M // 128, I), **f32))
    fg.fp8_swiglu_bwd(qh, sh, da, **g, n_rows=n_rows)
    H = mlp.decode_1x128(_n(qh)[:live], _n(sh)[:, :live])
    dh, mag = mlp.swiglu_grads(H, da[:live].double().cpu().numpy())
    a = mlp.swiglu(H)
    _cols_ok(g["qdhT"][:, :live], g["sdhT"][:live // 128], dh, ERR * mag)
    _cols_ok(g["qaT"][:, :live], g["saT"][:live // 128], a, ERR * np.abs(a))
    qxT, sxT = fg.requant_1x128_to_128x1(rows["q"], rows["sA"])
    qyT, syT = fg.quant_act_128x1(dy)
    empty = 0
    for e in range(G):
        r = slice(off[e], off[e + 1])
        b = slice(off[e] // 128, off[e + 1] // 128)
        if off[e] == off[e + 1]:
            empty += 1
            continue
        for (A, sA), (B, sB) in ((("qdhT", "sdhT"), (qxT, sxT)), ((qyT, syT), ("qaT", "saT"))):
            A, sA = (g[A], g[sA]) if isinstance(A, str) else (A, sA)
            B, sB = (g[B], g[sB]) if isinstance(B, str) else (B, sB)
            A, B, sA, sB = A[:, r].contiguous(), B[:, r].contiguous(), sA[b], sB[b]
            dw = fg.gemm(A, sA, B, sB, torch.float32, sb_gran=1)
            va, vb = _cols(A, sA), _cols(B, sB)
            assert_gemm_close(d2h(dw), va @ vb.T, np.abs(va) @ np.abs(vb).T, False, f"expert {e}")
    assert empty < G and fg.fp8_get_status() == fg.FP8_OK
