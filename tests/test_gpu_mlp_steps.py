"""The gated-MLP operators together with the GEMMs, quantizers and MoE calls
around them, as the steps of linear.py run them.

Every stage is compared with FP64 on the operands the GPU itself handed it: a
GEMM within 1e-4 of its sum of magnitudes (plus half a BF16 step), a quantizer's
or the SwiGLU's codes within half a step of their values.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import linear, synth
from oracle import mlp

from gpu_util import assert_gemm_close, d2h, dev, to_dev

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -20          # FP32 rounding of the SwiGLU's arithmetic


def _n(t):
    return t.cpu().numpy()


def _cols(qT, s):
    """128x1 codes [C, T], scales [T/128, C] -> values [C, T]."""
    return mlp.decode(_n(qT)) * np.repeat(_n(s).astype(np.float64).T, 128, axis=1)


def _product(got, A, B, what):
    """got = A . B^T"""
    assert_gemm_close(d2h(got), A @ B.T, np.abs(A) @ np.abs(B).T, got.dtype == torch.bfloat16, what)


def _rows_ok(q, s, v, err):
    S = np.repeat(s.astype(np.float64).T, 128, axis=1)
    assert mlp.code_excess(q, S, v, err) <= 0.0


def _mlp(M, K, I, N, mode, dtype=torch.bfloat16):
    x = synth.activations(M, K, seed=1, dtype=dtype)
    w13, w2 = synth.normal((2 * I, K), K ** -0.5, 2), synth.normal((N, I), I ** -0.5, 3)
    return linear.GatedMlpStep(x.to(dev()), w13.to(dev()), w2.to(dev()), scale_mode=mode)


@pytest.mark.parametrize("mode", [fg.SCALE_FP32, fg.SCALE_POW2])
@pytest.mark.parametrize("M,K,I,N", [(128, 256, 128, 256), (384, 512, 256, 384)])
def test_gated_mlp_forward_and_backward(M, K, I, N, mode):
    step = _mlp(M, K, I, N, mode)
    y = step()
    dy = synth.normal((M, N), 1e-3, 4).to(dev())
    dx, dw13, dw2 = step.backward(dy)
    assert fg.fp8_get_status() == fg.FP8_OK
    X = mlp.decode_1x128(_n(step.qx), _n(step.sx))
    W13 = mlp.decode_128x128(_n(step.qw13), _n(step.sw13))
    W2 = mlp.decode_128x128(_n(step.qw2), _n(step.sw2))
    _product(step.h, X, W13, "h")
    h = d2h(step.h)
    _rows_ok(_n(step.qa), _n(step.sa), mlp.swiglu(h), ERR * np.abs(mlp.swiglu(h)) + 2.0 ** -126)
    A = mlp.decode_1x128(_n(step.qa), _n(step.sa))
    _product(y, A, W2, "y")

    g = step._grad
    DY = mlp.decode_1x128(_n(g["qdy"]), _n(g["sdy"]))
    _product(g["da"], DY, W2.T, "da")
    H = mlp.decode_1x128(_n(step.qh), _n(step.sh))
    dh, mag = mlp.swiglu_grads(H, d2h(g["da"]))
    _rows_ok(_n(g["qdh"]), _n(g["sdh"]), dh, ERR * mag + 2.0 ** -126)
    DH = mlp.decode_1x128(_n(g["qdh"]), _n(g["sdh"]))
    _product(dx, DH, W13.T, "dx")
    _product(dw13, _cols(g["qdhT"], g["sdhT"]), _cols(g["qxT"], g["sxT"]), "dw13")
    _product(dw2, _cols(g["qdyT"], g["sdyT"]), _cols(g["qaT"], g["saT"]), "dw2")
    # the 128x1 operands hold the same gradient and activation as the 1x128 ones: every value of
    # each is within half an E4M3 step (2^-4, subnormals: of its group's smallest step) of the other's source
    cols = _cols(g["qdhT"], g["sdhT"]).T
    step_c = np.repeat(_n(g["sdhT"]).astype(np.float64), 128, axis=0) * 2.0 ** -10
    assert np.all(np.abs(cols - dh) <= np.abs(dh) * 2.0 ** -4 * (1 + 2.0 ** -10) + step_c + ERR * mag)


def test_gated_mlp_gradients_follow_the_formula():
    """Against FP64 gradients of the unquantized MLP.  Eight roundings to E4M3 (x, w13, h, da, w2, dy, a, dh),
    each off by at most 2^-4 of its value, lie on the way to a gradient; independent of one another
    they add up in quadrature to at most sqrt(8) * 2^-4 = 0.177 of the gradient's norm."""
    M, K, I, N = 256, 512, 256, 512
    step = _mlp(M, K, I, N, fg.SCALE_FP32)
    step()
    dy = synth.normal((M, N), 1e-3, 5)
    grads = step.backward(dy.to(dev()))
    x, w13, w2, gy = (t.cpu().double().requires_grad_(True) for t in (step.x, step.w13, step.w2, dy))
    h = x @ w13.t()
    a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    (a @ w2.t()).backward(gy.detach())
    for got, ref in zip(grads, (x.grad, w13.grad, w2.grad)):
        off = (got.cpu().double() - ref).norm() / ref.norm()
        assert off <= 0.177, float(off)


def test_gated_mlp_ragged_forward_and_refused_backward():
    step = _mlp(200, 256, 128, 256, fg.SCALE_FP32)
    y = step()
    X, W13 = mlp.decode_1x128(_n(step.qx), _n(step.sx)), mlp.decode_128x128(_n(step.qw13), _n(step.sw13))
    _product(step.h, X, W13, "h")
    _product(y, mlp.decode_1x128(_n(step.qa), _n(step.sa)), mlp.decode_128x128(_n(step.qw2), _n(step.sw2)), "y")
    with pytest.raises(ValueError, match="128 tokens"):
        step.backward(torch.zeros((200, 256), dtype=torch.bfloat16, device=dev()))


def test_gated_mlp_captured_forward_and_backward():
    step = _mlp(256, 256, 256, 256, fg.SCALE_FP32)
    dy = synth.normal((256, 256), 1e-3, 6).to(dev())
    ref = [step().clone()] + [t.clone() for t in step.backward(dy)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = (step(s),) + step.backward(dy, s)
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def _layer(T, k, G, K, I, N, seed=0):
    x = synth.activations(T, K, seed=seed).to(dev())
    topk = synth.zipf_topk_routing(T, G, k, seed=seed + 1).to(torch.int32).to(dev())
    w = torch.from_numpy(np.random.default_rng(seed).uniform(0.1, 1.0, (T, k)).astype(np.float32)).to(dev())
    q = []
    for n, c, sd in ((2 * I, K, 2), (N, I, 3)):
        codes = torch.empty((G, n, c), dtype=torch.uint8, device=dev())
        scales = torch.empty((G, n // 128, c // 128), dtype=torch.float32, device=dev())
        fg.fp8_quant_w_128x128(synth.normal((G * n, c), c ** -0.5, seed + sd).to(dev()), codes.view(G * n, c),
                               scales.view(G * n // 128, c // 128))
        q += [codes, scales]
    return (x, topk, w, *q)


def test_moe_mlp_dispatched_stage_by_stage():
    T, k, G, K, I, N = 300, 3, 6, 256, 128, 384
    args = _layer(T, k, G, K, I, N)
    step = linear.MoeMlpStep(*args)
    assert not step.few
    out = step()
    assert fg.fp8_get_status() == fg.FP8_OK
    off = _n(step.offsets)
    rows = off[-1]
    R = mlp.decode_1x128(_n(step.qr), _n(step.sr))
    h, y = d2h(step.h), d2h(step.y)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        _product(step.h[r], R[r], mlp.decode_128x128(_n(args[3])[e], _n(args[4])[e]), "h")
        A = mlp.decode_1x128(_n(step.qa)[r], _n(step.sa)[:, r])
        _product(step.y[r], A, mlp.decode_128x128(_n(args[5])[e], _n(args[6])[e]), "y")
    a = mlp.swiglu(h[:rows])
    _rows_ok(_n(step.qa)[:rows], _n(step.sa)[:, :rows], a, ERR * np.abs(a) + 2.0 ** -126)
    tr, w = _n(step.token_row), _n(args[2]).astype(np.float64)
    ref = np.einsum("tj,tjn->tn", w, y[tr])
    tol = np.einsum("tj,tjn->tn", np.abs(w), np.abs(y[tr]))
    assert np.all(np.abs(d2h(out) - ref) <= 2.0 ** -20 * tol + 2.0 ** -8 * np.abs(ref) + 1e-30)


@pytest.mark.parametrize("T", [1, 20, 128])
def test_moe_mlp_few_and_dispatched_agree(T):
    """The two forms differ in H (FP32 against BF16, 2^-9 off) and through it in which way activations
    round to E4M3: an element by one step, 2^-3 of it, at most.  About 2^-9 / 2^-4 = 3 % of the
    elements change, so the outputs' norm of the difference stays below sqrt(0.03) * 2^-3 + 2^-8 = 2.6 %;
    twice that is allowed."""
    args = _layer(T, 4, 8, 512, 256, 512, seed=T)
    a, b = linear.MoeMlpStep(*args), linear.MoeMlpStep(*args, few=False)
    assert a.few and not b.few
    ya, yb = a().double(), b().double()
    assert fg.fp8_get_status() == fg.FP8_OK
    assert float((ya - yb).norm() / yb.norm()) <= 0.052


def test_moe_mlp_refusals():
    args = _layer(129, 2, 4, 256, 128, 256)
    with pytest.raises(ValueError, match="few-token"):
        linear.MoeMlpStep(*args, few=True)
    with pytest.raises(ValueError, match="BF16"):
        linear.MoeMlpStep(*args, out_dtype=torch.float32)
    x = torch.zeros((128, 256), dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError, match="fit"):
        linear.GatedMlpStep(x, torch.zeros((256, 128), device=dev()), torch.zeros((256, 128), device=dev()))


def test_gated_mlp_backward_refusals():
    x = torch.zeros((128, 256), dtype=torch.bfloat16, device=dev())
    step = linear.GatedMlpStep(x, torch.zeros((256, 256), device=dev()), torch.zeros((384, 128), device=dev()))
    dy = torch.zeros((128, 384), dtype=torch.bfloat16, device=dev())
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(dy)
    step()
    for bad in (dy[:64], dy[:, :256], torch.zeros((256, 384), dtype=torch.bfloat16, device=dev()), dy.cpu()):
        with pytest.raises(ValueError, match="dy"):
            step.backward(bad)
    assert all(bool((g == 0).all()) for g in step.backward(dy))
    assert fg.fp8_get_status() == fg.FP8_OK
