"""The SwiGLU's sigmoid over FP32's whole range of gates, against FP64: gates far
below zero, where silu(g) = g / (1 + exp(-g)) is tiny but a normal FP32 number,
with up values and gradients large enough for the products to be normal too.

Tolerances, in units of 2^-22: the exponential instruction is off by at most 1
(two units in the last place), the FP32 ln(2) that makes its argument's
rounding good by |g| * 2.8e-9, 1.1 at most here; 1 + exp(-g) is two roundings (1/4
each), its reciprocal one unit in the last place (1/2).  So a sigmoid is off by at
most 3.1, and by 4.35 where it is made of two factors (below about -86.6: one more
exponential and product).  The activation adds two products (1/4 each), 4.85 together;
the gate's gradient the three roundings of 1 + g (1 - s) and of its product with s (3/4),
and two products, 5.6 together; the up half's gradient is like the activation.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
from oracle import mlp

from gpu_util import dev, half_ulp_bf16, to_dev

pytestmark = pytest.mark.gpu

ACT, GRAD = 4.85 * 2.0 ** -22, 5.6 * 2.0 ** -22
MODES = [fg.SCALE_FP32, fg.SCALE_POW2]


def _np(t):
    return t.cpu().numpy()


def _decoded(q, s):
    """What the backward takes from a checkpoint: code * scale, an FP32 product."""
    return mlp.decode_1x128(q, s).astype(np.float32).astype(np.float64)


def _rows_ok(q, s, v, err, mode):
    def amax(x):
        return np.abs(x).reshape(x.shape[0], -1, 128).max(2).T
    S = np.repeat(s.astype(np.float64).T, 128, axis=1)
    assert mlp.scale_error(s, amax(v), amax(err), mode) <= 2.0 ** -22
    assert mlp.code_excess(q, S, v, err) <= 0.0


def _cols_ok(qT, s, v, err, mode):
    def amax(x):
        return np.abs(x).reshape(-1, 128, x.shape[1]).max(1)
    S = np.repeat(s.astype(np.float64), 128, axis=0)
    assert mlp.scale_error(s, amax(v), amax(err), mode) <= 2.0 ** -22
    assert mlp.code_excess(qT.T, S, v, err) <= 0.0


def _gates(kind, shape, rng):
    """`low` ends where silu(g) is still normal; `around` lies on both sides of ln(2^126) = 87.34."""
    lo, hi = dict(moderate=(-20.0, -8.0), far=(-85.0, -60.0), around=(-88.5, -86.0), low=(-91.5, -87.5))[kind]
    return rng.uniform(lo, hi, shape)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["moderate", "far", "around", "low"])
def test_forward(kind, dtype, mode):
    M, I = 200, 256
    rng = np.random.default_rng(1)
    h = np.concatenate((_gates(kind, (M, I), rng), rng.normal(0, 1e10, (M, I))), 1).astype(np.float32)
    x = to_dev(h)
    if dtype == "bf16":
        x = x.to(torch.bfloat16)
    val = x.double().cpu().numpy()
    a = mlp.swiglu(val)
    for keep in (True, False):
        qa, sa, _, _ = fg.swiglu_quant(x, keep, mode)
        _rows_ok(_np(qa), _np(sa), a, ACT * np.abs(a), mode)


def _codes(values):
    """E4M3 codes of values that the format holds."""
    table = {float(mlp.decode(np.uint8(c))): c for c in range(256) if c not in (0x7F, 0xFF)}
    return np.vectorize(table.__getitem__, otypes=[np.uint8])(values)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale,codes", [(91.5 / 448, (-448, -416)), (91.5 / 448, (-448, -416, -384, -288)),
                                         (0.25, (-352, -344 + 24)), (0.03, (-448, -416, -352))])
def test_backward(scale, codes, dtype, mode):
    """Gates that are codes times a scale: -91.5 .. -58, -88 and -80, -13.4 .. -10.6."""
    M, I = 256, 256
    rng = np.random.default_rng(2)
    q = np.concatenate((_codes(rng.choice(np.array(codes, np.float64), (M, I))),
                        rng.choice(np.array([0x38, 0x40, 0x7E, 0xB9, 0xF0], np.uint8), (M, I))), 1)
    s = np.concatenate((np.full((I // 128, M), scale), np.full((I // 128, M), 1e8))).astype(np.float32)
    h = _decoded(q, s)
    da = to_dev(rng.normal(0, 1e20, (M, I)).astype(np.float32))
    da = da.to(torch.bfloat16) if dtype == "bf16" else da
    dv = da.double().cpu().numpy()
    dh, mag = mlp.swiglu_grads(h, dv)
    a = mlp.swiglu(h)
    out = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh", "qdh", "qdhT", "qaT"), mode)
    got = out["dh"].double().cpu().numpy()
    assert np.all(np.abs(got - dh) <= half_ulp_bf16(np.maximum(np.abs(dh), np.abs(got))) + GRAD * mag)
    _rows_ok(_np(out["qdh"]), _np(out["sdh"]), dh, GRAD * mag, mode)
    _cols_ok(_np(out["qdhT"]), _np(out["sdhT"]), dh, GRAD * mag, mode)
    _cols_ok(_np(out["qaT"]), _np(out["saT"]), a, ACT * np.abs(a), mode)
    rows = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh", "qdh"), mode)      # the kernel without operands along tokens
    assert torch.equal(rows["dh"], out["dh"]) and torch.equal(rows["qdh"], out["qdh"])
    assert torch.equal(rows["sdh"], out["sdh"])


EXTREME = [3.3e38, 2.5e38, 1e38, 1e30, 200.0, 104.0, 88.0, 87.0, 86.0, 1.0, 1e-30, 0.0, -1e-30, -1.0, -86.0, -87.0, -88.0,
           -104.0, -200.0, -1e30, -1e38, -3.3e38]


@pytest.mark.parametrize("mode", MODES)
def test_forward_at_the_ends_of_fp32(mode):
    """One such gate to a group (the others 1): finite, and right but for what is below FP32's normal numbers."""
    M, I = len(EXTREME), 128
    h = np.ones((M, 2 * I), np.float32)
    h[:, 37] = EXTREME
    h[:, I:] = 1e-3
    qa, sa, _, _ = fg.swiglu_quant(to_dev(h), True, mode)
    a = mlp.swiglu(h.astype(np.float64))
    _rows_ok(_np(qa), _np(sa), a, ACT * np.abs(a) + 2.0 ** -126, mode)


@pytest.mark.parametrize("mode", MODES)
def test_backward_at_the_ends_of_fp32(mode):
    """Whole groups of one such gate (a code of 448 times its 448th part)."""
    g = np.array([v for v in EXTREME if abs(v) > 1e-20])
    M, I = 128, 128
    s = np.ones((2, M), np.float32)
    s[0, :g.size] = np.abs(g) / 448
    s[1] = 1e-3
    q = np.full((M, 2 * I), 0x38, np.uint8)
    q[:g.size, :I] = np.where(g > 0, 0x7E, 0xFE)[:, None]
    h = _decoded(q, s)
    da = np.full((M, I), 1e-3, np.float32)
    out = fg.swiglu_bwd(to_dev(q), to_dev(s), to_dev(da), ("qdh", "qdhT", "qaT"), mode)
    dh, mag = mlp.swiglu_grads(h, da.astype(np.float64))
    a = mlp.swiglu(h)
    tiny = 2.0 ** -126
    # beyond g = 17.4, exp(-g) < 2^-25: 1 + exp(-g) rounds to 1, whose reciprocal is 1, and 1 + g (1 - s) is 1
    mag = np.where(np.concatenate((h[:, :I], h[:, :I]), 1) > 17.4, np.abs(dh), mag)
    # groups of nothing but numbers below FP32's normal ones may count as zeros, whose scale is 1
    sdh = _np(out["sdh"])
    amax = np.abs(dh).reshape(M, -1, 128).max(2).T
    none = amax < tiny
    assert none.any() and np.isin(sdh[none], np.array([1.0, 2.0 ** -126], np.float32)).all()
    sdh = np.where(none, np.where(amax == 0, 1.0, 2.0 ** -126).astype(np.float32), sdh)
    _rows_ok(_np(out["qdh"]), sdh, dh, GRAD * mag + tiny, mode)
    _cols_ok(_np(out["qdhT"]), _np(out["sdhT"]), dh, GRAD * mag + tiny, mode)
    _cols_ok(_np(out["qaT"]), _np(out["saT"]), a, ACT * np.abs(a) + tiny, mode)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [5, 20, 40])
def test_few_tokens(T, mode):
    """Experts whose gates are all -80, -88.5 and -91: every activation of a group is the same, its code the largest.
    h = 128 equal products, exact but for the scales' roundings (2 * 2^-24) and its own sum (2^-22 at most):
    |g| times that, 3.3e-5, is the relative error of exp(g); with the activation's, the scales' and the second
    product's (1e-4 of the sum of magnitudes, all of one sign) at most 1.4e-4."""
    G, K, I, N = 3, 128, 128, 256
    gate, up = np.array([-80.0, -88.5, -91.0]), 1e10
    one = np.full((G, 2 * I, K), 0x7E, np.uint8)                        # 448
    one[:, :I] = 0xFE
    s13 = np.empty((G, 2, 1), np.float32)
    s13[:, 0, 0], s13[:, 1, 0] = -gate / (128 * 448), up / (128 * 448)
    w2, s2 = np.full((G, N, I), 0x38, np.uint8), np.ones((G, N // 128, 1), np.float32)
    x = torch.ones((T, K), dtype=torch.bfloat16, device=dev())
    topk = (np.arange(T) % G).astype(np.int32)[:, None]
    out = fg.moe_mlp_few(x, to_dev(topk), to_dev(np.ones((T, 1), np.float32)), to_dev(one), to_dev(s13), to_dev(w2),
                         to_dev(s2), torch.float32, mode)
    assert fg.fp8_get_status() == fg.FP8_OK
    g64 = -(s13[:, 0, 0].astype(np.float64) * 128 * 448)
    ref = g64 / (1 + np.exp(-g64)) * (s13[:, 1, 0].astype(np.float64) * 128 * 448) * I
    got = out.double().cpu().numpy()
    want = ref[topk[:, 0]][:, None]
    # POW2 scales: the activation's code is its value over a power of two, half an E4M3 step (2^-4) off
    tol = 1.4e-4 + (2.0 ** -4 if mode == fg.SCALE_POW2 else 0.0)
    assert np.all(np.abs(got - want) <= tol * np.abs(want))


def test_infinite_gates():
    """silu of +inf is +inf, of -inf and NaN NaN: the group's FP32 scale is infinite after the first, and its own
    element a NaN code after all three."""
    h = torch.ones((3, 256), device=dev())
    h[:, 37] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    for dtype in (torch.float32, torch.bfloat16):
        qa, sa, _, _ = fg.swiglu_quant(h.to(dtype))
        assert bool(((qa[:, 37] & 0x7F) == 0x7F).all())
        assert float(sa[0, 0]) == float("inf") and bool(torch.isfinite(sa[0, 1:]).all())
    q = torch.full((128, 256), 0x38, dtype=torch.uint8, device=dev())
    s = torch.ones((2, 128), device=dev())
    s[0, 5] = float("inf")                                # all gates of a token
    out = fg.swiglu_bwd(q, s, torch.ones((128, 128), device=dev()), ("dh", "qaT"))
    assert bool(torch.isnan(out["dh"][5, :128]).all()) and bool((out["dh"][5, 128:] == float("inf")).all())
    keep = torch.arange(128, device=dev()) != 5
    assert bool(torch.isfinite(out["dh"][keep]).all())
    assert bool((out["saT"] == float("inf")).all())
