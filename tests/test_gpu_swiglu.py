"""The FP8 SwiGLU (forward with its checkpoint, backward from it) on the GPU
against FP64 formulas.

Tolerances: the kernels compute in FP32, so a value may be off by ERR = 2^-20
of the magnitude of the terms it is made of (about ten FP32 roundings and
approximations of at most 2^-23 each: exp, sum, quotient, three or four
products); a code may then lie half an E4M3 step plus that error from its
value, a scale 2^-22 beyond its max-abs's own error, a BF16 result half a BF16
step.  The checkpoint of given inputs is exact, bit for bit.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
import oracle
from oracle import mlp

from gpu_util import bits_to_bf16_dev, dev, half_ulp_bf16, to_dev

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -20
JUNK = 0x5A


def _bf16(v):
    """float32 array -> (uint16 BF16 bits, their float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16), t.float().numpy().astype(np.float64)


def _input(v, dtype, pad=0):
    """Device tensor (its rows `pad` elements apart beyond their width) and its FP64 values."""
    if dtype == "bf16":
        bits, val = _bf16(v)
        t = bits_to_bf16_dev(bits)
    else:
        t, val = to_dev(np.asarray(v, np.float32)), np.asarray(v, np.float32).astype(np.float64)
    if pad:
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
        wide[:, :t.shape[1]] = t
        t = wide[:, :v.shape[1]]
    return t, val


def _h(M, I, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    h = rng.normal(0, 2.0, (M, 2 * I))
    if kind == "wild":      # groups of zeros, gates far out on both sides, tiny and huge values
        h[:, :128] = 0.0
        h[::3, 128:140] = -200.0
        h[1::3, 128:140] = 200.0
        h[2::3, I:I + 64] = 1e-30
        h[0, I + 64:I + 70] = 1e15
        h[-1] = 0.0
    return h.astype(np.float32)


def _junk(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=dev())
    t.view(torch.uint8).fill_(JUNK)
    return t


def _untouched(t):
    return bool((t.contiguous().view(torch.uint8) == JUNK).all())


def _np(t):
    return t.cpu().numpy()


def _amax_rows(v):
    return np.abs(v).reshape(v.shape[0], -1, 128).max(2).T


def _amax_cols(v):
    return np.abs(v).reshape(-1, 128, v.shape[1]).max(1)


def _check_rows(q, s, v, err, mode):
    """1x128 codes and scales of FP64 values v known to within err."""
    S = np.repeat(s.astype(np.float64).T, 128, axis=1)
    assert mlp.scale_error(s, _amax_rows(v), _amax_rows(err), mode) <= 2.0 ** -22
    assert mlp.code_excess(q, S, v, err) <= 0.0


def _check_cols(qT, s, v, err, mode):
    S = np.repeat(s.astype(np.float64), 128, axis=0)
    assert mlp.scale_error(s, _amax_cols(v), _amax_cols(err), mode) <= 2.0 ** -22
    assert mlp.code_excess(qT.T, S, v, err) <= 0.0


# ------------------------------------------------------------ forward

@pytest.mark.parametrize("mode", [fg.SCALE_FP32, fg.SCALE_POW2])
@pytest.mark.parametrize("M,I,dtype,kind", [(1, 128, "bf16", "normal"), (1, 128, "fp32", "wild"),
                                            (63, 256, "bf16", "wild"), (65, 384, "fp32", "normal"),
                                            (200, 1152, "bf16", "normal")])
def test_forward(M, I, dtype, kind, mode):
    x, val = _input(_h(M, I, M + I, kind), dtype, pad=16)
    qa, sa, qh, sh = fg.swiglu_quant(x, True, mode)
    if dtype == "bf16":
        oq, os_ = oracle.quant_act_1x128(_bf16(val)[0], mode)
    else:
        oq, os_ = oracle.quant_act_1x128(val.astype(np.float32), mode)
    assert np.array_equal(_np(qh), oq) and np.array_equal(_np(sh), os_)
    a = mlp.swiglu(val)
    # results below FP32's smallest normal number may be flushed to zero
    _check_rows(_np(qa), _np(sa), a, ERR * np.abs(a) + 2.0 ** -126, mode)
    # without a checkpoint the same activation, bit for bit
    qa2, sa2, none, none2 = fg.swiglu_quant(x, False, mode)
    assert none is None and none2 is None
    assert torch.equal(qa, qa2) and torch.equal(sa, sa2)


def test_forward_empty_and_rows_in_use():
    x, val = _input(_h(300, 256, 5), "bf16")
    full = fg.swiglu_quant(x)
    for n, want in ((0, 0), (1, 1), (64, 64), (129, 129), (300, 300), (-5, 0), (1 << 30, 300)):
        qa, sa, qh, sh = (_junk(t.shape, t.dtype) for t in full)
        poisoned = x.clone()
        poisoned[want:] = float("nan")                # rows behind are not read
        fg.fp8_swiglu_quant(poisoned, qa, sa, qh, sh, n_rows=torch.tensor([n], dtype=torch.int32, device=dev()))
        for got, ref, axis in ((qa, full[0], 0), (sa, full[1], 1), (qh, full[2], 0), (sh, full[3], 1)):
            assert torch.equal(got.narrow(axis, 0, want), ref.narrow(axis, 0, want)), n
            assert _untouched(got.narrow(axis, want, 300 - want)), n
    e = torch.empty((0, 512), dtype=torch.bfloat16, device=dev())
    assert fg.swiglu_quant(e)[0].shape == (0, 256)


# ------------------------------------------------------------ backward

def _checkpoint(M, I, seed, kind="normal", mode=fg.SCALE_FP32):
    q, s = oracle.quant_act_1x128(_h(M, I, seed, kind), mode)
    return q, s, mlp.decode_1x128(q, s)


def _da(M, I, seed):
    d = np.random.default_rng(seed).normal(0, 1e-3, (M, I)).astype(np.float32)
    d[:, 5] = 0.0
    return d


@pytest.mark.parametrize("mode", [fg.SCALE_FP32, fg.SCALE_POW2])
@pytest.mark.parametrize("M,I,dtype,kind", [(128, 128, "bf16", "normal"), (128, 256, "fp32", "wild"),
                                            (384, 384, "bf16", "wild"), (256, 1152, "bf16", "normal")])
def test_backward_all_outputs(M, I, dtype, kind, mode):
    q, s, h = _checkpoint(M, I, M + I, kind, mode)
    da, dv = _input(_da(M, I, 3), dtype, pad=8)
    out = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh", "qdh", "qdhT", "qaT"), mode)
    dh, mag = mlp.swiglu_grads(h, dv)
    a = mlp.swiglu(h)
    tiny = 2.0 ** -126 * (1.0 + np.abs(np.concatenate((dv, dv), 1)))
    err, aerr = ERR * mag + tiny, ERR * np.abs(a) + 2.0 ** -126
    got = out["dh"].float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - dh) <= half_ulp_bf16(np.maximum(np.abs(dh), np.abs(got))) + err)
    _check_rows(_np(out["qdh"]), _np(out["sdh"]), dh, err, mode)
    _check_cols(_np(out["qdhT"]), _np(out["sdhT"]), dh, err, mode)
    _check_cols(_np(out["qaT"]), _np(out["saT"]), a, aerr, mode)


@pytest.mark.parametrize("M", [1, 7, 127, 129, 300])
def test_backward_ragged_rows(M):
    I = 256
    q, s, h = _checkpoint(M, I, M)
    da, dv = _input(_da(M, I, 4), "bf16")
    out = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh", "qdh"))
    dh, mag = mlp.swiglu_grads(h, dv)
    _check_rows(_np(out["qdh"]), _np(out["sdh"]), dh, ERR * mag, fg.SCALE_FP32)
    got = out["dh"].float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - dh) <= half_ulp_bf16(np.maximum(np.abs(dh), np.abs(got))) + ERR * mag)


def test_backward_any_subset_is_the_same():
    M, I = 256, 384
    q, s, _ = _checkpoint(M, I, 8)
    da, _ = _input(_da(M, I, 5), "bf16")
    args = (to_dev(q), to_dev(s), da)
    names = ("dh", "qdh", "qdhT", "qaT")
    full = fg.swiglu_bwd(*args, names)
    for bits in range(1, 16):
        part = fg.swiglu_bwd(*args, [n for i, n in enumerate(names) if bits >> i & 1])
        for n, t in part.items():
            assert torch.equal(t, full[n]), (bits, n)


def test_backward_rows_in_use():
    M, I = 384, 256
    q, s, h = _checkpoint(M, I, 9)
    da, dv = _input(_da(M, I, 6), "bf16")
    for n in (0, 1, 128, 200, 256, 384, -1, 1 << 30):
        want = min(max(n, 0), M)
        blocks = (want + 127) // 128 * 128
        o = dict(dh=_junk((M, 2 * I), torch.bfloat16), qdh=_junk((M, 2 * I), torch.uint8),
                 sdh=_junk((2 * I // 128, M), torch.float32), qdhT=_junk((2 * I, M), torch.uint8),
                 sdhT=_junk((M // 128, 2 * I), torch.float32), qaT=_junk((I, M), torch.uint8),
                 saT=_junk((M // 128, I), torch.float32))
        bad = da.clone()
        bad[want:] = float("nan")
        qb, sb = q.copy(), s.copy()
        qb[want:], sb[:, want:] = 0x7F, np.nan                 # rows behind are not read
        fg.fp8_swiglu_bwd(to_dev(qb), to_dev(sb), bad, **o,
                          n_rows=torch.tensor([n], dtype=torch.int32, device=dev()))
        hz, dz = h.copy(), dv.copy()
        hz[want:], dz[want:] = 0.0, 0.0
        dh, mag = mlp.swiglu_grads(hz, dz)
        a = mlp.swiglu(hz)
        for name, axis, live in (("dh", 0, want), ("qdh", 0, want), ("sdh", 1, want), ("qdhT", 1, blocks),
                                 ("sdhT", 0, blocks // 128), ("qaT", 1, blocks), ("saT", 0, blocks // 128)):
            assert _untouched(o[name].narrow(axis, live, o[name].shape[axis] - live)), (n, name)
        if want:
            _check_rows(_np(o["qdh"])[:want], _np(o["sdh"])[:, :want], dh[:want], ERR * mag[:want], fg.SCALE_FP32)
            _check_cols(_np(o["qdhT"])[:, :blocks], _np(o["sdhT"])[:blocks // 128], dh[:blocks],
                        ERR * mag[:blocks], fg.SCALE_FP32)
            _check_cols(_np(o["qaT"])[:, :blocks], _np(o["saT"])[:blocks // 128], a[:blocks],
                        ERR * np.abs(a[:blocks]), fg.SCALE_FP32)


@pytest.mark.parametrize("mode", [fg.SCALE_FP32, fg.SCALE_POW2])
def test_gates_far_below_zero(mode):
    """Whole groups of gates between -85 and -16, where exp(-g) is large.  exp(-g) is 2^(g * -log2(e)) with the
    product and the constant rounded to FP32: half a step of the exponent each at most, |g| * 2^-23 of the
    sigmoid together, beside the other errors."""
    M, I = 256, 256
    rng = np.random.default_rng(21)
    h = np.concatenate((rng.uniform(-85.0, -16.0, (M, I)), rng.normal(0, 1e18, (M, I))), 1).astype(np.float32)
    x, val = _input(h, "fp32")
    qa, sa, qh, sh = fg.swiglu_quant(x, True, mode)
    a = mlp.swiglu(val)
    _check_rows(_np(qa), _np(sa), a, (ERR + np.abs(val[:, :I]) * 2.0 ** -23) * np.abs(a), mode)
    back = mlp.decode_1x128(_np(qh), _np(sh))
    da, dv = _input(_da(M, I, 9), "fp32")
    out = fg.swiglu_bwd(qh, sh, da, ("qdh", "qdhT", "qaT"), mode)
    dh, mag = mlp.swiglu_grads(back, dv)
    a, g = mlp.swiglu(back), np.abs(back[:, :I])
    err = (ERR + np.concatenate((g, g), 1) * 2.0 ** -23) * mag
    _check_rows(_np(out["qdh"]), _np(out["sdh"]), dh, err, mode)
    _check_cols(_np(out["qdhT"]), _np(out["sdhT"]), dh, err, mode)
    _check_cols(_np(out["qaT"]), _np(out["saT"]), a, (ERR + g * 2.0 ** -23) * np.abs(a), mode)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_stays_in_its_groups(bad):
    M, I = 256, 384
    x, _ = _input(_h(M, I, 31), "bf16")
    ref = fg.swiglu_quant(x)
    y = x.clone()
    y[70, 130] = bad                      # a gate of the second channel block
    y[71, I + 3] = bad                    # an up value of the first
    got = fg.swiglu_quant(y)
    for codes, scales, width in ((0, 1, I // 128), (2, 3, 2 * I // 128)):
        same = torch.ones((M, width), dtype=torch.bool, device=dev())
        same[70, 1] = False
        same[71, 0 if codes == 0 else I // 128] = False
        assert torch.equal(got[codes].view(M, width, 128)[same], ref[codes].view(M, width, 128)[same])
        assert torch.equal(got[scales].t()[same], ref[scales].t()[same])
    da, _ = _input(_da(M, I, 10), "bf16")
    back = fg.swiglu_bwd(ref[2], ref[3], da)
    sh = ref[3].clone()
    sh[1, 70] = bad
    out = fg.swiglu_bwd(ref[2], sh, da)
    same = torch.ones((M, 2 * I // 128), dtype=torch.bool, device=dev())
    same[70, [1, 1 + I // 128]] = False
    assert torch.equal(out["qdh"].view(M, -1, 128)[same], back["qdh"].view(M, -1, 128)[same])
    assert torch.equal(out["sdh"].t()[same], back["sdh"].t()[same])
    # the other 128 tokens' and the other channels' groups along tokens
    ch = torch.ones(2 * I, dtype=torch.bool, device=dev())
    ch[128:256] = ch[I + 128:I + 256] = False
    assert torch.equal(out["qdhT"][:, 128:], back["qdhT"][:, 128:]) and torch.equal(out["qdhT"][ch], back["qdhT"][ch])
    assert torch.equal(out["qaT"][:, 128:], back["qaT"][:, 128:]) and torch.equal(out["qaT"][ch[:I]], back["qaT"][ch[:I]])
    assert fg.fp8_get_status() == fg.FP8_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [1, 31, 200])
def test_backward_by_rows_in_use_and_strided(M, dtype):
    """Without outputs along tokens: the bits of the full call's rows, rows behind those in use neither read
    nor written, outputs in slices of wider buffers."""
    I = 384
    q, s, h = _checkpoint(256, I, 17)
    da, dv = _input(_da(256, I, 11), dtype, pad=8)
    full = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh", "qdh", "qaT"))
    q, s = to_dev(q)[:M].contiguous(), to_dev(s)[:, :M].contiguous()
    for n in (None, 0, 1, M - 1, M, M + 5, -3):
        want = M if n is None else min(max(n, 0), M)
        dh, qdh = _junk((M, 2 * I + 16), torch.bfloat16), _junk((M, 2 * I + 32), torch.uint8)
        sdh = _junk((2 * I // 128, M), torch.float32)
        bad, qb, sb = da[:M].clone(), q.clone(), s.clone()
        bad[want:], qb[want:], sb[:, want:] = float("nan"), 0x7F, float("nan")
        fg.fp8_swiglu_bwd(qb, sb, bad, dh=dh[:, :2 * I], qdh=qdh[:, :2 * I], sdh=sdh,
                          n_rows=None if n is None else torch.tensor([n], dtype=torch.int32, device=dev()))
        assert torch.equal(dh[:want, :2 * I], full["dh"][:want]) and torch.equal(qdh[:want, :2 * I], full["qdh"][:want])
        assert torch.equal(sdh[:, :want], full["sdh"][:, :want])
        assert _untouched(dh[want:]) and _untouched(dh[:, 2 * I:]) and _untouched(qdh[want:])
        assert _untouched(qdh[:, 2 * I:]) and _untouched(sdh[:, want:])
    grad, mag = mlp.swiglu_grads(h, dv)
    _check_rows(_np(full["qdh"]), _np(full["sdh"]), grad, ERR * mag, fg.SCALE_FP32)
    assert fg.fp8_get_status() == fg.FP8_OK


def test_strided_outputs():
    """Codes written into slices of wider buffers, the rest of them untouched."""
    M, I = 128, 256
    x, _ = _input(_h(M, I, 11), "bf16")
    ref = fg.swiglu_quant(x)
    qa, qh = _junk((M, I + 32), torch.uint8), _junk((M, 2 * I + 48), torch.uint8)
    sa, sh = torch.empty_like(ref[1]), torch.empty_like(ref[3])
    fg.fp8_swiglu_quant(x, qa[:, :I], sa, qh[:, :2 * I], sh)
    assert torch.equal(qa[:, :I], ref[0]) and _untouched(qa[:, I:])
    assert torch.equal(qh[:, :2 * I], ref[2]) and _untouched(qh[:, 2 * I:])
    da, _ = _input(_da(M, I, 7), "bf16")
    full = fg.swiglu_bwd(ref[2], ref[3], da)
    qT, qd = _junk((2 * I, M + 64), torch.uint8), _junk((M, 2 * I + 16), torch.uint8)
    o = dict(full)
    o.update(qdhT=qT[:, :M], qdh=qd[:, :2 * I])
    fg.fp8_swiglu_bwd(qh[:, :2 * I], sh, da, **o)
    assert torch.equal(qT[:, :M], full["qdhT"]) and _untouched(qT[:, M:])
    assert torch.equal(qd[:, :2 * I], full["qdh"]) and _untouched(qd[:, 2 * I:])


def test_gradient_against_differences():
    """dh of sum(dA * a) against central differences of the FP64 forward."""
    M, I = 2, 128
    q, s, h = _checkpoint(M, I, 13)
    da, dv = _input(_da(M, I, 8), "fp32")
    dh = fg.swiglu_bwd(to_dev(q), to_dev(s), da, ("dh",))["dh"].float().cpu().numpy().astype(np.float64)
    eps = 1e-5
    ref = np.zeros_like(h)
    for j in range(2 * I):
        step = np.zeros_like(h)
        step[:, j] = eps
        diff = mlp.swiglu(h + step) - mlp.swiglu(h - step)
        ref[:, j] = (dv * diff).sum(1) / (2 * eps)
    _, mag = mlp.swiglu_grads(h, dv)
    # third derivatives of the SwiGLU are below |u| + 1: the differences are off by eps^2 of that
    tol = half_ulp_bf16(np.maximum(np.abs(ref), np.abs(dh))) + ERR * mag + 1e-9 * np.abs(dv).max() * (np.abs(h).max() + 1)
    assert np.all(np.abs(dh - ref) <= tol)


def test_other_stream_and_captured():
    M, I = 256, 256
    x, _ = _input(_h(M, I, 17), "bf16")
    da, _ = _input(_da(M, I, 9), "bf16")
    ref = fg.swiglu_quant(x)
    refb = fg.swiglu_bwd(ref[2], ref[3], da)
    outs = [torch.empty_like(t) for t in ref]
    outb = {n: torch.empty_like(t) for n, t in refb.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        fg.fp8_swiglu_quant(x, *outs)
        fg.fp8_swiglu_bwd(outs[2], outs[3], da, **outb)
    for _ in range(2):
        for t in (*outs, *outb.values()):
            t.view(torch.uint8).fill_(JUNK)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        assert all(torch.equal(outb[n], refb[n]) for n in refb)
    explicit = [torch.empty_like(t) for t in ref]
    torch.cuda.synchronize()
    fg.fp8_swiglu_quant(x, *explicit, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(explicit, ref))


def test_offsets_beyond_32_bits():
    """Rows whose codes lie more than 2^32 bytes into the buffers."""
    I, M = 128 * 64, 300_000                      # h: 9.8 GB, checkpoint 4.9 GB
    d = dev()
    h = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device=d)
    tail = _input(_h(300, I, 21), "bf16")[0]
    h[-300:] = tail
    qa, sa, qh, sh = fg.swiglu_quant(h)
    ref = fg.swiglu_quant(tail.contiguous())
    assert torch.equal(qa[-300:], ref[0]) and torch.equal(sa[:, -300:], ref[1])
    assert torch.equal(qh[-300:], ref[2]) and torch.equal(sh[:, -300:], ref[3])
    del h, qa
    da = torch.zeros((M, I), dtype=torch.bfloat16, device=d)
    dt = _input(_da(300, I, 10), "bf16")[0]
    da[-300:] = dt
    out = fg.swiglu_bwd(qh, sh, da, ("qdh",))
    refb = fg.swiglu_bwd(ref[2], ref[3], dt, ("qdh",))
    assert torch.equal(out["qdh"][-300:], refb["qdh"]) and torch.equal(out["sdh"][:, -300:], refb["sdh"])


def test_transposed_offsets_beyond_32_bits():
    """The last token blocks of tensors of more than 2^32 elements give the bits that they give alone."""
    I = 2048
    M = 2 ** 32 // (2 * I) + 256
    d = dev()
    q, s, _ = _checkpoint(256, I, 23)
    qh = torch.zeros((M, 2 * I), dtype=torch.uint8, device=d)
    sh = torch.ones((2 * I // 128, M), dtype=torch.float32, device=d)
    da = torch.zeros((M, I), dtype=torch.bfloat16, device=d)
    qh[-256:], sh[:, -256:] = to_dev(q), to_dev(s)
    tail = _input(_da(256, I, 12), "bf16")[0]
    da[-256:] = tail
    outputs = ("dh", "qdh", "qdhT", "qaT")
    got, ref = fg.swiglu_bwd(qh, sh, da, outputs), fg.swiglu_bwd(to_dev(q), to_dev(s), tail.contiguous(), outputs)
    for name in ("dh", "qdh"):
        assert torch.equal(got[name][-256:], ref[name]), name
    for name in ("sdh", "qdhT", "qaT"):
        assert torch.equal(got[name][:, -256:], ref[name]), name
    for name in ("sdhT", "saT"):
        assert torch.equal(got[name][-2:], ref[name]), name
    assert fg.fp8_get_status() == fg.FP8_OK
