"""The gated-MLP operators on the host: argument checks of the library and of
the Python calls (no GPU needed, nothing launched), and the FP64 oracle's own
formulas against differences and against a direct sum.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
import oracle
from fp8_fine_grained_x1_b200 import build as fgbuild
from oracle import mlp

P = [0x10000 * i for i in range(1, 16)]      # fake aligned device addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.load_library()


def test_swiglu_quant_validation(lib):
    def call(h=P[0], dt=0, M=100, I=256, ldh=512, qa=P[1], ldqa=256, sa=P[2], qh=P[3], ldqh=512, sh=P[4],
             n=0, mode=0):
        return lib.fp8_swiglu_quant(h, dt, M, I, ldh, qa, ldqa, sa, qh, ldqh, sh, n, mode, None)
    assert call(dt=2) == fg.FP8_ERR_DTYPE
    assert call(mode=2) == fg.FP8_ERR_DTYPE
    assert call(M=-1) == fg.FP8_ERR_SHAPE
    for I in (0, -128, 100, 1 << 30):
        assert call(I=I, ldh=1 << 31, ldqa=1 << 31, ldqh=1 << 31) == fg.FP8_ERR_SHAPE
    assert call(ldh=511) == fg.FP8_ERR_SHAPE
    assert call(ldqa=255) == fg.FP8_ERR_SHAPE
    assert call(ldqh=256) == fg.FP8_ERR_SHAPE
    assert call(M=0, h=0, qa=0, sa=0, qh=0, sh=0) == fg.FP8_OK
    for name in ("h", "qa", "sa", "qh", "sh"):       # a checkpoint needs codes and scales
        assert call(**{name: 0}) == fg.FP8_ERR_NULL
    assert call(qh=0, sh=0, ldqh=0) in (fg.FP8_ERR_DEVICE, fg.FP8_OK)
    for name in ("h", "qa", "qh"):
        assert call(**{name: P[9] + 8}) == fg.FP8_ERR_ALIGN
    for name in ("sa", "sh", "n"):
        assert call(**{name: P[9] + 2}) == fg.FP8_ERR_ALIGN
    assert call(ldh=516) == fg.FP8_ERR_ALIGN
    assert call(ldqa=264) == fg.FP8_ERR_ALIGN
    assert call() in (fg.FP8_ERR_DEVICE, fg.FP8_OK) if not torch.cuda.is_available() else True


def test_swiglu_bwd_validation(lib):
    base = dict(qh=P[0], ldqh=512, sh=P[1], da=P[2], dt=0, ldda=256, M=128, I=256, dh=P[3], lddh=512,
                qdh=P[4], ldqdh=512, sdh=P[5], qdhT=P[6], ldqdhT=128, sdhT=P[7], qaT=P[8], ldqaT=128,
                saT=P[9], n=0, mode=0)

    def call(**kw):
        return lib.fp8_swiglu_bwd(*dict(base, **kw).values(), None)
    assert call(dt=3) == fg.FP8_ERR_DTYPE
    assert call(M=100, ldqdhT=128) == fg.FP8_ERR_SHAPE          # whole groups along tokens
    none_t = dict(qdhT=0, sdhT=0, ldqdhT=0, qaT=0, saT=0, ldqaT=0)
    if not torch.cuda.is_available():
        assert call(M=100, **none_t) == fg.FP8_ERR_DEVICE       # rows alone may be ragged
    for kw in (dict(I=200), dict(I=0), dict(ldqh=256), dict(ldda=128), dict(lddh=511), dict(ldqdh=256),
               dict(ldqdhT=127), dict(ldqaT=64), dict(M=-128)):
        assert call(**kw) == fg.FP8_ERR_SHAPE, kw
    assert call(M=0, qh=0) == fg.FP8_OK
    for name in ("qh", "sh", "da", "qdh", "sdh", "qdhT", "sdhT", "qaT", "saT"):
        assert call(**{name: 0}) == fg.FP8_ERR_NULL, name
    assert call(dh=0, qdh=0, sdh=0, **none_t) == fg.FP8_ERR_NULL      # nothing wanted
    for name in ("qh", "da", "dh", "qdh", "qdhT", "qaT"):
        assert call(**{name: P[10] + 8}) == fg.FP8_ERR_ALIGN, name
    for kw in (dict(ldqh=520), dict(ldda=260), dict(lddh=516), dict(ldqdh=520), dict(ldqdhT=136),
               dict(ldqaT=136), dict(sdhT=P[10] + 1), dict(n=P[10] + 2)):
        assert call(**kw) == fg.FP8_ERR_ALIGN, kw


def test_moe_mlp_few_validation(lib):
    base = dict(x=P[0], dt=0, T=4, K=256, ldx=256, topk=P[1], w=P[2], k=2, G=8, W13=P[3], s13=P[4], W2=P[5],
                s2=P[6], I=128, N=384, out=P[7], od=0, ldo=384, ws=P[8], wsb=1 << 40, mode=0)

    def call(**kw):
        return lib.fp8_moe_mlp_few(*dict(base, **kw).values(), None)
    need = fg.fp8_moe_mlp_few_workspace_bytes(4, 2, 8, 256, 128, 384)
    assert need > 0
    for kw in (dict(dt=2), dict(od=2), dict(mode=2)):
        assert call(**kw) == fg.FP8_ERR_DTYPE
    for kw in (dict(T=-1), dict(T=fg.MOE_FEW_MAX_TOKENS + 1), dict(k=0), dict(k=129), dict(G=0), dict(G=1025),
               dict(K=200), dict(K=0), dict(I=64), dict(I=0), dict(N=100), dict(N=0), dict(ldx=128),
               dict(ldo=256), dict(wsb=need - 1), dict(G=1024, I=1 << 21), dict(G=1024, N=1 << 22, ldo=1 << 22)):
        assert call(**kw) == fg.FP8_ERR_SHAPE, kw
    assert call(T=0, x=0, topk=0, ws=0, wsb=0) == fg.FP8_OK
    for name in ("x", "topk", "w", "W13", "s13", "W2", "s2", "out", "ws"):
        assert call(**{name: 0}) == fg.FP8_ERR_NULL, name
    for name, off in (("x", 8), ("W13", 8), ("W2", 8), ("out", 8), ("ws", 128), ("topk", 2), ("w", 2), ("s13", 2),
                      ("s2", 2)):
        assert call(**{name: P[10] + off}) == fg.FP8_ERR_ALIGN, name
    assert call(ldx=260) == fg.FP8_ERR_ALIGN and call(ldo=388) == fg.FP8_ERR_ALIGN
    for bad in ((129, 2, 8, 256, 128, 384), (4, 0, 8, 256, 128, 384), (4, 2, 8, 250, 128, 384)):
        assert fg.fp8_moe_mlp_few_workspace_bytes(*bad) == 0


def test_python_calls_refuse_host_tensors_and_wrong_layouts(lib):
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    h = torch.zeros((128, 512), dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        fg.swiglu_quant(h)
    with pytest.raises(ValueError, match="CUDA"):
        fg.swiglu_bwd(torch.zeros((128, 512), dtype=u8), torch.zeros((4, 128)), torch.zeros((128, 256)))
    with pytest.raises(ValueError, match="CUDA"):
        fg.moe_mlp_few(h, torch.zeros((128, 2), dtype=torch.int32), torch.zeros((128, 2)),
                       torch.zeros((4, 256, 512), dtype=u8), torch.zeros((4, 2, 4)),
                       torch.zeros((4, 512, 128), dtype=u8), torch.zeros((4, 4, 1)))

    class Fake:      # what the checks look at, without a device
        def __init__(self, shape, dtype, stride=None, cont=True, dev=0):
            self.shape, self.dtype, self.device = torch.Size(shape), dtype, f"cuda:{dev}"
            self._st, self._c, self._d = stride or (shape[-1], 1), cont, dev

        def get_device(self):
            return self._d

        def dim(self):
            return len(self.shape)

        def stride(self, i=None):
            return self._st if i is None else self._st[i]

        def is_contiguous(self):
            return self._c

        def data_ptr(self):
            return 64
    assert fg._rows(Fake((4, 8), u8), "q", u8, (4, 8), 0) == 8
    assert fg._rows(Fake((4, 8), u8, (24, 1), False), "q", u8, (4, 8), 0) == 24
    assert fg._flat(Fake((4, 8), u8), "q", u8, (4, 8), 0) == 64
    for check in (fg._rows, fg._flat):
        with pytest.raises(TypeError):
            check(Fake((4, 8), f32), "q", u8, (4, 8), 0)
        with pytest.raises(ValueError, match="shape"):
            check(Fake((4, 9), u8), "q", u8, (4, 8), 0)
        with pytest.raises(ValueError, match="stride"):
            check(Fake((4, 8), u8, (1, 4), False), "q", u8, (4, 8), 0)
        with pytest.raises(ValueError, match="device"):
            check(Fake((4, 8), u8), "q", u8, (4, 8), 1)
        with pytest.raises(ValueError, match="device"):
            check(Fake((4, 8), u8, dev=-1), "q", u8, (4, 8), -1)
    with pytest.raises(ValueError, match="stride"):
        fg._flat(Fake((4, 8), u8, (24, 1), False), "q", u8, (4, 8), 0)
    with pytest.raises(ValueError, match="together"):
        fg._pair(h, None, "qh and sh")


def test_oracle_gradient_is_the_derivative():
    rng = np.random.default_rng(0)
    h, da = rng.normal(0, 3, (3, 16)), rng.normal(0, 1, (3, 8))
    dh, mag = mlp.swiglu_grads(h, da)
    eps = 1e-5
    for j in range(16):
        step = np.zeros_like(h)
        step[:, j] = eps
        num = (da * (mlp.swiglu(h + step) - mlp.swiglu(h - step))).sum(1) / (2 * eps)
        assert np.allclose(num, dh[:, j], rtol=1e-6, atol=1e-8)
    assert np.all(np.abs(dh) <= mag * (1 + 1e-12))
    assert mlp.swiglu(np.array([[-1e4, 2.0], [0.0, 5.0]])).tolist() == [[-0.0], [0.0]]


def test_oracle_moe_mlp_against_a_direct_sum():
    rng = np.random.default_rng(1)
    T, k, G, K, I, N = 3, 2, 3, 256, 128, 128
    xq, sx = oracle.quant_act_1x128(rng.normal(0, 1, (T, K)).astype(np.float32))
    w13 = np.empty((G, 2 * I, K), np.uint8)
    s13 = np.empty((G, 2 * I // 128, K // 128), np.float32)
    w2, s2 = np.empty((G, N, I), np.uint8), np.empty((G, N // 128, I // 128), np.float32)
    for e in range(G):
        w13[e], s13[e] = oracle.quant_w_128x128(rng.normal(0, 0.06, (2 * I, K)).astype(np.float32))
        w2[e], s2[e] = oracle.quant_w_128x128(rng.normal(0, 0.09, (N, I)).astype(np.float32))
    topk = np.array([[0, 2], [1, 1], [2, 0]], np.int32)
    w = rng.uniform(0, 1, (T, k)).astype(np.float32)
    out, tol = mlp.moe_mlp(xq, sx, topk, w, w13, s13, w2, s2, oracle.SCALE_FP32, 1e-9)
    for t in range(T):
        ref = np.zeros(N)
        for j in range(k):
            e = topk[t, j]
            x = mlp.decode(xq[t]) * np.repeat(sx[:, t].astype(np.float64), 128)
            h = mlp.decode_128x128(w13[e], s13[e]) @ x
            a = mlp.swiglu(h[None])[0].astype(np.float32)
            qa, sa = oracle.quant_act_1x128(a[None])
            ref += w[t, j] * (mlp.decode_128x128(w2[e], s2[e]) @ (mlp.decode(qa[0]) * np.repeat(sa[:, 0].astype(np.float64), 128)))
        assert np.all(np.abs(out[t] - ref) <= tol[t] + 1e-6 * np.abs(ref).max())
        assert tol[t].max() <= 0.05 * np.abs(ref).max()


def test_code_checks_see_a_wrong_code():
    v = np.random.default_rng(2).normal(0, 1, (4, 128)).astype(np.float32)
    q, s = oracle.quant_act_1x128(v)
    S = np.repeat(s.astype(np.float64).T, 128, axis=1)
    assert mlp.code_excess(q, S, v, 1e-7 * np.abs(v)) <= 0.0
    assert mlp.scale_error(s, np.abs(v).max(1)[None], 0.0, oracle.SCALE_FP32) <= 2.0 ** -22
    wrong = q.copy()
    wrong[2, 5] ^= 1
    assert mlp.code_excess(wrong, S, v, 1e-7 * np.abs(v)) > 0.0
    assert mlp.scale_error(s * 1.001, np.abs(v).max(1)[None], 0.0, oracle.SCALE_FP32) > 2.0 ** -22
    assert mlp.scale_error(s, np.abs(v).max(1)[None], 0.0, oracle.SCALE_POW2) == float("inf")
