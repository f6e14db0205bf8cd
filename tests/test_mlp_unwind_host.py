"""Argument checks of the gated-MLP kernels' failure-path self-tests (nothing is launched)."""
import pytest

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import build as fgbuild

P = [0x10000 * i for i in range(1, 16)]      # fake aligned device addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.load_library()


def test_swiglu_bwd_unwind_validation(lib):
    base = dict(qh=P[0], sh=P[1], da=P[2], dt=0, M=128, I=256, qdhT=P[3], sdhT=P[4])

    def call(**kw):
        return lib.fp8_selftest_swiglu_bwd_unwind(*dict(base, **kw).values(), None)
    assert call(dt=2) == fg.FP8_ERR_DTYPE
    for kw in (dict(M=0), dict(M=100), dict(I=0), dict(I=100), dict(M=-128)):
        assert call(**kw) == fg.FP8_ERR_SHAPE, kw
    for name in ("qh", "sh", "da", "qdhT", "sdhT"):
        assert call(**{name: 0}) == fg.FP8_ERR_NULL, name
        assert call(**{name: P[9] + 2}) == fg.FP8_ERR_ALIGN, name


def test_moe_mlp_few_unwind_validation(lib):
    base = dict(phase=1, x=P[0], dt=0, T=4, K=256, topk=P[1], w=P[2], k=2, G=8, W13=P[3], s13=P[4], W2=P[5], s2=P[6],
                I=128, N=384, out=P[7], od=0, ws=P[8], wsb=1 << 40)

    def call(**kw):
        return lib.fp8_selftest_moe_mlp_few_unwind(*dict(base, **kw).values(), None)
    for kw in (dict(phase=0), dict(phase=3), dict(dt=2), dict(od=2)):
        assert call(**kw) == fg.FP8_ERR_DTYPE, kw
    for kw in (dict(T=0), dict(T=129), dict(K=100), dict(wsb=16)):
        assert call(**kw) == fg.FP8_ERR_SHAPE, kw
    for name in ("x", "topk", "w", "W13", "s13", "W2", "s2", "out", "ws"):
        assert call(**{name: 0}) == fg.FP8_ERR_NULL, name
    assert call(ws=P[9] + 128) == fg.FP8_ERR_ALIGN
