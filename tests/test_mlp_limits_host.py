"""Limits and sizes that include/fp8fg.h states for the gated-MLP calls, against
the library (no GPU needed, nothing launched)."""
import os
import re

import pytest

import fp8_fine_grained_x1_b200 as fg
from fp8_fine_grained_x1_b200 import build as fgbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x10000 * i for i in range(1, 16)]      # fake aligned device addresses: never dereferenced
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    fgbuild.build()
    return fg.load_library()


def _comment(function):
    """The header's comment above a function, its lines joined."""
    text = open(os.path.join(ROOT, "include", "fp8fg.h")).read()
    above = text[:re.search(r"^int(64_t)? " + function + r"\(", text, re.M).start()]
    return re.sub(r"\s*\n \*\s*", " ", above[above.rindex("/*"):])


@pytest.mark.parametrize("blocks", [1, 8, 1 << 10])
def test_rows_times_channels_are_limited_as_documented(lib, blocks):
    """ceil(M / 16) * I / 128 <= 2^31 - 1, in both calls."""
    for name in ("fp8_swiglu_quant", "fp8_swiglu_bwd"):
        assert "ceil(M / 16) * (I / 128) <= 2^31 - 1" in _comment(name), name
    I = 128 * blocks
    most = min(MAX, MAX // blocks * 16)
    for M, ok in ((most, True), (most + 1, False)):
        if M > MAX:
            continue
        fwd = lib.fp8_swiglu_quant(P[0] + 8, 0, M, I, 2 * I, P[1], I, P[2], 0, 0, 0, 0, 0, None)
        bwd = lib.fp8_swiglu_bwd(P[0] + 8, 2 * I, P[1], P[2], 0, I, M, I, P[3], 2 * I, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, None)
        want = fg.FP8_ERR_ALIGN if ok else fg.FP8_ERR_SHAPE        # (a misaligned input: nothing is ever launched)
        assert fwd == bwd == want, M


@pytest.mark.parametrize("T,k,G,K,I,N", [(128, 8, 256, 7168, 2048, 7168), (128, 8, 32, 7168, 2048, 7168),
                                         (1, 8, 32, 7168, 2048, 7168), (33, 2, 5, 512, 256, 640), (17, 128, 1024, 128, 128, 128)])
def test_workspace_is_as_large_as_documented(T, k, G, K, I, N):
    """min(T k, G) * I * (8 T + Tp), Tp = T rounded up to 16, and beside it 311,296 T for the parts of tiles, x's codes,
    and tables that are small next to these: 4 bytes per expert and token, per 128 channels and token."""
    assert "min(T k, G) * I * (8 T + T')" in _comment("fp8_moe_mlp_few_workspace_bytes")
    A, Tp = min(T * k, G), (T + 15) // 16 * 16
    main = A * I * (8 * T + Tp) + 311_296 * T + T * K
    small = 4 + 4 * A + 4 * G * Tp + 4 * (K // 128) * Tp + 4 * A * (I // 128) * Tp + 9 * 256
    got = fg.fp8_moe_mlp_few_workspace_bytes(T, k, G, K, I, N)
    assert main <= got <= main + small
