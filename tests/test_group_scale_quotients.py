"""The group scales' two quotients, amax/448 and 448/amax, correctly rounded for
every FP32 maximum: on the CPU the steps that the quantizers take in place of
two divisions (a reciprocal, and one correction by the remainder), over all
2^23 significands of a binade; on a GPU the quantizer itself over the same
significands, and around the ends of the range in which those steps are taken
(2^-96 to 2^96; beyond it the quantizer divides).

A power of two in amax goes through every step unchanged as long as nothing
under- or overflows, so one binade stands for all of the range.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg


def _fma(a, b, c):
    """fl32(a * b + c) of float32 arrays, rounded once: the product is exact in float64, the sum's own
    rounding error is known (two-sum), and decides where the sum lies halfway between two float32."""
    p, c = a.astype(np.float64) * b.astype(np.float64), np.asarray(c, np.float32).astype(np.float64)
    s = p + c
    t = s - p
    e = (p - (s - t)) + (c - t)
    f = s.astype(np.float32)
    other = np.nextafter(f, np.where(s > f, np.inf, -np.inf).astype(np.float32))
    half = (s != f) & (np.abs(s - f) == np.abs(other.astype(np.float64) - s))
    up = np.maximum(f, other)
    down = np.minimum(f, other)
    return np.where(half & (e > 0), up, np.where(half & (e < 0), down, f))


def _significands():
    return (np.arange(2 ** 23, dtype=np.uint32) + 0x3F800000).view(np.float32)      # [1, 2)


def test_fma_against_integers():
    """The float32 FMA above against exact rational sums, halfway cases among them."""
    from fractions import Fraction
    rng = np.random.default_rng(0)
    a, b = (rng.integers(1 << 23, 1 << 24, 2000).astype(np.float32) for _ in range(2))
    c = (rng.integers(-(1 << 24), 1 << 24, 2000) * 2.0 ** rng.integers(0, 26, 2000)).astype(np.float32)
    c[:500] = -(a[:500].astype(np.float64) * b[:500]).astype(np.float32)             # cancellation
    c[500:600], a[500:600], b[500:600] = 2.0 ** 24, 1.0 + 2.0 ** -12, 1.0 - 2.0 ** -12   # just below halfway
    got = _fma(a, b, c)
    for x, y, z, g in zip(a, b, c, got):
        exact = Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))
        near = [np.float32(g), np.nextafter(g, np.float32(np.inf)), np.nextafter(g, np.float32(-np.inf))]
        best = min(abs(Fraction(float(n)) - exact) for n in near)
        assert abs(Fraction(float(g)) - exact) == best


def test_both_quotients_are_correctly_rounded_for_every_significand():
    amax, one = _significands(), np.float32(1.0)
    top = np.full_like(amax, 448.0)
    r448 = np.float32(1.0) / np.float32(448.0)
    q = amax * r448
    s = _fma(_fma(-top, q, amax), np.full_like(amax, r448), q)
    assert np.array_equal(s, amax / top)
    r = one / amax                                                                   # correctly rounded
    p = top * r
    inv = _fma(_fma(-amax, p, top), r, p)
    assert np.array_equal(inv, top / amax)
    # so close to it that the theorem's premises would be met they are not: this is shown by exhaustion alone
    ulp = np.spacing(amax / top).astype(np.float64)
    assert (np.abs(q - amax.astype(np.float64) / 448.0) / ulp).max() > 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["all significands", "ends of the range"])
def test_quantizer_scales_are_correctly_rounded_quotients(which):
    if which == "all significands":
        v = _significands()
    else:
        at = np.array([0x0F800000, 0x6F800000], np.int64)[:, None]                   # 2^-96, 2^96
        v = (at + np.arange(-200_000, 200_000)).astype(np.uint32).ravel().view(np.float32)
    dev = torch.device("cuda", 0)
    for part in np.array_split(v, 8):
        x = torch.zeros((part.size, 128), dtype=torch.float32, device=dev)
        x[:, 77] = torch.from_numpy(part).to(dev)
        q, s = fg.quant_act_1x128(x)
        want = torch.from_numpy((part / np.float32(448.0)).view(np.int32)).to(dev)
        assert torch.equal(s.view(torch.int32)[0], want)
        assert bool((q[:, 77] == 0x7E).all()) and int((q != 0).sum()) == part.size
    assert fg.fp8_get_status() == fg.FP8_OK
