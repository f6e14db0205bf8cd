"""CPU oracle of the gated MLP's operators -- TEST INFRASTRUCTURE ONLY
(imported by tests/ only; shares no code with the CUDA path).

Plain FP64 formulas: the SwiGLU, its gradient, the decode of quantized
operands, the MoE MLP of a few tokens, and how far E4M3 codes may lie from
FP64 values that the GPU had in FP32.
"""
from __future__ import annotations

import numpy as np

import oracle


def sigmoid(g):
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    """h [M, 2I] -> silu(gate) * up [M, I]."""
    g, u = np.split(np.asarray(h, np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grads(h, da):
    """dH [M, 2I] for dA [M, I], and the scale of its FP32 error: FP32 rounding
    errors are relative to |dA u| s (1 + |g|) for the gate half (the sum
    1 + g (1 - s) can cancel) and to |dU| for the up half."""
    g, u = np.split(np.asarray(h, np.float64), 2, axis=1)
    da = np.asarray(da, np.float64)
    s = sigmoid(g)
    dg = da * u * s * (1.0 + g * (1.0 - s))
    du = da * g * s
    mag = np.concatenate((np.abs(da * u) * s * (1.0 + np.abs(g)), np.abs(du)), axis=1)
    return np.concatenate((dg, du), axis=1), mag


_VALUES = None


def decode(q):
    """Values of E4M3 codes."""
    global _VALUES
    if _VALUES is None:
        _VALUES = np.array([oracle.e4m3_decode(b) for b in range(256)])
    return _VALUES[np.asarray(q, np.uint8)]


def decode_1x128(q, s):
    """codes [M, C], scales [C/128, M] -> values [M, C]."""
    return decode(q) * np.repeat(np.asarray(s, np.float64).T, 128, axis=1)


def decode_128x128(q, s):
    return decode(q) * np.repeat(np.repeat(np.asarray(s, np.float64), 128, 0), 128, 1)


def e4m3_step(v):
    """Spacing of E4M3 values at |v| (subnormals included)."""
    a = np.maximum(np.abs(np.asarray(v, np.float64)), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(a)) - 3.0)


def code_excess(q, s, v, err):
    """How far codes q with group scales s (broadcast to q's shape) lie beyond
    half an E4M3 step from FP64 values v known to within err: <= 0 is right.
    Returns max over elements of (|code - v/s| - half step) / 1 in code units,
    after allowing err/s and two FP32 roundings (of v*inv and of inv)."""
    c = decode(q)
    x = np.asarray(v, np.float64) / s
    half = 0.5 * e4m3_step(np.minimum(np.maximum(np.abs(c), np.abs(x)), 448.0))
    allow = half + np.asarray(err, np.float64) / s + np.abs(x) * 2.0 ** -22
    return float(np.max(np.abs(c - np.clip(x, -448.0, 448.0)) - allow)) if c.size else 0.0


def scale_error(s, amax, err, mode):
    """Relative error of scales s of groups with FP64 max-abs `amax` known to
    within err (FP32 mode), or 0 / inf as POW2 scales are the least power of
    two whose 448-fold covers amax (either neighbour within err of a border)."""
    s, amax, err = (np.asarray(x, np.float64) for x in (s, amax, err))
    zero = amax == 0
    if mode == oracle.SCALE_FP32:
        ref = np.where(zero, 1.0, np.maximum(amax / 448.0, 2.0 ** -126))
        return float(np.max((np.abs(s - ref) - np.where(zero, 0.0, err / 448.0)) / ref)) if s.size else 0.0
    lo, hi = (np.exp2(np.maximum(np.ceil(np.log2(np.maximum(a, 2.0 ** -140) / 448.0)), -126.0))
              for a in (np.maximum(amax - err, 0.0), amax + err))
    ok = np.where(zero, s == 1.0, (s == lo) | (s == hi))
    return 0.0 if ok.all() else float("inf")


def moe_mlp(xq, sx, topk, weights, w13, s13, w2, s2, mode, rel):
    """FP64 MoE MLP on quantized operands (xq [T, K], sx [K/128, T]).  Returns
    (out [T, N], tol [T, N]): tol covers products off by `rel` of their sums of
    magnitudes, and activations whose E4M3 rounding such an error can flip (a
    whole step)."""
    T = xq.shape[0]
    x = decode_1x128(xq, sx)
    N, I = w2.shape[1:]
    out, tol = np.zeros((T, N)), np.zeros((T, N))
    for e in range(w13.shape[0]):
        hit = topk == e
        t = np.flatnonzero(hit.any(1))
        if not t.size:
            continue
        w = (np.asarray(weights, np.float64) * hit).sum(1)[t]
        W1, W2 = decode_128x128(w13[e], s13[e]), decode_128x128(w2[e], s2[e])
        h, mag = x[t] @ W1.T, np.abs(x[t]) @ np.abs(W1).T
        g, u = np.split(h, 2, axis=1)
        mg, mu = np.split(rel * mag, 2, axis=1)
        a = swiglu(h)
        # |d silu/dg| <= 1.1; the second-order term is negligible against rel
        err = 1.1 * mg * np.abs(u) + mu * np.abs(g * sigmoid(g)) + np.abs(a) * 2.0 ** -20
        grp = np.abs(a).reshape(len(t), I // 128, 128)
        gerr = err.reshape(len(t), I // 128, 128)
        amax, aerr = grp.max(2), gerr.max(2)
        if mode == oracle.SCALE_FP32:
            s = np.where(amax == 0, 1.0, amax / 448.0)
        else:
            s = np.where(amax == 0, 1.0, np.exp2(np.maximum(np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0)), -126.0)))
        S = np.repeat(s, 128, axis=1)
        v = a / S
        step = e4m3_step(np.minimum(np.abs(v), 448.0))
        c = np.clip(np.round(v / step) * step, -448.0, 448.0)
        # how far v is from the nearest rounding border, against its error and its scale's
        verr = err / S + np.abs(v) * np.repeat(aerr / np.maximum(amax, 1e-300), 128, axis=1)
        flip = (0.5 * step - np.abs(v - c)) <= verr
        serr = np.repeat(aerr / np.maximum(amax, 1e-300), 128, axis=1)     # relative error of the scale
        if mode == oracle.SCALE_POW2:                                      # a scale that err can double
            lo = np.exp2(np.ceil(np.log2(np.maximum(amax - aerr, 1e-300) / 448.0)))
            hi = np.exp2(np.ceil(np.log2(np.maximum(amax + aerr, 1e-300) / 448.0)))
            flip |= np.repeat(lo != hi, 128, axis=1)
            serr = np.zeros_like(serr)
        aerr_q = S * (np.where(flip, step, 0.0) + np.abs(c) * serr)
        y = (c * S) @ W2.T
        ymag = np.abs(c * S) @ np.abs(W2).T
        out[t] += w[:, None] * y
        tol[t] += np.abs(w)[:, None] * (rel * ymag + aerr_q @ np.abs(W2).T)
    return out, tol
