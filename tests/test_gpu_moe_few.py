"""fp8_moe_mlp_few on the GPU against an FP64 MoE MLP on the same quantized
operands.

Tolerance: every block-scaled product within REL = 1e-4 of its sum of
magnitudes (the GEMMs' own bound), activations whose E4M3 rounding such an
error can flip a whole step off, BF16 outputs half a BF16 step more.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_x1_b200 as fg
import oracle
from fp8_fine_grained_x1_b200 import synth
from oracle import mlp

from gpu_util import REL_TOL, dev, half_ulp_bf16, to_dev

pytestmark = pytest.mark.gpu


def _weights(G, N, K, seed, mode):
    rng = np.random.default_rng(seed)
    q, s = np.empty((G, N, K), np.uint8), np.empty((G, N // 128, K // 128), np.float32)
    for e in range(G):
        q[e], s[e] = oracle.quant_w_128x128(rng.normal(0, K ** -0.5, (N, K)).astype(np.float32), mode)
    return q, s


def _case(T, k, G, K, I, N, seed=0, mode=fg.SCALE_FP32, dtype="bf16"):
    x = torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (T, K)).astype(np.float32))
    x[:, ::97] *= 50.0
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    topk = synth.zipf_topk_routing(max(T, 1), G, k, seed=seed + 1)[:T].numpy().astype(np.int32)
    w = np.random.default_rng(seed + 2).uniform(0.05, 1.0, (T, k)).astype(np.float32)
    w13, s13 = _weights(G, 2 * I, K, seed + 3, mode)
    w2, s2 = _weights(G, N, I, seed + 4, mode)
    return x, topk, w, w13, s13, w2, s2


def _run(case, out_dtype=None, mode=fg.SCALE_FP32, x=None):
    x0, topk, w, w13, s13, w2, s2 = case
    return fg.moe_mlp_few(x0.to(dev()) if x is None else x, to_dev(topk), to_dev(w), to_dev(w13), to_dev(s13),
                          to_dev(w2), to_dev(s2), out_dtype, mode)


def _reference(case, mode=fg.SCALE_FP32):
    x, topk, w, w13, s13, w2, s2 = case
    src = x.view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()
    xq, sx = oracle.quant_act_1x128(src, mode)
    return mlp.moe_mlp(xq, sx, topk, w, w13, s13, w2, s2, mode, REL_TOL)


def _check(got, case, mode=fg.SCALE_FP32):
    ref, tol = _reference(case, mode)
    g = got.float().cpu().numpy().astype(np.float64)
    if got.dtype == torch.bfloat16:
        tol = tol + half_ulp_bf16(np.maximum(np.abs(ref), np.abs(g)))
    else:
        tol = tol + np.abs(ref) * 2.0 ** -22
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - ref)[bad].max()))


@pytest.mark.parametrize("T,k,G,K,I,N", [
    (1, 1, 1, 128, 128, 128),          # one unit of work
    (1, 8, 32, 512, 256, 512),
    (3, 4, 6, 512, 256, 384),          # an odd number of 128-column blocks
    (15, 2, 5, 384, 128, 256), (16, 3, 7, 256, 384, 128), (17, 2, 4, 256, 256, 640),
    (33, 8, 40, 256, 128, 256), (64, 4, 8, 1024, 128, 256), (65, 2, 3, 256, 256, 256),
    (100, 8, 16, 256, 256, 256), (128, 6, 9, 384, 256, 384),
])
def test_against_fp64(T, k, G, K, I, N):
    case = _case(T, k, G, K, I, N, seed=T + G)
    got = _run(case)
    assert fg.fp8_get_status() == fg.FP8_OK
    _check(got, case)
    assert torch.equal(got, _run(case))                  # fixed order of sums


@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("dtype,out,mode", [("fp32", torch.float32, fg.SCALE_FP32),
                                            ("bf16", torch.float32, fg.SCALE_POW2),
                                            ("fp32", torch.bfloat16, fg.SCALE_POW2)])
def test_types_and_scale_modes(T, dtype, out, mode):
    case = _case(T, 3, 6, 384, 256, 384, seed=T, mode=mode, dtype=dtype)
    _check(_run(case, out, mode), case, mode)


def test_full_width_layer():
    """The MoE workload's layer (hidden 7168, expert width 2048) on a few of its experts."""
    case = _case(9, 2, 3, synth.HIDDEN, synth.EXPERT_HIDDEN, synth.HIDDEN, seed=2)
    _check(_run(case), case)


def test_strides_and_no_write_outside():
    case = _case(6, 2, 4, 256, 128, 256, seed=3)
    x, topk, w, w13, s13, w2, s2 = case
    wide = torch.full((6, 512), float("nan"), dtype=torch.bfloat16, device=dev())
    wide[:, 64:320] = x.to(dev())
    out = torch.full((6, 264), 7.0, dtype=torch.bfloat16, device=dev())
    n = fg.fp8_moe_mlp_few_workspace_bytes(6, 2, 4, 256, 128, 256)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device=dev())
    fg.fp8_moe_mlp_few(wide[:, 64:320], to_dev(topk), to_dev(w), to_dev(w13), to_dev(s13), to_dev(w2), to_dev(s2),
                       out[:, :256], ws[:n])
    assert torch.equal(out[:, :256], _run(case))
    assert bool((out[:, 256:] == 7.0).all()) and bool((ws[n:] == 0x5A).all())


def test_repeated_expert_zero_weight_and_invalid_ids():
    case = list(_case(5, 4, 6, 256, 128, 256, seed=4))
    topk, w = case[1], case[2]
    topk[0] = 3                       # one expert four times: the sum of its weights
    w[1, 2] = 0.0                     # adds nothing
    w[2] = 0.0                        # a token of zero weights: exactly zero
    got = _run(case)
    _check(got, case)
    assert bool((got[2] == 0).all())
    assert fg.fp8_get_status() == fg.FP8_OK
    bad = list(case)
    bad[1] = topk.copy()
    bad[1][3] = [-1, 6, 2 ** 31 - 1, topk[3, 3]]
    got = _run(bad)
    assert fg.fp8_get_status() == fg.FP8_ERR_SHAPE
    _check(got, bad)                  # the other pairs count as ever
    bad[1] = np.full_like(topk, -1)
    got = _run(bad)
    assert fg.fp8_get_status() == fg.FP8_ERR_SHAPE
    assert bool((got == 0).all())


def test_one_token_does_not_disturb_another():
    """A token of infinities (NaN out) leaves the others' bits alone, though they share every MMA."""
    case = list(_case(20, 2, 4, 256, 128, 256, seed=6))
    ref = _run(case)
    x = case[0].to(dev())
    x[7, :130] = float("inf")
    got = _run(case, x=x)
    keep = [t for t in range(20) if t != 7]
    assert torch.equal(got[keep], ref[keep])
    assert fg.fp8_get_status() == fg.FP8_OK
    # a row's result does not depend on who else is in the batch
    one = list(case)
    one[0], one[1], one[2] = case[0][3:4], case[1][3:4], case[2][3:4]
    _check(_run(one), one)


def test_captured_and_replayed_beside_another_call():
    """Two graphs with a workspace each, replayed at once on two streams."""
    runs = []
    for i in range(2):
        case = _case(4 + 30 * i, 2, 8, 512, 256, 512, seed=8 + i)
        t = [case[0].to(dev())] + [to_dev(a) for a in case[1:]]
        ref = _run(case)
        T = 4 + 30 * i
        out = torch.empty_like(ref)
        ws = torch.empty(fg.fp8_moe_mlp_few_workspace_bytes(T, 2, 8, 512, 256, 512), dtype=torch.uint8, device=dev())
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fg.fp8_moe_mlp_few(*t, out, ws)
        runs.append((g, s, out, ref, t, ws))
    for _ in range(20):
        for g, s, out, *_ in runs:
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    assert fg.fp8_get_status() == fg.FP8_OK
    for _, _, out, ref, *_ in runs:
        assert torch.equal(out, ref)


def test_no_tokens():
    case = _case(0, 2, 4, 256, 128, 256, seed=1)
    assert _run(case).shape == (0, 256)


@pytest.mark.parametrize("T", [5, 32, 33, 128])
def test_a_bad_expert_spoils_only_its_tokens(T):
    """NaN codes and infinite scales of one expert's weights reach the tokens routed to it, no other:
    though every expert's products are made with every token."""
    G, e = 6, 2
    case = list(_case(T, 2, G, 256, 256, 384, seed=T))
    case[1][0] = [e, 5]                           # picked by one token at least,
    case[1][T - 1] = [0, 1]                       # and not by all
    ref = _run(case)
    hit = torch.from_numpy((case[1] == e).any(1)).to(dev())
    assert bool(hit.any()) and not bool(hit.all())
    for i, bad in ((3, 0x7F), (4, np.inf), (5, 0x7F), (5, 0xFF), (6, np.inf), (6, np.nan)):
        spoilt = list(case)
        spoilt[i] = case[i].copy()
        spoilt[i][e] = bad
        got = _run(spoilt)
        assert torch.equal(got[~hit], ref[~hit]), i
        assert not bool(torch.isfinite(got[hit]).any()), i
    assert fg.fp8_get_status() == fg.FP8_OK


@pytest.mark.parametrize("T,k,G,K,I,N", [(1, 1, 3, 4096, 128, 128), (30, 3, 4, 2048, 128, 256),
                                         (32, 4, 5, 256, 2048, 128), (87, 1, 4, 2048, 128, 1152),
                                         (128, 2, 3, 256, 2048, 128)])
def test_few_tiles_in_many_parts(T, k, G, K, I, N):
    """Long products of few tiles, whose parts many CTAs hold; all tokens of an expert in one tile."""
    case = _case(T, k, G, K, I, N, seed=T + K)
    got = _run(case)
    _check(got, case)
    assert torch.equal(got, _run(case)) and fg.fp8_get_status() == fg.FP8_OK


@pytest.mark.parametrize("T,out", [(3, torch.bfloat16), (40, torch.float32), (128, torch.bfloat16)])
def test_many_output_columns(T, out):
    """More output tiles than CTAs: whole tiles are rounded and stored by the CTA that added them up."""
    case = _case(T, 2, 3, 128, 128, 128 * 601, seed=T)
    got = _run(case, out)
    _check(got, case)
    assert torch.equal(got, _run(case, out))


@pytest.mark.parametrize("T", [2, 33])
def test_most_experts_and_picks(T):
    """1024 experts, 128 picks a token."""
    case = _case(T, 128, 1024, 128, 128, 128, seed=T)
    _check(_run(case), case)
    assert fg.fp8_get_status() == fg.FP8_OK


@pytest.mark.parametrize("T", [1, 40])
def test_weights_past_32_bit_offsets(T):
    """Experts whose weights lie past 2^32 bytes give the bits of the same experts side by side."""
    G, K, I, N = 400, synth.HIDDEN, 1024, synth.HIDDEN
    pick = [0, 250, G - 1]
    x, _, _, w13, s13, w2, s2 = _case(T, 1, len(pick), K, I, N, seed=T)
    assert (pick[1] + 1) * 2 * I * K > 2 ** 31 and pick[2] * 2 * I * K > 2 ** 32
    topk = np.stack([np.arange(3, dtype=np.int32)] * T)
    w = np.random.default_rng(T).uniform(0.1, 1.0, topk.shape).astype(np.float32)
    near = _run((x, topk, w, w13, s13, w2, s2))
    far = []
    for a in (w13, s13, w2, s2):
        t = torch.empty((G,) + a.shape[1:], dtype=torch.uint8 if a.dtype == np.uint8 else torch.float32, device=dev())
        t.fill_(0x7F if a.dtype == np.uint8 else float("nan"))
        for i, e in enumerate(pick):
            t[e] = to_dev(a[i])
        far.append(t)
    got = fg.moe_mlp_few(x.to(dev()), to_dev(np.array(pick, np.int32)[topk]), to_dev(w), *far)
    assert torch.equal(got, near)
    assert fg.fp8_get_status() == fg.FP8_OK
