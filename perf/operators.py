"""Measured cases of the gated-MLP operators: the FP8 SwiGLU forward with its
8-bit checkpoint, its backward from that checkpoint, and the whole MoE MLP for
a few tokens.

`own` False computes each operator in plain torch (FP32 elementwise work and
products, one rounding where the operator defines one); `own` True makes the
library calls.  E4M3 results come back as float8_e4m3fn tensors (the values of
the codes) next to their FP32 group scales.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
HIDDEN = 7168            # model width of the MoE workload
EXPERT_HIDDEN = 2048     # expert width
DENSE_HIDDEN = 9216      # gated dense MLP: gate and up together are the 18432 columns of the dense Fprop workload


def listed():
    """Real uses, smallest to largest, for each operator."""
    return [
        # forward: a decode-sized batch through a small expert, where latency is all
        dict(name="fwd_7x512", op="fwd", M=7, I=512, dtype="fp32", keep=True, rows=1.0),
        # forward without a checkpoint (inference), a ragged number of tokens
        dict(name="fwd_1000x2048_infer", op="fwd", M=1000, I=EXPERT_HIDDEN, dtype="bf16", keep=False, rows=1.0),
        # forward of the dense MLP, 4096 tokens, checkpoint kept
        dict(name="fwd_4096x9216", op="fwd", M=4096, I=DENSE_HIDDEN, dtype="bf16", keep=True, rows=1.0),
        # forward over the expert rows of the MoE workload: 16384 tokens x top-8, groups padded to 128,
        # in buffers sized for the worst padding (rows behind the last group are left alone)
        dict(name="fwd_moe_135168x2048", op="fwd", M=135168, I=EXPERT_HIDDEN, dtype="bf16", keep=True, rows=0.985),
        # backward, one 128-token tile of a small expert, FP32 gradients
        dict(name="bwd_128x512", op="bwd", M=128, I=512, dtype="fp32", outs="qta", rows=1.0),
        # backward where only the input gradient is wanted (frozen weights), a ragged number of tokens
        dict(name="bwd_1000x2048_dgrad", op="bwd", M=1000, I=EXPERT_HIDDEN, dtype="bf16", outs="qd", rows=1.0),
        # backward of the dense MLP with every operand of the two Wgrads and the Dgrad
        dict(name="bwd_4096x9216", op="bwd", M=4096, I=DENSE_HIDDEN, dtype="bf16", outs="qta", rows=1.0),
        # backward over the expert rows of the MoE workload
        dict(name="bwd_moe_135168x2048", op="bwd", M=135168, I=EXPERT_HIDDEN, dtype="bf16", outs="qta", rows=0.985),
        # one MoE layer, few tokens: small experts (latency), one token and a batch of the MoE workload's layer,
        # and the largest batch this form takes
        dict(name="few_3_small", op="few", T=3, k=4, G=6, K=512, I=256, N=512),
        dict(name="few_1", op="few", T=1, k=8, G=32, K=HIDDEN, I=EXPERT_HIDDEN, N=HIDDEN),
        dict(name="few_17", op="few", T=17, k=8, G=32, K=HIDDEN, I=EXPERT_HIDDEN, N=HIDDEN),
        dict(name="few_128", op="few", T=128, k=8, G=32, K=HIDDEN, I=EXPERT_HIDDEN, N=HIDDEN),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "bwd", "few"))
    if op == "few":
        K = 128 * _log(rng, 2, 56)
        N = rng.choice((K, 128 * _log(rng, 2, 56)))
        I = 128 * _log(rng, 1, 16)
        # no more weight bytes than the largest listed case
        G = max(4, min(_log(rng, 4, 256), 32 * 3 * HIDDEN * EXPERT_HIDDEN // (I * (2 * K + N))))
        return dict(op=op, T=_log(rng, 1, 128), k=rng.randint(1, min(8, G)), G=G, K=K, I=I, N=N)
    I = 128 * _log(rng, 1, 72)
    M = max(1, min(_log(rng, 1, 110000), 110000 * EXPERT_HIDDEN // I))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if dtype == "fp32":
        M = max(1, M // 4)
    rows = rng.choice((1.0, 1.0, rng.uniform(0.2, 1.0)))
    if op == "fwd":
        return dict(op=op, M=M, I=I, dtype=dtype, keep=rng.random() < 0.7, rows=rows)
    outs = rng.choice(("qta", "qt", "qd", "ta", "d"))
    if "t" in outs or "a" in outs:
        M = max(128, M // 128 * 128)     # the 128x1 groups run over whole blocks of 128 tokens
    return dict(op=op, M=M, I=I, dtype=dtype, outs=outs, rows=rows)


def _n_rows(case):
    """Rows in use: the last group ends on a multiple of 128 in a padded layout."""
    M = case["M"]
    if case["rows"] >= 1.0:
        return M
    n = int(M * case["rows"])
    return max(128, n // 128 * 128) if M >= 128 else max(1, n)


def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(shape, g, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _store_1x128(v):
    """FP32 [M, C] -> E4M3 codes (uint8) and FP32 scales [C/128, M]: how a cached activation comes into being."""
    M, C = v.shape
    g = v.view(M, C // 128, 128)
    amax = g.abs().amax(-1, keepdim=True).clamp_(min=1e-30)
    q = (g * (448.0 / amax)).clamp_(-448, 448).to(E4M3).view(M, C).view(torch.uint8)
    return q, (amax / 448.0).view(M, C // 128).t().contiguous()


def _store_128x128(w):
    """FP32 [N, K] -> E4M3 codes (uint8) and FP32 scales [N/128, K/128]: a weight quantized once."""
    N, K = w.shape
    b = w.view(N // 128, 128, K // 128, 128)
    amax = b.abs().amax((1, 3), keepdim=True).clamp_(min=1e-30)
    q = (b * (448.0 / amax)).clamp_(-448, 448).to(E4M3).view(N, K).view(torch.uint8)
    return q, (amax / 448.0).view(N // 128, K // 128)


def _weights(G, N, K, g):
    q = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((G, N // 128, K // 128), dtype=torch.float32, device="cuda")
    for e in range(G):
        q[e], s[e] = _store_128x128(_randn((N, K), g, 0.006 if K > 1024 else 0.05, torch.float32))
    return q, s


def _routing(T, k, G, g):
    """k distinct experts per token, Zipf(1.1) over the experts, softmaxed gate weights."""
    logp = -1.1 * torch.log(torch.arange(1, G + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((T, G), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    score, topk = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1)
    return topk.to(torch.int32).contiguous(), torch.softmax(score, 1).contiguous()


def prepare(case, seed):
    op = case["op"]
    if op == "few":
        T, k, G, K, I, N = (case[n] for n in ("T", "k", "G", "K", "I", "N"))
        g = _gen(seed, 3)
        x = torch.randn((T, K), generator=g, device="cuda")
        x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 50.0   # outlier channels
        topk, gate = _routing(T, k, G, g)
        w13, s13 = _weights(G, 2 * I, K, g)
        w2, s2 = _weights(G, N, I, g)
        return dict(case, x=x.to(torch.bfloat16), topk=topk, gate=gate, w13=w13, s13=s13, w2=w2, s2=s2,
                    out=torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), ws=None)
    M, I = case["M"], case["I"]
    g = _gen(seed, 1 if op == "fwd" else 2)
    u8 = dict(dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    n = _n_rows(case)
    st = dict(case, n=None if case["rows"] >= 1.0 else torch.tensor([n], dtype=torch.int32, device="cuda"))
    h = _randn((M, 2 * I), g, 2.0, torch.bfloat16 if op == "bwd" else _dtype(case))
    # buffers a training program keeps from step to step; rows behind the last group stay zero
    if op == "fwd":
        st.update(h=h, qa=torch.zeros((M, I), **u8), sa=torch.zeros((I // 128, M), **f32))
        if case["keep"]:
            st.update(qh=torch.zeros((M, 2 * I), **u8), sh=torch.zeros((2 * I // 128, M), **f32))
        return st
    qh, sh = _store_1x128(h.float())
    del h
    st.update(qh=qh, sh=sh, da=_randn((M, I), g, 1e-3, _dtype(case)))
    outs = case["outs"]
    if "d" in outs:
        st["dh"] = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device="cuda")
    if "q" in outs:
        st.update(qdh=torch.zeros((M, 2 * I), **u8), sdh=torch.zeros((2 * I // 128, M), **f32))
    if "t" in outs:
        st.update(qdhT=torch.zeros((2 * I, M), **u8), sdhT=torch.zeros((M // 128, 2 * I), **f32))
    if "a" in outs:
        st.update(qaT=torch.zeros((I, M), **u8), saT=torch.zeros((M // 128, I), **f32))
    return st


# ------------------------------------------------------------------ plain forms

_TINY = 1.75 * 2.0 ** -118       # below it amax/448 is no normal FP32


def _scale(amax):
    """(stored scale, factor before the cast) of groups with these max-abs values."""
    safe = torch.where(amax == 0, torch.ones_like(amax), amax)
    # both quotients correctly rounded (a number over a tensor would be a reciprocal and a product)
    top = torch.full_like(safe, 448.0)
    s, inv = safe / top, top / safe
    s = torch.where(amax < _TINY, torch.full_like(s, 2.0 ** -126), s)
    inv = torch.where(amax < _TINY, torch.full_like(s, 2.0 ** 126), inv)
    one = torch.ones_like(s)
    return torch.where(amax == 0, one, s), torch.where(amax == 0, one, inv)


def _q_1x128(v):
    M, C = v.shape
    b = v.view(M, C // 128, 128)
    s, inv = _scale(b.abs().amax(-1, keepdim=True))
    return (b * inv).clamp(-448, 448).to(E4M3).view(M, C), s.view(M, C // 128).t().contiguous()


def _q_128x1(v):
    T, C = v.shape
    b = v.view(T // 128, 128, C)
    s, inv = _scale(b.abs().amax(1, keepdim=True))
    return (b * inv).clamp(-448, 448).to(E4M3).view(T, C).t().contiguous(), s.view(T // 128, C)


def _decode_1x128(q, s):
    M, C = q.shape
    return (q.view(E4M3).float().view(M, C // 128, 128) * s.t().unsqueeze(-1)).view(M, C)


def _decode_128x128(q, s):
    *lead, N, K = q.shape
    return (q.view(E4M3).float().view(*lead, N // 128, 128, K // 128, 128)
            * s.view(*lead, N // 128, 1, K // 128, 1)).view(*lead, N, K)


def _live(st, M):
    return None if st["n"] is None else torch.arange(M, device="cuda") < st["n"]


def _cut(live, **out):
    """Zero what lies behind the last row in use (rows, scale columns, transposed columns, 128-row groups)."""
    if live is None:
        return out
    keep = {"row": live.view(-1, 1), "column": live.view(1, -1)}
    if live.numel() % 128 == 0:
        keep["block"] = live.view(-1, 128)[:, :1]
    along = dict(qa="row", sa="column", qh="row", sh="column", dh="row", qdh="row", sdh="column",
                 qdhT="column", sdhT="block", qaT="column", saT="block")
    zero = torch.zeros((), device="cuda")
    return {n: torch.where(keep[along[n]], v.float(), zero).to(v.dtype) for n, v in out.items()}


def _plain_fwd(st):
    h = st["h"].float()
    g, u = h.chunk(2, 1)
    a = g / (1.0 + torch.exp(-g)) * u
    qa, sa = _q_1x128(a)
    out = dict(qa=qa, sa=sa)
    if st["keep"]:
        out["qh"], out["sh"] = _q_1x128(h)
    return _cut(_live(st, h.shape[0]), **out)


def _plain_bwd(st):
    h = _decode_1x128(st["qh"], st["sh"])
    da = st["da"].float()
    M = h.shape[0]
    live = _live(st, M)
    if live is not None:
        h = torch.where(live.view(-1, 1), h, torch.zeros((), device="cuda"))
        da = torch.where(live.view(-1, 1), da, torch.zeros((), device="cuda"))
    g, u = h.chunk(2, 1)
    s = 1.0 / (1.0 + torch.exp(-g))
    silu = g * s
    dh = torch.cat((da * u * (s * (1.0 + g * (1.0 - s))), da * silu), 1)
    outs, out = st["outs"], {}
    if "d" in outs:
        out["dh"] = dh.to(torch.bfloat16)
    if "q" in outs:
        out["qdh"], out["sdh"] = _q_1x128(dh)
    if "t" in outs:
        out["qdhT"], out["sdhT"] = _q_128x1(dh)
    if "a" in outs:
        out["qaT"], out["saT"] = _q_128x1(silu * u)
    return _cut(live, **out)


def _plain_few(st):
    T, G, I = st["T"], st["G"], st["I"]
    x = _decode_1x128(*_q_1x128(st["x"].float()))
    h = torch.matmul(x, _decode_128x128(st["w13"], st["s13"]).transpose(1, 2))         # [G, T, 2I]
    g, u = h.view(G * T, 2 * I).chunk(2, 1)
    qa, sa = _q_1x128(g / (1.0 + torch.exp(-g)) * u)
    a = _decode_1x128(qa, sa).view(G, T, I)
    y = torch.matmul(a, _decode_128x128(st["w2"], st["s2"]).transpose(1, 2))           # [G, T, N]
    hot = st["topk"].unsqueeze(-1) == torch.arange(G, device="cuda", dtype=torch.int32)
    gate = (hot * st["gate"].unsqueeze(-1)).sum(1)                                     # [T, G]
    return (y * gate.t().unsqueeze(-1)).sum(0).to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls

_fg = None


def _library():
    global _fg
    if _fg is None:
        import fp8_fine_grained_x1_b200 as fg
        _fg = fg
    return _fg


def _values(st, *names):
    return {n: (st[n].view(E4M3) if n[0] == "q" else st[n]) for n in names if n in st}


def _own(st):
    fg = _library()
    if st["op"] == "fwd":
        fg.fp8_swiglu_quant(st["h"], st["qa"], st["sa"], st.get("qh"), st.get("sh"), n_rows=st["n"])
        return _values(st, "qa", "sa", "qh", "sh")
    if st["op"] == "bwd":
        fg.fp8_swiglu_bwd(st["qh"], st["sh"], st["da"], dh=st.get("dh"), qdh=st.get("qdh"), sdh=st.get("sdh"),
                          qdhT=st.get("qdhT"), sdhT=st.get("sdhT"), qaT=st.get("qaT"), saT=st.get("saT"),
                          n_rows=st["n"])
        return _values(st, "dh", "qdh", "sdh", "qdhT", "sdhT", "qaT", "saT")
    if st["ws"] is None:
        n = fg.fp8_moe_mlp_few_workspace_bytes(st["T"], st["k"], st["G"], st["K"], st["I"], st["N"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    fg.fp8_moe_mlp_few(st["x"], st["topk"], st["gate"], st["w13"], st["s13"], st["w2"], st["s2"], st["out"],
                       st["ws"])
    return st["out"]


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "few": _plain_few}[state["op"]](state)


# ------------------------------------------------------------------ work

def _active(case):
    """Experts that at least one token picks, averaged over draws of the routing law."""
    T, k, G = case["T"], case["k"], case["G"]
    g = torch.Generator().manual_seed(5)
    logp = -1.1 * torch.log(torch.arange(1, G + 1, dtype=torch.float64))
    seen = 0.0
    for _ in range(8):
        u = torch.rand((T, G), generator=g, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
        seen += torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices.unique().numel()
    return seen / 8


def work(case):
    if case["op"] == "few":
        T, k, K, I, N = (case[n] for n in ("T", "k", "K", "I", "N"))
        per = 2 * I * K + N * I
        return {"bytes": _active(case) * per * (1 + 4 / 16384) + T * K * 2 + T * N * 2 + T * k * 8,
                "flops": 2.0 * T * k * per}
    n, I, b = _n_rows(case), case["I"], 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "fwd":
        per = 2 * b + 1 + 4 / 128 + (2 + 8 / 128 if case["keep"] else 0)
        flops = 8
    else:
        o = case["outs"]
        per = 2 + 8 / 128 + b + ("d" in o) * 4 + ("q" in o) * (2 + 8 / 128) + ("t" in o) * (2 + 8 / 128) \
            + ("a" in o) * (1 + 4 / 128)
        flops = 20
    return {"bytes": max(1.0, float(n) * I * per), "flops": float(flops) * n * I}


# ------------------------------------------------------------------ the definition in 64 bits

def _f32(v):
    """Round to FP32 where the definition of a group scale says so."""
    return v.to(torch.float32).to(torch.float64)


def _e4m3_exact(v):
    """Nearest E4M3 value, ties to even, saturating, by arithmetic on float64."""
    mag = v.abs().clamp(max=448.0)
    _, e = torch.frexp(mag)                                  # mag = m * 2^e, m in [0.5, 1)
    step = torch.exp2((e - 4).clamp(min=-9).to(torch.float64))
    return torch.copysign(torch.round(mag / step) * step, v).clamp(-448.0, 448.0)


def _group_exact(v, dim):
    """Codes' values and scales of groups along `dim` (of size 128) of float64 values."""
    amax = v.abs().amax(dim, keepdim=True)
    s = torch.where(amax > 0, _f32(amax / 448.0).clamp(min=2.0 ** -126), torch.ones_like(amax))
    inv = torch.where(amax > 0, _f32(448.0 / amax).clamp(max=2.0 ** 126), torch.ones_like(amax))
    return _e4m3_exact(_f32(v * inv)), s


def _rows_exact(v):
    M, C = v.shape
    q, s = _group_exact(v.reshape(M, C // 128, 128), 2)
    return q.reshape(M, C), s.reshape(M, C // 128).t()


def _cols_exact(v):
    T, C = v.shape
    q, s = _group_exact(v.reshape(T // 128, 128, C), 1)
    return q.reshape(T, C).t(), s.reshape(T // 128, C)


def _codes64(q):
    """Values of E4M3 codes from their bit fields."""
    c = q.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).to(torch.float64)
    mag = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2((e - 7).to(torch.float64)), m * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _exact_few(st):
    T, K, I, N = st["T"], st["K"], st["I"], st["N"]
    q, s = _rows_exact(st["x"].double())
    x = (q.reshape(T, K // 128, 128) * s.t().unsqueeze(-1)).reshape(T, K)
    out = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for e in st["topk"].unique().tolist():
        hit = st["topk"] == e
        t = hit.any(1).nonzero().flatten()
        w = (hit * st["gate"].double()).sum(1)[t]

        def times(rows, wq, ws):
            n, c = wq.shape
            full = _codes64(wq).reshape(n // 128, 128, c // 128, 128) * ws.double().reshape(n // 128, 1, c // 128, 1)
            return rows @ full.reshape(n, c).t()

        h = times(x[t], st["w13"][e], st["s13"][e])
        g, u = h[:, :I], h[:, I:]
        qa, sa = _rows_exact(g * torch.sigmoid(g) * u)
        a = (qa.reshape(-1, I // 128, 128) * sa.t().unsqueeze(-1)).reshape(-1, I)
        out[t] += w.unsqueeze(1) * times(a, st["w2"][e], st["s2"][e])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "few":
        return _exact_few(st)
    n, M, I = _n_rows(case), case["M"], case["I"]
    out = {}

    def put(name, v, axis, size):
        full = torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
        full.narrow(axis, 0, size).copy_(v)
        out[name] = full

    if case["op"] == "fwd":
        h = st["h"][:n].double()
        g, u = h[:, :I], h[:, I:]
        q, s = _rows_exact(g * torch.sigmoid(g) * u)
        put("qa", q, 0, n)
        put("sa", s, 1, n)
        if case["keep"]:
            q, s = _rows_exact(h)
            put("qh", q, 0, n)
            put("sh", s, 1, n)
        return out
    h = (_codes64(st["qh"][:n]).reshape(n, 2 * I // 128, 128)
         * st["sh"][:, :n].double().t().unsqueeze(-1)).reshape(n, 2 * I)
    da = st["da"][:n].double()
    g, u = h[:, :I], h[:, I:]
    s = torch.sigmoid(g)
    dh = torch.cat((da * u * s * (1.0 + g * (1.0 - s)), da * g * s), 1)
    outs = case["outs"]
    if "d" in outs:
        put("dh", dh, 0, n)
    if "q" in outs:
        q, sc = _rows_exact(dh)
        put("qdh", q, 0, n)
        put("sdh", sc, 1, n)
    if "t" in outs:
        q, sc = _cols_exact(dh)
        put("qdhT", q, 1, n)
        put("sdhT", sc, 0, n // 128)
    if "a" in outs:
        q, sc = _cols_exact(g * s * u)
        put("qaT", q, 1, n)
        put("saT", sc, 0, n // 128)
    return out
