"""The fine-grained FP8 Linear's three GEMM passes and the MoE expert pass, as
ready-to-run steps over device-resident inputs.

Each step owns its output buffers (allocated once with torch) and, when
called, issues only library calls: on the caller's stream (torch's current
one by default), and for one of its two quantizers on a side stream forked
from it and joined back before the GEMM:

  FpropStep    X[M,K] --1x128--> (qX, sX);  W[N,K] --128x128--> (qW, sW);
               Y[M,N] = qX . qW^T                      (BF16 or FP32 out)
  DgradStep    dY[M,N_out] --1x128--> ;  W[N_out,K_in] --128x128--> (stored
               orientation); dX[M,K_in] = dY . W, W read MN-major
  WgradStep    X[T,C_in], dY[T,C_out] --128x1--> token-contiguous codes with
               per-channel scales; dW[C_out,C_in] = dY^T . X, FP32 out
  WgradCachedStep  as WgradStep, with X taken from its cached 1x128 FP8
               form and requantized into 128x1 groups
  MoeStep      tokens X[T,K] --1x128, written straight to their expert-
               contiguous, 128-padded FP8 rows-->; W[G,N,K] --128x128-->;
               grouped GEMM (or, gather=True, quantized once and gathered by
               the GEMM)
  GatedMlpStep X[M,K] . W13[2I,K]^T -> SwiGLU -> . W2[N,I]^T, forward and
               backward: what backward needs is kept in FP8 (X's codes and the
               SwiGLU's 8-bit checkpoint), and the SwiGLU writes and reads the
               operands of the GEMMs around it
  MoeMlpStep   the MoE layer's MLP with weights already in FP8: up to
               MOE_FEW_MAX_TOKENS tokens in one call (fp8_moe_mlp_few), more
               through the dispatch and two grouped GEMMs

("5 Ways You can get More Deepseek While Spending Less", Figure 6: Fprop,
Dgrad and Wgrad all run in FP8; why-be.co.kr / cameseeing.com posts and
"Three Fast Methods To Study Deepseek", Figure 7 (a): 1x128 / 128x128
grouping; gnrental.net post: BF16 or FP32 GEMM outputs.)

Constructors allocate on torch's current stream: a step that is called on
another stream has to be ordered behind it first, as its inputs have to be.
A step's buffers are its own: its calls, and graphs captured from them, run one
after the other.

`kernel_calls` on each step counts the kernels one call launches.

With scale_mode=SCALE_POW2 the dense steps accept tensor_core_scaling=True:
the GEMM then applies the power-of-two scales inside the tensor cores
(fp8_blockscaled_gemm_pow2, UE8M0 block scaling) instead of promoting every
128-K partial in software.
"""
from __future__ import annotations

import contextlib

import torch

from . import (B_KMAJOR, B_MNMAJOR, MOE_FEW_MAX_TOKENS, SCALE_FP32, SCALE_POW2, fp8_blockscaled_gemm,
               fp8_blockscaled_gemm_pow2, fp8_grouped_gemm, fp8_grouped_gemm_gather,
               fp8_grouped_gemm_pow2,
               fp8_moe_combine, fp8_moe_dispatch_workspace_bytes, fp8_moe_mlp_few,
               fp8_moe_mlp_few_workspace_bytes, fp8_moe_quant_dispatch,
               fp8_moe_route, fp8_quant_act_128x1, fp8_quant_act_1x128, fp8_quant_w_128x128,
               fp8_requant_1x128_to_128x1, fp8_swiglu_bwd, fp8_swiglu_quant, moe_capacity)


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


class _Fork:
    """Each step's two quantizers share no input, so one of them runs on a
    side stream forked from the caller's stream and joined back before the
    GEMM: the tail of one overlaps the other, and short launches overlap
    each other's start-up."""

    def __init__(self, device):
        self.side = torch.cuda.Stream(device=device)
        self.fork, self.join = torch.cuda.Event(), torch.cuda.Event()
        self.device = device

    def begin(self, stream):
        cur = stream if stream is not None else torch.cuda.current_stream(self.device)
        self.fork.record(cur)
        self.side.wait_event(self.fork)
        return cur, self.side

    def end(self, cur):
        self.join.record(self.side)
        cur.wait_event(self.join)


def _gemm_fn(scale_mode, tensor_core_scaling):
    if not tensor_core_scaling:
        return fp8_blockscaled_gemm
    if scale_mode != SCALE_POW2:
        raise ValueError("tensor-core scaling needs power-of-two scales (SCALE_POW2)")
    return fp8_blockscaled_gemm_pow2


class FpropStep:
    kernel_calls = 3

    def __init__(self, x, w, out_dtype=torch.bfloat16, scale_mode=SCALE_FP32,
                 tensor_core_scaling=False):
        M, K = x.shape
        N = w.shape[0]
        d = x.device
        self.x, self.w, self.mode = x, w, scale_mode
        self._gemm = _gemm_fn(scale_mode, tensor_core_scaling)
        self.qx, self.sx = _empty((M, K), torch.uint8, d), _empty((K // 128, M), torch.float32, d)
        self.qw, self.sw = _empty((N, K), torch.uint8, d), _empty((N // 128, K // 128), torch.float32, d)
        self.y = _empty((M, N), out_dtype, d)
        self.flops = 2 * M * N * K
        self.inputs, self.output = [x, w], self.y
        self._fork = _Fork(d)

    def quantize(self, stream=None):
        cur, side = self._fork.begin(stream)
        fp8_quant_w_128x128(self.w, self.qw, self.sw, self.mode, side)
        fp8_quant_act_1x128(self.x, self.qx, self.sx, self.mode, cur)
        self._fork.end(cur)

    def gemm(self, stream=None):
        self._gemm(self.qx, self.sx, self.qw, self.sw, self.y, B_KMAJOR, 128, stream)

    def __call__(self, stream=None):
        self.quantize(stream)
        self.gemm(stream)
        return self.y


class DgradStep:
    kernel_calls = 3

    def __init__(self, dy, w, out_dtype=torch.bfloat16, scale_mode=SCALE_FP32,
                 tensor_core_scaling=False):
        M, N_out = dy.shape
        N_out2, K_in = w.shape
        assert N_out == N_out2
        d = dy.device
        self.dy, self.w, self.mode = dy, w, scale_mode
        self._gemm = _gemm_fn(scale_mode, tensor_core_scaling)
        self.qdy = _empty((M, N_out), torch.uint8, d)
        self.sdy = _empty((N_out // 128, M), torch.float32, d)
        self.qw = _empty((N_out, K_in), torch.uint8, d)
        self.sw = _empty((N_out // 128, K_in // 128), torch.float32, d)
        self.dx = _empty((M, K_in), out_dtype, d)
        self.flops = 2 * M * K_in * N_out
        self.inputs, self.output = [dy, w], self.dx
        self._fork = _Fork(d)

    def quantize(self, stream=None):
        cur, side = self._fork.begin(stream)
        fp8_quant_w_128x128(self.w, self.qw, self.sw, self.mode, side)
        fp8_quant_act_1x128(self.dy, self.qdy, self.sdy, self.mode, cur)
        self._fork.end(cur)

    def gemm(self, stream=None):
        # B = W stored [K = N_out][N = K_in]: MN-major; its block scales
        # sW[N_out/128][K_in/128] are [K/128][N/128] in GEMM terms.
        self._gemm(self.qdy, self.sdy, self.qw, self.sw, self.dx, B_MNMAJOR, 128, stream)

    def __call__(self, stream=None):
        self.quantize(stream)
        self.gemm(stream)
        return self.dx


class WgradStep:
    kernel_calls = 3

    def __init__(self, x, dy, scale_mode=SCALE_FP32, tensor_core_scaling=False):
        T, C_in = x.shape
        T2, C_out = dy.shape
        assert T == T2
        d = x.device
        self.x, self.dy, self.mode = x, dy, scale_mode
        self._gemm = _gemm_fn(scale_mode, tensor_core_scaling)
        self.qxT = _empty((C_in, T), torch.uint8, d)
        self.sx = _empty((T // 128, C_in), torch.float32, d)
        self.qdyT = _empty((C_out, T), torch.uint8, d)
        self.sdy = _empty((T // 128, C_out), torch.float32, d)
        self.dw = _empty((C_out, C_in), torch.float32, d)
        self.flops = 2 * C_out * C_in * T
        self.inputs, self.output = [x, dy], self.dw
        self._fork = _Fork(d)

    def quantize(self, stream=None):
        cur, side = self._fork.begin(stream)
        fp8_quant_act_128x1(self.dy, self.qdyT, self.sdy, self.mode, side)
        fp8_quant_act_128x1(self.x, self.qxT, self.sx, self.mode, cur)
        self._fork.end(cur)

    def gemm(self, stream=None):
        self._gemm(self.qdyT, self.sdy, self.qxT, self.sx, self.dw, B_KMAJOR, 1, stream)

    def __call__(self, stream=None):
        self.quantize(stream)
        self.gemm(stream)
        return self.dw


class WgradCachedStep:
    """Wgrad with X kept from the forward pass as 1x128 FP8 (codes qx [T, C_in],
    scales sx [C_in/128, T]): the cache is requantized into 128x1 groups along
    tokens instead of quantizing a BF16 copy of X; dY is quantized 128x1."""
    kernel_calls = 3

    def __init__(self, qx, sx, dy, scale_mode=SCALE_FP32):
        T, C_in = qx.shape
        T2, C_out = dy.shape
        assert T == T2
        d = qx.device
        self.qx, self.sx, self.dy, self.mode = qx, sx, dy, scale_mode
        self.qxT = _empty((C_in, T), torch.uint8, d)
        self.sxT = _empty((T // 128, C_in), torch.float32, d)
        self.qdyT = _empty((C_out, T), torch.uint8, d)
        self.sdy = _empty((T // 128, C_out), torch.float32, d)
        self.dw = _empty((C_out, C_in), torch.float32, d)
        self.flops = 2 * C_out * C_in * T
        self.inputs, self.output = [qx, sx, dy], self.dw
        self._fork = _Fork(d)

    def quantize(self, stream=None):
        cur, side = self._fork.begin(stream)
        fp8_quant_act_128x1(self.dy, self.qdyT, self.sdy, self.mode, side)
        fp8_requant_1x128_to_128x1(self.qx, self.sx, self.qxT, self.sxT, self.mode, cur)
        self._fork.end(cur)

    def gemm(self, stream=None):
        fp8_blockscaled_gemm(self.qdyT, self.sdy, self.qxT, self.sxT, self.dw, B_KMAJOR, 1, stream)

    def __call__(self, stream=None):
        self.quantize(stream)
        self.gemm(stream)
        return self.dw


class MoeStep:
    """MoE expert layer forward.  Tokens X[T,K] are quantized 1x128 straight
    into their expert-contiguous, 128-padded rows (fp8_moe_quant_dispatch),
    W[G,N,K] is quantized 128x128, and the grouped GEMM reads A in place.
    With gather=True the tokens are instead quantized once in token order,
    routed without moving rows (fp8_moe_route), and the grouped GEMM reads
    each row's token codes through TMA gathers (fp8_grouped_gemm_gather): the
    dispatched copy (k rows per token) is never written, at the price of a
    slower GEMM (the gathers issue 32 TMA operations per K-block where a
    tiled load issues one).  `combine(weights)` adds the weighted return to
    token order."""

    def __init__(self, x, topk, w, out_dtype=torch.bfloat16, scale_mode=SCALE_FP32,
                 tensor_core_scaling=False, gather=False):
        T, K = x.shape
        G, N, K2 = w.shape
        assert K == K2
        if tensor_core_scaling and scale_mode != SCALE_POW2:
            raise ValueError("tensor-core scaling needs power-of-two scales (SCALE_POW2)")
        if tensor_core_scaling and gather:
            raise ValueError("the tensor-core-scaled grouped GEMM reads dispatched rows only")
        self.gather = gather
        self._gemm = fp8_grouped_gemm_pow2 if tensor_core_scaling else fp8_grouped_gemm
        # gather: routing (count, scan, rank), token quantizer, weight quantizer
        # (side stream), gathered grouped GEMM; else routing, fused quantizer,
        # padding rows, weight quantizer, grouped GEMM (+1 memset either way)
        self.kernel_calls = 6 if self.gather else 7
        k = topk.shape[1]
        d = x.device
        self.x, self.topk, self.w, self.mode, self.G = x, topk, w, scale_mode, G
        self.M_cap = moe_capacity(T, k, G)
        if self.gather:
            self.qx = _empty((T, K), torch.uint8, d)
            self.sx = _empty((K // 128, T), torch.float32, d)
        else:
            self.qa = _empty((self.M_cap, K), torch.uint8, d)
            self.sa = _empty((K // 128, self.M_cap), torch.float32, d)
        self.offsets = _empty((G + 1,), torch.int32, d)
        self.token_row = _empty((T, k), torch.int32, d)
        self.row_token = _empty((self.M_cap,), torch.int32, d)
        self.ws = _empty((max(1, fp8_moe_dispatch_workspace_bytes(T, k, G) // 4),), torch.int32, d)
        self.qw = _empty((G, N, K), torch.uint8, d)
        self.sw = _empty((G, N // 128, K // 128), torch.float32, d)
        self.y = _empty((self.M_cap, N), out_dtype, d)
        self.out = None
        self.inputs, self.output = [x, w, topk], self.y
        # the weight quantizer on the side stream: the short routing kernels
        # and the token path overlap it
        self._fork = _Fork(d)

    def quantize(self, stream=None):
        cur, side = self._fork.begin(stream)
        G, N, K = self.w.shape
        fp8_quant_w_128x128(self.w.view(G * N, K), self.qw.view(G * N, K),
                            self.sw.view(G * N // 128, K // 128), self.mode, side)
        if self.gather:
            fp8_moe_route(self.topk, self.G, self.offsets, self.token_row, self.row_token, self.ws,
                          cur)
            fp8_quant_act_1x128(self.x, self.qx, self.sx, self.mode, cur)
        else:
            fp8_moe_quant_dispatch(self.x, self.topk, self.G, self.qa, self.sa, self.offsets,
                                   self.token_row, self.row_token, self.ws, self.mode, cur)
        self._fork.end(cur)

    def gemm(self, stream=None):
        if self.gather:
            fp8_grouped_gemm_gather(self.qx, self.sx, self.row_token, self.qw, self.sw,
                                    self.offsets, self.y, stream)
        else:
            self._gemm(self.qa, self.sa, self.qw, self.sw, self.offsets, self.y, stream)

    def combine(self, weights, stream=None):
        T = self.x.shape[0]
        if self.out is None:
            self.out = _empty((T, self.y.shape[1]), torch.bfloat16, self.x.device)
        fp8_moe_combine(self.y, self.token_row, weights, self.out, stream)
        return self.out

    def __call__(self, stream=None):
        self.quantize(stream)
        self.gemm(stream)
        return self.y


class GatedMlpStep:
    """Gated MLP, forward and backward: H = X . W13^T (W13 [2I, K]: gate rows,
    then up rows), A = silu(gate) * up, Y = A . W2^T (W2 [N, I]).

    Calling the step runs the forward pass and returns Y.  `backward(dy)` (dy
    [M, N] BF16 or FP32, M a multiple of 128) returns dX (out_dtype), dW13 and
    dW2 (FP32).  Between the two the step needs, in FP8, X's 1x128 codes and H's
    (`qx`, `qh`: K + 2 I bytes a token and their scales, where BF16 X, H and A would
    take 2 K + 6 I); A is recomputed.  Weights are quantized in the forward pass and
    reused by backward.

    H and dA are rounded to `hidden_dtype` between the GEMMs and the SwiGLU: to BF16
    unless FP32 is asked for, which keeps their sums as they are for 4 bytes an element
    more on the way (BF16 halves that traffic, and the E4M3 codes made of them keep 4
    bits of significand where BF16 has 8).

    H, A's codes and the operands of backward's GEMMs are scratch.  Each step
    has its own unless it is given another's: `share` is a step of the same sizes
    (another layer) whose scratch this one uses too, so that a model of many layers
    holds it once (with hidden_dtype the same).  Steps that share run one after the
    other, in any order of forward and backward passes."""
    kernel_calls = 6             # x, w13, w2 quantizers, two GEMMs, the SwiGLU
    kernel_calls_backward = 8    # dy twice, cached x, the SwiGLU, four GEMMs

    def __init__(self, x, w13, w2, out_dtype=torch.bfloat16, scale_mode=SCALE_FP32, share=None,
                 hidden_dtype=torch.bfloat16):
        M, K = x.shape
        C, K2 = w13.shape
        N, I = w2.shape
        if K != K2 or C != 2 * I:
            raise ValueError(f"x {tuple(x.shape)}, w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit: "
                             "w13 is [2I, K] and w2 [N, I]")
        d = x.device
        u8, f32 = torch.uint8, torch.float32
        self.x, self.w13, self.w2, self.mode, self.out_dtype = x, w13, w2, scale_mode, out_dtype
        self.qx, self.sx = _empty((M, K), u8, d), _empty((K // 128, M), f32, d)
        self.qw13, self.sw13 = _empty((C, K), u8, d), _empty((C // 128, K // 128), f32, d)
        self.qw2, self.sw2 = _empty((N, I), u8, d), _empty((N // 128, I // 128), f32, d)
        self.qh, self.sh = _empty((M, C), u8, d), _empty((C // 128, M), f32, d)
        if share is None:
            self._scratch = dict(sizes=(M, K, I, N, hidden_dtype, d), h=_empty((M, C), hidden_dtype, d),
                                 qa=_empty((M, I), u8, d), sa=_empty((I // 128, M), f32, d), grad=None)
        else:
            if share._scratch["sizes"] != (M, K, I, N, hidden_dtype, d):
                raise ValueError(f"share: a step of (M, K, I, N, hidden_dtype, device) = {share._scratch['sizes']}, "
                                 f"this one has {(M, K, I, N, hidden_dtype, d)}")
            self._scratch = share._scratch
        self.h, self.qa, self.sa = (self._scratch[n] for n in ("h", "qa", "sa"))
        self.y = _empty((M, N), out_dtype, d)
        self.flops = 2 * M * (C * K + N * I)
        self.inputs, self.output = [x, w13, w2], self.y
        self._fork = _Fork(d)
        self._grad = None
        self._ran = False

    def __call__(self, stream=None):
        self._ran = False
        cur, side = self._fork.begin(stream)
        fp8_quant_w_128x128(self.w13, self.qw13, self.sw13, self.mode, side)
        fp8_quant_w_128x128(self.w2, self.qw2, self.sw2, self.mode, side)
        fp8_quant_act_1x128(self.x, self.qx, self.sx, self.mode, cur)
        self._fork.end(cur)
        fp8_blockscaled_gemm(self.qx, self.sx, self.qw13, self.sw13, self.h, B_KMAJOR, 128, cur)
        fp8_swiglu_quant(self.h, self.qa, self.sa, self.qh, self.sh, None, self.mode, cur)
        fp8_blockscaled_gemm(self.qa, self.sa, self.qw2, self.sw2, self.y, B_KMAJOR, 128, cur)
        self._ran = True
        return self.y

    def _gradient_buffers(self, stream):
        """Backward's buffers, allocated at its first call: on the stream it runs on (the side stream
        is forked from that), so that memory still in use elsewhere is not taken."""
        if self._grad is None:
            M, K = self.x.shape
            N, I = self.w2.shape
            d, u8, f32 = self.x.device, torch.uint8, torch.float32
            if M % 128:
                raise ValueError(f"backward needs whole groups of 128 tokens, got {M}")
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                if self._scratch["grad"] is None:
                    self._scratch["grad"] = dict(
                        qdy=_empty((M, N), u8, d), sdy=_empty((N // 128, M), f32, d),
                        qdyT=_empty((N, M), u8, d), sdyT=_empty((M // 128, N), f32, d),
                        da=_empty((M, I), self.h.dtype, d),
                        qdh=_empty((M, 2 * I), u8, d), sdh=_empty((2 * I // 128, M), f32, d),
                        qdhT=_empty((2 * I, M), u8, d), sdhT=_empty((M // 128, 2 * I), f32, d),
                        qaT=_empty((I, M), u8, d), saT=_empty((M // 128, I), f32, d),
                        qxT=_empty((K, M), u8, d), sxT=_empty((M // 128, K), f32, d))
                self._grad = dict(
                    self._scratch["grad"],
                    dx=_empty((M, K), self.out_dtype, d), dw13=_empty((2 * I, K), f32, d), dw2=_empty((N, I), f32, d))
        return self._grad

    def backward(self, dy, stream=None):
        if not self._ran:
            raise RuntimeError("backward needs a forward pass before it")
        if dy.shape != self.y.shape or dy.device != self.y.device:
            raise ValueError(f"dy must have y's shape {tuple(self.y.shape)} and device {self.y.device}, "
                             f"got {tuple(dy.shape)} on {dy.device}")
        g = self._gradient_buffers(stream)
        cur, side = self._fork.begin(stream)
        # dy along tokens and x's cached codes regrouped, for the two Wgrads
        fp8_quant_act_128x1(dy, g["qdyT"], g["sdyT"], self.mode, side)
        fp8_requant_1x128_to_128x1(self.qx, self.sx, g["qxT"], g["sxT"], self.mode, side)
        fp8_quant_act_1x128(dy, g["qdy"], g["sdy"], self.mode, cur)
        fp8_blockscaled_gemm(g["qdy"], g["sdy"], self.qw2, self.sw2, g["da"], B_MNMAJOR, 128, cur)
        fp8_swiglu_bwd(self.qh, self.sh, g["da"], qdh=g["qdh"], sdh=g["sdh"], qdhT=g["qdhT"], sdhT=g["sdhT"],
                       qaT=g["qaT"], saT=g["saT"], scale_mode=self.mode, stream=cur)
        fp8_blockscaled_gemm(g["qdh"], g["sdh"], self.qw13, self.sw13, g["dx"], B_MNMAJOR, 128, cur)
        self._fork.end(cur)
        fp8_blockscaled_gemm(g["qdhT"], g["sdhT"], g["qxT"], g["sxT"], g["dw13"], B_KMAJOR, 1, cur)
        fp8_blockscaled_gemm(g["qdyT"], g["sdyT"], g["qaT"], g["saT"], g["dw2"], B_KMAJOR, 1, cur)
        return g["dx"], g["dw13"], g["dw2"]


class MoeMlpStep:
    """The MLP of an MoE layer in inference: out[t] = sum_j weights[t, j] *
    W2_e . (silu(gate) * up) with [gate | up] = W13_e . x[t], e = topk[t, j], on
    weights quantized beforehand (qw13 [G, 2I, K], sw13; qw2 [G, N, I], sw2).

    Up to MOE_FEW_MAX_TOKENS tokens take one call that reads each active
    expert's weights once (fp8_moe_mlp_few).  More tokens are quantized and
    dispatched to 128-padded groups, and the SwiGLU between the two grouped GEMMs
    quantizes the rows in use for the second; H is `hidden_dtype` there (BF16 unless
    FP32 is asked for) and FP32 in the few-token form.  On 32 experts of 7168 x 2048, top-8, the few-token form took
    70, 196, 240, 249 and 272 us for 1, 8, 32, 64 and 128 tokens, the dispatched
    form 177, 389, 461, 496 and 512: it is taken wherever it can be.  `few`
    overrides the choice."""

    def __init__(self, x, topk, weights, qw13, sw13, qw2, sw2, out_dtype=torch.bfloat16, scale_mode=SCALE_FP32,
                 few=None, hidden_dtype=torch.bfloat16):
        T, K = x.shape
        k = topk.shape[1]
        G, C, _ = qw13.shape
        N, I = qw2.shape[1:]
        d, u8, f32 = x.device, torch.uint8, torch.float32
        self.few = T <= MOE_FEW_MAX_TOKENS if few is None else few
        if self.few and T > MOE_FEW_MAX_TOKENS:
            raise ValueError(f"the few-token form takes {MOE_FEW_MAX_TOKENS} tokens, got {T}")
        if not self.few and out_dtype != torch.bfloat16:
            raise ValueError("the combine of the dispatched form writes BF16")
        self.x, self.topk, self.weights, self.mode, self.G = x, topk, weights, scale_mode, G
        self.qw13, self.sw13, self.qw2, self.sw2 = qw13, sw13, qw2, sw2
        self.out = _empty((T, N), out_dtype, d)
        self.inputs, self.output = [x, topk, weights], self.out
        # the few-token form: preparation, two GEMMs, SwiGLU, output sums; the other: routing (3), fused
        # quantizer, padding rows, two grouped GEMMs, SwiGLU, combine (+1 memset)
        self.kernel_calls = 5 if self.few else 9
        if self.few:
            n = fp8_moe_mlp_few_workspace_bytes(T, k, G, K, I, N)
            self.ws = _empty((max(n, 1),), u8, d)
            return
        M = moe_capacity(T, k, G)
        self.qr, self.sr = _empty((M, K), u8, d), _empty((K // 128, M), f32, d)
        self.offsets = _empty((G + 1,), torch.int32, d)
        self.token_row = _empty((T, k), torch.int32, d)
        self.row_token = _empty((M,), torch.int32, d)
        self.ws = _empty((max(1, fp8_moe_dispatch_workspace_bytes(T, k, G) // 4),), torch.int32, d)
        self.h = _empty((M, C), hidden_dtype, d)
        self.qa, self.sa = _empty((M, I), u8, d), _empty((I // 128, M), f32, d)
        self.y = _empty((M, N), torch.bfloat16, d)

    def __call__(self, stream=None):
        if self.few:
            fp8_moe_mlp_few(self.x, self.topk, self.weights, self.qw13, self.sw13, self.qw2, self.sw2, self.out,
                            self.ws, self.mode, stream)
            return self.out
        fp8_moe_quant_dispatch(self.x, self.topk, self.G, self.qr, self.sr, self.offsets, self.token_row,
                               self.row_token, self.ws, self.mode, stream)
        fp8_grouped_gemm(self.qr, self.sr, self.qw13, self.sw13, self.offsets, self.h, stream)
        fp8_swiglu_quant(self.h, self.qa, self.sa, n_rows=self.offsets[self.G:], scale_mode=self.mode, stream=stream)
        fp8_grouped_gemm(self.qa, self.sa, self.qw2, self.sw2, self.offsets, self.y, stream)
        fp8_moe_combine(self.y, self.token_row, self.weights, self.out, stream)
        return self.out
