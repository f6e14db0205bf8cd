// moe_few.cu -- a whole FP8 MoE MLP for a few tokens (T <= 128), sm_100a.
//
//   xq = 1x128 codes of x; per active expert e: h = W13_e . xq (FP32),
//   a = silu(gate half) * up half, quantized 1x128; out[t] = sum over t's
//   experts of w * (W2_e . a), rounded once to the output type.
//
// With this few tokens the layer is bound by reading the active experts'
// weights once from HBM ("Three Fast Methods To Study Deepseek": top-8
// routing; gnrental.net post: the MoE part reads one expert's weights per
// group).  So the weights are the M operand (128 rows per MMA) and the tokens
// its N columns, and no rows are gathered or padded to 128: every column of an
// expert's products is a token, whether it was routed to that expert or not.
// The columns the tensor cores compute in vain cost nothing next to the
// weight stream, the B operand is the same token matrix for every expert, and
// the combine happens in the accumulator: column t of expert e's second
// product is promoted with its activation's scale times t's gate weight for e
// (0 where e was not picked).
//
// Kernels, in stream order:
//   k_few_prep      codes and scales of x, the list of active experts, the
//                   gate-weight table [expert][token], zeroed tile counters
//   k_few_gemm<1>   persistent; tile = 128 gate + 128 up rows of an expert over
//                   K; ends in SwiGLU + 1x128 quantization of those 128 channels
//   k_few_gemm<2>   persistent; tile = 256 output columns over all (expert, I)
//
// Both GEMM kernels lay their tiles' K-blocks end to end and give every CTA an
// equal contiguous range of them (stream-K), so all SMs stream weights for the
// same time whatever the tile count.  Parts of a tile meet in global scratch:
// the CTA that finishes a tile last adds them in CTA order (so results do not
// depend on timing) and runs the tile's epilogue.  No CTA waits for another.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "fp8fg_device.cuh"
#include "fp8fg_host.h"
#include "fp8fg_quant.cuh"

namespace fp8fg {

namespace {

constexpr int kFewMaxCtas = 152;                // scratch is sized for this many
constexpr int BK = 128;
constexpr uint32_t WBLK_BYTES = 128 * BK;       // 128 weight rows of one K-block
constexpr uint32_t W_BYTES = 2 * WBLK_BYTES;    // two row blocks per stage
constexpr int NUM_PROMO_WARPS = 8;              // warps 0-3: block 0, 4-7: block 1
constexpr int PROMO_THREADS = 32 * NUM_PROMO_WARPS;
constexpr int WARP_TMA = 8, WARP_MMA = 9;
constexpr int NUM_THREADS = PROMO_THREADS + 64;
constexpr uint32_t RING_BUDGET = 200 * 1024;
constexpr int MAX_STAGES = 6;

__host__ __device__ constexpr uint32_t stage_bytes(int nb) { return W_BYTES + (uint32_t)nb * BK; }
__host__ __device__ constexpr int num_stages(int nb)
{
    const int n = (int)(RING_BUDGET / stage_bytes(nb));
    return n < MAX_STAGES ? n : MAX_STAGES;
}
__host__ __device__ constexpr uint32_t dyn_smem(int nb) { return 1024 + num_stages(nb) * stage_bytes(nb); }

// ------------------------------------------------------------ workspace

struct Few {
    // problem
    const int32_t* topk;    // [T][k]
    const float* weights;   // [T][k]
    const float* s13;       // [G][2I/128][K/128]
    const float* s2;        // [G][N/128][I/128]
    void* out;
    int64_t ldo;
    int64_t K, I, N;
    int T, Tp, k, G;        // Tp: T rounded up to 16, the row stride of per-token tables
    int out_dtype, mode;
    uint64_t timeout_ns;
    // workspace
    int32_t* n_act;         // [1]
    int32_t* act;           // [A] active experts, ascending
    float* gate;            // [G][Tp] summed gate weight of token t for expert e
    int32_t* cnt;           // [A * I/128 + ceil(N/256)] parts finished per split tile
    uint8_t* xq;            // [T][K] codes, xs [K/128][Tp] scales
    float* xs;
    uint8_t* aq;            // [A * Tp][I] codes, as [A][I/128][Tp] scales * gate weight
    float* as;
    float* part;            // [2 * CTAs][2][T][128] partial tiles
};

int few_tp(int64_t T) { return (int)((T + 15) / 16 * 16); }

// Section sizes in order; returns the total, and fills `f` when base is given.
int64_t few_layout(Few* f, uint8_t* base, int64_t T, int k, int G, int64_t K, int64_t I, int64_t N)
{
    const int64_t Tp = few_tp(T);
    const int64_t A = T * k < G ? T * k : G;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += (bytes + 255) / 256 * 256;
        return base + at;
    };
    uint8_t* n_act = take(4);
    uint8_t* act = take(4 * A);
    uint8_t* gate = take(4 * G * Tp);
    uint8_t* cnt = take(4 * (A * (I / 128) + (N + 255) / 256));
    uint8_t* xq = take(T * K);
    uint8_t* xs = take(4 * (K / 128) * Tp);
    uint8_t* aq = take(A * Tp * I);
    uint8_t* as = take(4 * A * (I / 128) * Tp);
    uint8_t* part = take(4 * 2 * (int64_t)kFewMaxCtas * 2 * T * 128);
    if (f) {
        f->n_act = reinterpret_cast<int32_t*>(n_act);
        f->act = reinterpret_cast<int32_t*>(act);
        f->gate = reinterpret_cast<float*>(gate);
        f->cnt = reinterpret_cast<int32_t*>(cnt);
        f->xq = xq;
        f->xs = reinterpret_cast<float*>(xs);
        f->aq = aq;
        f->as = reinterpret_cast<float*>(as);
        f->part = reinterpret_cast<float*>(part);
    }
    return off;
}

// ------------------------------------------------------------ preparation

constexpr int kMaxExperts = 1024;

// Block 0 lists the active experts in ascending order; the others quantize x
// (a half-warp per 1x128 group, as k_quant_1x128) and share the gate table and
// the counters' zeroing.
template <typename Tin>
__global__ void __launch_bounds__(256) k_few_prep(const Few f, const Tin* __restrict__ x, int64_t ldx)
{
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        __shared__ int32_t flag[kMaxExperts];
        __shared__ int32_t wsum[8];
        for (int e = tid; e < kMaxExperts; e += 256) flag[e] = 0;
        __syncthreads();
        for (int64_t i = tid; i < (int64_t)f.T * f.k; i += 256) {
            const int32_t e = __ldg(f.topk + i);
            if (e >= 0 && e < f.G)
                flag[e] = 1;
            else
                report_error(FP8_ERR_SHAPE);
        }
        __syncthreads();
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += flag[4 * tid + i];
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, d);
            if ((tid & 31) >= d) incl += t;
        }
        if ((tid & 31) == 31) wsum[tid >> 5] = incl;
        __syncthreads();
        int at = incl - mine;
        for (int wq = 0; wq < (tid >> 5); ++wq) at += wsum[wq];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (flag[4 * tid + i]) f.act[at++] = 4 * tid + i;
        if (tid == 255) *f.n_act = at;
        return;
    }
    const int64_t nkb = f.K / 128;
    const int64_t b = blockIdx.x - 1, nb = gridDim.x - 1;
    const int64_t grp = b * 16 + (tid >> 4);
    const int l = tid & 15;
    const bool live = grp < f.T * nkb;
    const int64_t t = live ? grp / nkb : 0, kb = live ? grp % nkb : 0;
    Chunk8<Tin> c;
    if (live)
        c.load(x + t * ldx + kb * 128 + l * 8);
    else
        c.zero();
    float v[8];
    c.get(v);
    float a = absmax8(v);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const GroupScale g = group_scale(a, f.mode);
    if (live) {
        *reinterpret_cast<uint2*>(f.xq + t * f.K + kb * 128 + l * 8) =
            make_uint2(encode4(v[0], v[1], v[2], v[3], g.inv), encode4(v[4], v[5], v[6], v[7], g.inv));
        if (l == 0) f.xs[kb * f.Tp + t] = g.s;
    }
    const int64_t A = (int64_t)f.T * f.k < f.G ? (int64_t)f.T * f.k : f.G;
    const int64_t ncnt = A * (f.I / 128) + (f.N + 255) / 256;
    for (int64_t i = b * 256 + tid; i < ncnt; i += nb * 256) f.cnt[i] = 0;
    for (int64_t i = b * 256 + tid; i < (int64_t)f.G * f.Tp; i += nb * 256) {
        const int e = (int)(i / f.Tp), tt = (int)(i % f.Tp);
        float sum = 0.0f;
        if (tt < f.T)
            for (int j = 0; j < f.k; ++j)
                if (__ldg(f.topk + (int64_t)tt * f.k + j) == e) sum += __ldg(f.weights + (int64_t)tt * f.k + j);
        f.gate[i] = sum;
    }
}

// ------------------------------------------------------------ single-CTA tcgen05 / TMA

__device__ __forceinline__ void tma_load_2d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void promo_sync()   // the promotion warps only
{
    asm volatile("bar.sync 1, %0;" ::"n"(PROMO_THREADS) : "memory");
}

// ------------------------------------------------------------ GEMM

struct __align__(16) FewShared {
    float vec[NUM_PROMO_WARPS][2][128];   // per-warp token scales, double-buffered
    float up[16][128];                    // SwiGLU epilogue: up values of 16 tokens
    float wmax[4][16];                    // its per-warp max-abs
    uint8_t codes[16][128];               // and its codes
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int last;
};

// The units (tile, K-block) of all tiles end to end, and this CTA's range.
struct Range {
    int64_t U, P, per;      // units, CTAs that have work, units per tile
    int64_t u0, u1;
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * U / P; }
    __device__ __forceinline__ int64_t owner(int64_t u) const { return ((u + 1) * P - 1) / U; }
};

template <int PHASE>
__device__ __forceinline__ Range few_range(const Few& f, int n_act)
{
    Range r;
    const int64_t J = f.I / 128;
    r.per = PHASE == 1 ? f.K / BK : n_act * J;
    r.U = (PHASE == 1 ? n_act * J : (n_act ? (f.N + 255) / 256 : 0)) * r.per;
    r.P = r.U < gridDim.x ? r.U : gridDim.x;
    r.u0 = blockIdx.x < r.P ? r.begin(blockIdx.x) : 0;
    r.u1 = blockIdx.x < r.P ? r.begin(blockIdx.x + 1) : 0;
    return r;
}

// Rows (of the weight map) of the two 128-row blocks of unit kb of a tile.
template <int PHASE>
__device__ __forceinline__ void few_rows(const Few& f, int64_t tile, int64_t kb, int32_t& r0, int32_t& r1,
                                         int32_t& xk, int32_t& yk)
{
    const int64_t J = f.I / 128;
    if (PHASE == 1) {
        const int64_t e = __ldcg(f.act + tile / J), j = tile % J;
        r0 = (int32_t)(e * 2 * f.I + j * 128);
        r1 = r0 + (int32_t)f.I;
        xk = (int32_t)(kb * BK);
        yk = 0;
    } else {
        const int64_t a = kb / J, e = __ldcg(f.act + a);
        r0 = (int32_t)(e * f.N + tile * 256);
        r1 = r0 + 128;      // past this expert's rows in an odd last tile: never stored
        xk = (int32_t)((kb % J) * BK);
        yk = (int32_t)(a * f.Tp);
    }
}

template <int PHASE, int NB>
__device__ void few_producer(const CUtensorMap* tmW, const CUtensorMap* tmX, const Few& f, const Range& r,
                             uint8_t* smem, FewShared& sh)
{
    constexpr int NS = num_stages(NB);
    const uint32_t x_bytes = (uint32_t)f.Tp * BK;
    int64_t it = 0;
    for (int64_t u = r.u0; u < r.u1; ++u, ++it) {
        const int s = (int)(it % NS);
        if (!mbar_wait(&sh.empty[s], (uint32_t)((it / NS) & 1) ^ 1u, &sh.abort, f.timeout_ns)) break;
        int32_t r0, r1, xk, yk;
        few_rows<PHASE>(f, u / r.per, u % r.per, r0, r1, xk, yk);
        uint8_t* dst = smem + s * stage_bytes(NB);
        mbar_arrive_expect_tx(&sh.full[s], W_BYTES + x_bytes);
        tma_load_2d(dst, tmW, &sh.full[s], xk, r0);
        tma_load_2d(dst + WBLK_BYTES, tmW, &sh.full[s], xk, r1);
        tma_load_2d(dst + W_BYTES, tmX, &sh.full[s], xk, yk);
    }
    // every copy issued lands before the CTA exits
    for (int s = 0; s < NS; ++s) {
        const int64_t count = it > s ? (it - s + NS - 1) / NS : 0;
        if (count) mbar_wait_drain(&sh.full[s], (uint32_t)((count - 1) & 1), f.timeout_ns);
    }
}

template <int NB>
__device__ void few_mma(const Few& f, const Range& r, uint8_t* smem, FewShared& sh)
{
    constexpr int NS = num_stages(NB);
    const uint32_t base = smem_u32(smem);
    const uint32_t idesc = idesc_e4m3_f32(128, (uint32_t)f.Tp, 0);
    int64_t it = 0;
    for (int64_t u = r.u0; u < r.u1; ++u, ++it) {
        const int s = (int)(it % NS);
        const uint32_t buf = (uint32_t)(it & 1);
        if (!mbar_wait(&sh.tempty[buf], (uint32_t)((it >> 1) & 1) ^ 1u, &sh.abort, f.timeout_ns) ||
            !mbar_wait(&sh.full[s], (uint32_t)((it / NS) & 1), &sh.abort, f.timeout_ns))
            break;
        tc_fence_after();
        const uint32_t w = base + s * stage_bytes(NB);
        const uint32_t d = sh.tmem_base + buf * 2 * NB;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {
            const uint64_t xd = smem_desc_sw128(w + W_BYTES + k * 32, 16, 1024);
            mma_f8f6f4(d, smem_desc_sw128(w + k * 32, 16, 1024), xd, idesc, k > 0);
            mma_f8f6f4(d + NB, smem_desc_sw128(w + WBLK_BYTES + k * 32, 16, 1024), xd, idesc, k > 0);
        }
        mma_commit(&sh.empty[s]);
        mma_commit(&sh.tfull[buf]);
    }
    mma_commit(&sh.drain);
    mbar_wait_drain(&sh.drain, 0, f.timeout_ns);
}

// Sum over the CTAs c0..c1 that hold parts of a tile, in CTA order, of element
// (blk, t, row): `slot(c)` is where CTA c left its part.
struct Parts {
    const float* part;
    int64_t c0, c1, tile_u0, stride;   // stride: floats per slot
    Range r;
    __device__ __forceinline__ const float* at(int64_t c) const
    {
        // a CTA whose range begins inside the tile left its part in slot 0
        return part + (2 * c + (r.begin(c) >= tile_u0 ? 0 : 1)) * stride;
    }
};

// One tile's 128 activation channels of expert act[tile / J]: SwiGLU of the
// summed gate and up rows and 1x128 quantization, 16 tokens at a time.
// Threads 0-127 hold the gate rows, 128-255 the up rows.
__device__ __forceinline__ void few_finish_swiglu(const Few& f, const Parts& p, int64_t tile, FewShared& sh,
                                                  int tid)
{
    const int64_t J = f.I / 128, a = tile / J, j = tile % J;
    const int blk = tid >> 7, row = tid & 127, lane = tid & 31, w4 = (tid >> 5) & 3;
    const float* gate = f.gate + (int64_t)__ldcg(f.act + a) * f.Tp;
    for (int t0 = 0; t0 < f.T; t0 += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        for (int64_t c = p.c0; c <= p.c1; ++c) {
            const float* src = p.at(c) + (int64_t)blk * f.T * 128 + (int64_t)t0 * 128 + row;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (t0 + i < f.T) v[i] += __ldcg(src + i * 128);
        }
        if (blk == 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sh.up[i][row] = v[i];
        }
        promo_sync();
        if (blk == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // a token not routed to this expert (gate weight 0) becomes a zero row
                const bool routed = t0 + i < f.T && __ldcg(gate + t0 + i) != 0.0f;
                const float g = v[i];
                v[i] = routed ? g * __fdividef(1.0f, 1.0f + expf(-g)) * sh.up[i][row] : 0.0f;
                float m = fabsf(v[i]);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                if (lane == 0) sh.wmax[w4][i] = m;
            }
        }
        promo_sync();
        if (blk == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float m = fmaxf(fmaxf(sh.wmax[0][i], sh.wmax[1][i]), fmaxf(sh.wmax[2][i], sh.wmax[3][i]));
                const GroupScale gs = group_scale(m, f.mode);
                sh.codes[i][row] = (uint8_t)encode4(v[i], 0.f, 0.f, 0.f, gs.inv);
                if (row == i && t0 + i < f.T)
                    f.as[(a * J + j) * f.Tp + t0 + i] = gs.s * __ldcg(gate + t0 + i);
            }
        }
        promo_sync();
        if (tid < 128) {
            const int i = tid >> 3, c16 = (tid & 7) * 16;
            if (t0 + i < f.T)
                *reinterpret_cast<uint4*>(f.aq + (a * f.Tp + t0 + i) * f.I + j * 128 + c16) =
                    *reinterpret_cast<const uint4*>(&sh.codes[i][c16]);
        }
        // No barrier here: sh.up and sh.wmax were last read before the third barrier
        // (sh.up: the second), and sh.codes is written again only after the next
        // round's first two, which follow these reads.
    }
}

// One tile's 256 output columns: the summed parts, rounded to the output type.
__device__ __forceinline__ void few_finish_out(const Few& f, const Parts& p, int64_t tile, int tid)
{
    const int blk = tid >> 7, row = tid & 127;
    const int64_t n = tile * 256 + tid;
    if (n >= f.N) return;
    for (int t0 = 0; t0 < f.T; t0 += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        for (int64_t c = p.c0; c <= p.c1; ++c) {
            const float* src = p.at(c) + (int64_t)blk * f.T * 128 + (int64_t)t0 * 128 + row;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (t0 + i < f.T) v[i] += __ldcg(src + i * 128);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (t0 + i >= f.T) break;
            if (f.out_dtype == FP8_OUT_BF16)
                static_cast<__nv_bfloat16*>(f.out)[(t0 + i) * f.ldo + n] = __float2bfloat16_rn(v[i]);
            else
                static_cast<float*>(f.out)[(t0 + i) * f.ldo + n] = v[i];
        }
    }
}

template <int PHASE, int NB>
__device__ void few_promotion(const Few& f, const Range& r, FewShared& sh)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = warp >> 2, row = tid & 127;
    const uint32_t tmem = sh.tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + blk * NB;
    const int64_t J = f.I / 128, nb128 = f.N / 128;
    const int64_t slot_floats = (int64_t)2 * f.T * 128;
    int64_t it = 0;
    int seg = 0;
    // Once a wait has run out the warp takes no further part in the work, but
    // still meets the others at every segment's barriers.
    bool ok = true;
    for (int64_t u = r.u0; u < r.u1; ++seg) {
        const int64_t tile = u / r.per, tile_u0 = tile * r.per;
        const int64_t end = r.u1 < tile_u0 + r.per ? r.u1 : tile_u0 + r.per;
        float acc[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = 0.0f;
        // this K-block's weight-block scale and token scales
        auto wscale = [&](int64_t uu) -> float {
            const int64_t kb = uu - tile_u0;
            if (PHASE == 1) {
                const int64_t e = __ldcg(f.act + tile / J), j = tile % J;
                return __ldg(f.s13 + (e * 2 * J + blk * J + j) * (f.K / BK) + kb);
            }
            const int64_t e = __ldcg(f.act + kb / J), nb = tile * 2 + blk;
            return nb < nb128 ? __ldg(f.s2 + (e * nb128 + nb) * J + kb % J) : 0.0f;
        };
        auto tscale = [&](int64_t uu) -> float4 {
            const float* v = (PHASE == 1 ? f.xs : f.as) + (uu - tile_u0) * f.Tp + 4 * lane;
            return 4 * lane < f.Tp ? __ldcg(reinterpret_cast<const float4*>(v)) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float sw = wscale(u);
        *reinterpret_cast<float4*>(&sh.vec[warp][it & 1][4 * lane]) = tscale(u);
        __syncwarp();
        for (; ok && u < end; ++u, ++it) {
            float sw_next = 0.0f;
            float4 ts_next = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u + 1 < end) {
                sw_next = wscale(u + 1);
                ts_next = tscale(u + 1);
            }
            const uint32_t buf = (uint32_t)(it & 1);
            // the whole warp goes on or gives up (TMEM loads are warp-wide)
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&sh.tfull[buf], (uint32_t)((it >> 1) & 1), &sh.abort, f.timeout_ns));
            if (!ok) break;
            tc_fence_after();
            const float* vec = sh.vec[warp][it & 1];
#pragma unroll
            for (int c = 0; c < NB; c += 16) {
                if (c >= f.Tp) break;
                uint32_t p[16];
                tmem_ld16(tmem + buf * 2 * NB + c, p);
                float s[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(vec + c + i);
                    fmul2(s[i], s[i + 1], q.x, q.y, sw, sw);
                    fmul2(s[i + 2], s[i + 3], q.z, q.w, sw, sw);
                }
                tmem_ld_wait(p);
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    ffma2(acc[c + i], acc[c + i + 1], __uint_as_float(p[i]), __uint_as_float(p[i + 1]), s[i],
                          s[i + 1]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.tempty[buf]);
            sw = sw_next;
            *reinterpret_cast<float4*>(&sh.vec[warp][(it + 1) & 1][4 * lane]) = ts_next;
            __syncwarp();
        }
        u = end;

        // this CTA's part of the tile, then (for the last CTA to get here) the tile
        float* dst = f.part + (2 * (int64_t)blockIdx.x + (seg ? 1 : 0)) * slot_floats +
                     (int64_t)blk * f.T * 128 + row;
#pragma unroll
        for (int t = 0; t < NB; ++t)
            if (t < f.T) __stcg(dst + t * 128, acc[t]);
        Parts p;
        p.part = f.part;
        p.r = r;
        p.tile_u0 = tile_u0;
        p.stride = slot_floats;
        p.c0 = r.owner(tile_u0);
        p.c1 = r.owner(tile_u0 + r.per - 1);
        __threadfence();
        promo_sync();
        if (tid == 0) {
            int last = !*static_cast<volatile int*>(&sh.abort);   // a tile with a missing part is never finished
            if (last && p.c1 > p.c0) {
                int32_t* cnt = f.cnt + (PHASE == 1 ? tile
                                                   : ((int64_t)f.T * f.k < f.G ? (int64_t)f.T * f.k : f.G) * J + tile);
                last = atomicAdd(cnt, 1) == (int)(p.c1 - p.c0);
            }
            sh.last = last;
            __threadfence();
        }
        promo_sync();
        if (sh.last) {
            if (PHASE == 1)
                few_finish_swiglu(f, p, tile, sh, tid);
            else
                few_finish_out(f, p, tile, tid);
        }
        promo_sync();     // slot 1 and sh.last are reused by the next segment
    }
}

template <int PHASE, int NB>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_few_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Few f)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewShared sh;
    constexpr int NS = num_stages(NB);
    constexpr uint32_t TMEM_COLS = 4 * NB;     // two buffers of two blocks' NB columns
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512 && NS >= 2, "TMEM columns and ring depth");
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.tfull[b], 1);
            mbar_init(&sh.tempty[b], NUM_PROMO_WARPS);
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const int n_act = __ldcg(f.n_act);
    const Range r = few_range<PHASE>(f, n_act);
    if (warp == WARP_TMA) {
        if (lane == 0) few_producer<PHASE, NB>(&tmW, &tmX, f, r, smem, sh);
        __syncwarp();
    } else if (warp == WARP_MMA) {
        if (lane == 0) few_mma<NB>(f, r, smem, sh);
        __syncwarp();
    } else {
        few_promotion<PHASE, NB>(f, r, sh);
        if (PHASE == 2 && n_act == 0) {      // no valid expert at all: the sum over none
            for (int64_t i = (int64_t)blockIdx.x * PROMO_THREADS + threadIdx.x; i < f.T * f.N;
                 i += (int64_t)gridDim.x * PROMO_THREADS) {
                const int64_t at = i / f.N * f.ldo + i % f.N;
                if (f.out_dtype == FP8_OUT_BF16)
                    static_cast<__nv_bfloat16*>(f.out)[at] = __float2bfloat16_rn(0.0f);
                else
                    static_cast<float*>(f.out)[at] = 0.0f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
}

// ------------------------------------------------------------ host side

template <auto kernel>
bool few_allow_smem(int bytes)
{
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev])
        ready[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
                     cudaSuccess;
    return ready[dev];
}

template <int NB>
int launch_few_gemms(const Few& f, const CUtensorMap& tmW13, const CUtensorMap& tmW2, const CUtensorMap& tmX,
                     const CUtensorMap& tmA, unsigned ctas, cudaStream_t st)
{
    constexpr uint32_t smem = dyn_smem(NB);
    if (!few_allow_smem<k_few_gemm<1, NB>>((int)smem) || !few_allow_smem<k_few_gemm<2, NB>>((int)smem))
        return FP8_ERR_LAUNCH;
    k_few_gemm<1, NB><<<ctas, NUM_THREADS, smem, st>>>(tmW13, tmX, f);
    if (cudaGetLastError() != cudaSuccess) return FP8_ERR_LAUNCH;
    k_few_gemm<2, NB><<<ctas, NUM_THREADS, smem, st>>>(tmW2, tmA, f);
    return cudaGetLastError() == cudaSuccess ? FP8_OK : FP8_ERR_LAUNCH;
}

}  // namespace

int64_t moe_mlp_few_workspace_bytes(int64_t T, int k, int G, int64_t K, int64_t I, int64_t N)
{
    return few_layout(nullptr, nullptr, T, k, G, K, I, N);
}

int launch_moe_mlp_few(const void* x, int in_dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* topk,
                       const float* weights, int k, int G, const uint8_t* W13, const float* s13,
                       const uint8_t* W2, const float* s2, int64_t I, int64_t N, void* out, int out_dtype,
                       int64_t ldo, void* workspace, int mode, cudaStream_t st)
{
    Few f;
    few_layout(&f, static_cast<uint8_t*>(workspace), T, k, G, K, I, N);
    f.topk = topk;
    f.weights = weights;
    f.s13 = s13;
    f.s2 = s2;
    f.out = out;
    f.ldo = ldo;
    f.K = K;
    f.I = I;
    f.N = N;
    f.T = (int)T;
    f.Tp = few_tp(T);
    f.k = k;
    f.G = G;
    f.out_dtype = out_dtype;
    f.mode = mode;
    f.timeout_ns = wait_timeout_ns();
    const int64_t A = T * k < G ? T * k : G;
    CUtensorMap tmW13, tmW2, tmX, tmA;
    if (!make_map(&tmW13, W13, (uint64_t)K, (uint64_t)G * 2 * I, (uint64_t)K, BK, 128) ||
        !make_map(&tmW2, W2, (uint64_t)I, (uint64_t)G * N, (uint64_t)I, BK, 128) ||
        !make_map(&tmX, f.xq, (uint64_t)K, (uint64_t)T, (uint64_t)K, BK, (uint32_t)f.Tp) ||
        !make_map(&tmA, f.aq, (uint64_t)I, (uint64_t)A * f.Tp, (uint64_t)I, BK, (uint32_t)f.Tp))
        return FP8_ERR_LAUNCH;
    const unsigned prep = 1 + (unsigned)((T * (K / 128) + 15) / 16);
    if (in_dtype == FP8_IN_BF16)
        k_few_prep<__nv_bfloat16><<<prep, 256, 0, st>>>(f, static_cast<const __nv_bfloat16*>(x), ldx);
    else
        k_few_prep<float><<<prep, 256, 0, st>>>(f, static_cast<const float*>(x), ldx);
    if (cudaGetLastError() != cudaSuccess) return FP8_ERR_LAUNCH;
    const int sms = device_sm_count();
    const unsigned ctas = (unsigned)(sms < 1 ? 1 : (sms < kFewMaxCtas ? sms : kFewMaxCtas));
    if (f.Tp <= 16) return launch_few_gemms<16>(f, tmW13, tmW2, tmX, tmA, ctas, st);
    if (f.Tp <= 32) return launch_few_gemms<32>(f, tmW13, tmW2, tmX, tmA, ctas, st);
    if (f.Tp <= 64) return launch_few_gemms<64>(f, tmW13, tmW2, tmX, tmA, ctas, st);
    return launch_few_gemms<128>(f, tmW13, tmW2, tmX, tmA, ctas, st);
}

int read_and_clear_few_status() { return read_and_clear_module_status(); }

}  // namespace fp8fg
