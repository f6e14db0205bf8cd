// moe_few.cu -- a whole FP8 MoE MLP for a few tokens (T <= 128), sm_100a.
//
//   xq = 1x128 codes of x; per active expert e: h = W13_e . xq (FP32),
//   a = silu(gate half) * up half, quantized 1x128; out[t] = sum over t's
//   experts of w * (W2_e . a), rounded once to the output type.
//
// With this few tokens the layer is bound by reading the active experts'
// weights once from HBM ("Three Fast Methods To Study Deepseek": top-8
// routing; gnrental.net post: the MoE part reads one expert's weights per
// group).  So no rows are gathered or padded to 128 per expert: the products
// of an expert's weights are made with all tokens, whether they were routed to
// it or not.  What the tensor cores compute in vain costs nothing next to the
// weight stream, the token operand is the same for every expert, and the
// combine happens in the accumulator: token t's part of expert e's second
// product is promoted with its activation's scale times t's gate weight for e,
// and left out where e was not picked.  Up to 32 tokens are the N columns of
// the MMAs and the weights their M rows, more tokens are the M rows (see
// MAX_COLUMN_TOKENS).
//
// Kernels, in stream order (each starts while the one before drains):
//   k_few_prep      codes and scales of x, the gate-weight table [expert][token],
//                   the list of active experts
//   k_few_gemm<1>   persistent; tile = 128 gate + 128 up rows of an expert over K;
//                   leaves the sums, or its parts of them, in scratch
//   k_few_act, k_few_act_rows   adds the parts; SwiGLU and 1x128 quantization
//   k_few_gemm<2>   persistent; tile = 256 output columns over all (expert, I);
//                   whole tiles are rounded and stored, parts left in scratch
//   k_few_out       adds the parts, rounds
//
// Both GEMM kernels lay their tiles' K-blocks end to end and give every CTA an
// equal contiguous range of them (stream-K), so all SMs stream weights whatever
// the tile count.  Parts of a tile are added in CTA order,
// so results do not depend on timing.  The adding is done by kernels of its own:
// inside the GEMMs, by the CTA that finished a tile last, it held up that CTA's
// weight stream (128 tokens: 15 us per tile of phase 1, 35 us per tile of phase
// 2), and for one token it took as long as the extra launches do.  No CTA waits
// for another.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fp8fg_device.cuh"
#include "fp8fg_host.h"
#include "fp8fg_quant.cuh"
#include "fp8fg_swiglu.cuh"

namespace fp8fg {

namespace {

constexpr int kFewMaxCtas = 152;                // scratch is sized for this many
constexpr int BK = 128;
constexpr uint32_t WBLK_BYTES = 128 * BK;       // 128 weight rows of one K-block
constexpr uint32_t W_BYTES = 2 * WBLK_BYTES;    // two row blocks per stage
constexpr int NUM_PROMO_WARPS = 8;              // warps 0-3: block 0, 4-7: block 1
constexpr int PROMO_THREADS = 32 * NUM_PROMO_WARPS;
constexpr int WARP_TMA = 8, WARP_MMA = 9;
// The row form's 128 accumulators need more promotion registers than an even split gives: the kernel
// then launches a third whole warpgroup (TMA, MMA, 2 idle warps), which hands its registers over.
// (Spilled, the accumulators went through L2 -- shared memory leaves no L1 -- at 3 us per unit.)
__host__ __device__ constexpr int num_threads(int nb) { return nb == 128 ? 384 : PROMO_THREADS + 64; }
constexpr uint32_t LAUNCH_REGS = 168, CTRL_REGS = 72, PROMO_REGS = 216;
static_assert(128 * CTRL_REGS + 256 * PROMO_REGS <= 384 * LAUNCH_REGS, "register split exceeds the launch allocation");
constexpr int SLOTS = 8;                        // scale slots (at least MAX_STAGES + 2, see FewShared)
constexpr int MAX_STAGES = 6;
// A CTA takes at least this many units (or a whole tile): fewer would only leave more parts to add.
constexpr uint32_t MIN_UNITS = 2;
// And no more CTAs than this share a tile on average, or the kernels behind are busy adding its parts: up
// to 32 tokens (27 tokens, 34 experts of 512 x 1664 x 384: 41 us; 48 with 16 parts, 63 with 8), and more
// (87 tokens, 10 of 4096 x 128 x 6272: 36 us; 47 with 16 parts, 68 tokens, 24 of 1024 x 640 x 768: 36;
// 64 without a limit).
constexpr uint32_t MAX_PARTS = 32, MAX_PARTS_ROWS = 8;
// Ring bytes: up to 16 tokens leave room for a CTA of each phase on an SM (phase 2's first weights
// then load while phase 1 drains); more tokens get one CTA with a deeper ring.
__host__ __device__ constexpr uint32_t ring_budget(int nb) { return (nb <= 16 ? 104 : 216) * 1024; }
__host__ __device__ constexpr uint32_t stage_bytes(int nb) { return W_BYTES + (uint32_t)nb * BK; }
// Up to MAX_COLUMN_TOKENS tokens are the columns of the products (NB of them: 16 or 32), more are the 128
// rows.  A thread of the column form needs every token's scale, from shared memory, for each unit, and
// the MMAs read the weights 128 rows at a time for few columns; one of the row form needs one scale, but
// its stage always holds 128 token rows (4 stages instead of 6).  Of 16 experts of 7168 x 2048, columns
// took 144 us for 17 tokens and 167 for 64 (accumulators of 64), rows 154 and 151 to 156.
constexpr int MAX_COLUMN_TOKENS = 32;
__host__ __device__ constexpr bool token_rows(int nb) { return nb == 128; }
__host__ __device__ constexpr int num_stages(int nb)
{
    const int n = (int)(ring_budget(nb) / stage_bytes(nb));
    return n < MAX_STAGES ? n : MAX_STAGES;
}

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
    int withhold;           // self-test: the phase (1, 2) whose CTAs never load their first unit's tokens
    uint64_t timeout_ns;
    // workspace
    int32_t* n_act;         // [1] number of active experts,
    int32_t* act;           // [A] and they, in ascending order
    float* gate;            // [G][Tp] summed gate weight of token t for expert e
    uint8_t* xq;            // [T][K] codes of x, xs [K/128][Tp] their scales
    float* xs;
    uint8_t* aq;            // [A * Tp][I] codes, as [A][I/128][Tp] scales * gate weight
    float* as;
    float* part;            // [2 * CTAs][2][T * 128] parts of tiles that several CTAs share
    float* whole;           // [A * I/128][2][T * 128] phase 1's other tiles
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
    uint8_t* xq = take(T * K);
    uint8_t* xs = take(4 * (K / 128) * Tp);
    uint8_t* aq = take(A * Tp * I);
    uint8_t* as = take(4 * A * (I / 128) * Tp);
    uint8_t* part = take(4 * 2 * (int64_t)kFewMaxCtas * 2 * T * 128);
    uint8_t* whole = take(4 * A * (I / 128) * 2 * T * 128);
    if (f) {
        f->n_act = reinterpret_cast<int32_t*>(n_act);
        f->act = reinterpret_cast<int32_t*>(act);
        f->gate = reinterpret_cast<float*>(gate);
        f->xq = xq;
        f->xs = reinterpret_cast<float*>(xs);
        f->aq = aq;
        f->as = reinterpret_cast<float*>(as);
        f->part = reinterpret_cast<float*>(part);
        f->whole = reinterpret_cast<float*>(whole);
    }
    return off;
}

// Programmatic dependent launch: let the next kernel of the stream start its set-up (and, in
// k_few_gemm<2>, its weight loads), and wait until the kernel before has completed.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------ preparation

constexpr int kMaxExperts = 1024;

// The experts some token picked.
struct ExpertList {
    int n;
    uint32_t mask[kMaxExperts / 32];
    uint16_t id[kMaxExperts];             // in ascending order
};

// Lists the active experts, by the whole block, from topk.
__device__ __forceinline__ void list_experts(const Few& f, ExpertList& x)
{
    const int tid = threadIdx.x;
    if (tid < kMaxExperts / 32) x.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < f.T * f.k; i += blockDim.x) {
        const int32_t e = __ldg(f.topk + i);
        if (e >= 0 && e < f.G) atomicOr(&x.mask[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (tid < 32) {
        uint32_t w = x.mask[tid];
        int incl = __popc(w);
        const int mine = incl;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, d);
            if (tid >= d) incl += t;
        }
        for (int at = incl - mine; w; w &= w - 1) x.id[at++] = (uint16_t)(tid * 32 + __ffs(w) - 1);
        if (tid == 31) x.n = incl;
    }
    __syncthreads();
}

// Quantizes x (a half-warp per 1x128 group, as k_quant_1x128), fills the gate table and reports
// expert ids outside [0, G); the last block lists the active experts.
template <typename Tin>
__global__ void __launch_bounds__(256) k_few_prep(const Few f, const Tin* __restrict__ x, int64_t ldx)
{
    const int tid = threadIdx.x;
    launch_dependents();
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ ExpertList experts;
        list_experts(f, experts);
        for (int i = tid; i < experts.n; i += 256) f.act[i] = experts.id[i];
        if (tid == 0) *f.n_act = experts.n;
        return;
    }
    const uint32_t nkb = (uint32_t)(f.K / 128);
    const uint32_t grp = blockIdx.x * 16 + (tid >> 4);
    const int l = tid & 15;
    const uint32_t t = grp / nkb, kb = grp - t * nkb;
    const bool live = t < (uint32_t)f.T;
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
        if (l == 0) f.xs[(int64_t)kb * f.Tp + t] = g.s;
    }
    const int64_t step = ((int64_t)gridDim.x - 1) * 256, i0 = (int64_t)blockIdx.x * 256 + tid;
    for (int64_t i = i0; i < (int64_t)f.G * f.Tp; i += step) {
        const int e = (int)((uint32_t)i / (uint32_t)f.Tp), tt = (int)((uint32_t)i % (uint32_t)f.Tp);
        float sum = 0.0f;
        if (tt < f.T)
            for (int j = 0; j < f.k; ++j)
                if (__ldg(f.topk + tt * f.k + j) == e) sum += __ldg(f.weights + tt * f.k + j);
        f.gate[i] = sum;
    }
    for (int64_t i = i0; i < (int64_t)f.T * f.k; i += step) {
        const int32_t e = __ldg(f.topk + i);
        if (e < 0 || e >= f.G) report_error(FP8_ERR_SHAPE);
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

// The same for data that is read once: its L2 lines are the first to go, so that the activations and
// partial sums written in between stay.
__device__ __forceinline__ uint64_t policy_evict_first()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_2d_once(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                                 int32_t y, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
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

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }

// ------------------------------------------------------------ GEMM

template <int NB>
struct __align__(16) FewShared {
    // A unit's scales arrive with its operands, in slot (unit number) % 8: the weight scale of
    // each row block and the tokens' scales.  A slot is refilled 8 units later, behind the MMA of the unit
    // that had the ring's stage before: at most 6 back (the ring's depth), and itself behind the promotion of
    // the unit 2 before it.  So the readers of a slot are done if NS + 2 <= SLOTS.
    float tok[SLOTS][NB];
    float wsc[SLOTS][2];
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    ExpertList experts;
};

// The units (tile, K-block) of all tiles end to end, and this CTA's range.  A unit is 32 KB of
// weights, so unit counts times 152 CTAs fit in 32 bits for any memory.
struct Range {
    uint32_t U, P, per;     // units, CTAs that have work, units per tile
    uint32_t u0, u1;
    __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * U / P; }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const { return ((u + 1) * P - 1) / U; }
};

template <int PHASE>
__device__ __forceinline__ Range few_range(const Few& f, int n_act, uint32_t ctas)
{
    Range r;
    const uint32_t J = (uint32_t)(f.I / 128);
    r.per = PHASE == 1 ? (uint32_t)(f.K / BK) : n_act * J;
    r.U = (PHASE == 1 ? n_act * J : (n_act ? (uint32_t)((f.N + 255) / 256) : 0)) * r.per;
    const uint32_t tiles = r.per ? r.U / r.per : 0, want = r.U / MIN_UNITS > tiles ? r.U / MIN_UNITS : tiles;
    r.P = min(min(want, ctas), tiles * (f.Tp > MAX_COLUMN_TOKENS ? MAX_PARTS_ROWS : MAX_PARTS));
    r.u0 = blockIdx.x < r.P ? r.begin(blockIdx.x) : 0;
    r.u1 = blockIdx.x < r.P ? r.begin(blockIdx.x + 1) : 0;
    return r;
}

// A walk over a range's units without divisions: tile, K-block in the tile, and the (active
// expert, 128-channel block of I) the unit's weights belong to.
template <int PHASE>
struct Walk {
    const uint16_t* act;
    uint32_t J, per, u, tile, kb, a, j;
    int32_t e;              // active expert a
    __device__ __forceinline__ Walk(const Few& f, const uint16_t* experts, const Range& r)
        : act(experts), J((uint32_t)(f.I / 128)), per(r.per), u(r.u0), tile(0), kb(0), a(0), j(0), e(0)
    {
        if (r.u0 >= r.u1) return;
        tile = u / per;
        kb = u - tile * per;
        const uint32_t aj = PHASE == 1 ? tile : kb;
        a = aj / J;
        j = aj - a * J;
        e = act[a];
    }
    __device__ __forceinline__ void next(uint32_t u1)
    {
        ++u;
        ++kb;
        bool step = PHASE == 2;
        if (kb == per) {
            kb = 0;
            ++tile;
            step = true;
        }
        if (!step) return;
        if (++j == J) {
            j = 0;
            ++a;
            if (PHASE == 2 && kb == 0) a = 0;
            if (u < u1) e = act[a];
        }
    }
};

// 16-byte multiples global -> shared, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// A tile into L2 only.
__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap* map, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// A CTA lets the next kernel start when this many of its units are left to load.
constexpr uint32_t TRIGGER_UNITS = 4;
// Units of its successor's that it fetches into L2 at its end (4 to 12 measure the same; 24 cost 3 us).
constexpr int PREFETCH_UNITS = 8;

// Run by the whole of a warp: lane 0 arms the stage barrier and issues its TMA and bulk copies,
// lanes 0 and 1 each copy one row block's weight scale (4 bytes, cp.async) and arrive when it
// has landed.
template <int PHASE, int NB>
__device__ void few_producer(const CUtensorMap* tmW, const CUtensorMap* tmX, const CUtensorMap* tmNext,
                             const Few& f, const Range& r,
                             uint8_t* smem, FewShared<NB>& sh, int lane)
{
    constexpr int NS = num_stages(NB);
    const int64_t J = f.I / 128, nb128 = f.N / 128, nkb = f.K / BK;
    const uint32_t bytes = W_BYTES + (uint32_t)f.Tp * (BK + 4);
    const uint64_t once = policy_evict_first();
    auto weights = [&](const Walk<PHASE>& k, uint32_t it) {
        const int s = (int)(it % NS);
        uint8_t* dst = smem + s * stage_bytes(NB);
        if (lane == 0) {
            mbar_arrive_expect_tx(&sh.full[s], bytes);
            // the second block of an odd last output tile lies past this expert's rows: never stored
            const int32_t r0 = (int32_t)(PHASE == 1 ? k.e * 2 * f.I + k.j * 128 : k.e * f.N + k.tile * 256);
            const int32_t r1 = PHASE == 1 ? r0 + (int32_t)f.I : r0 + 128;
            const int32_t x = (int32_t)((PHASE == 1 ? k.kb : k.j) * BK);
            tma_load_2d_once(dst, tmW, &sh.full[s], x, r0, once);
            tma_load_2d_once(dst + WBLK_BYTES, tmW, &sh.full[s], x, r1, once);
        }
        if (lane < 2) {
            const int64_t nb = 2 * (int64_t)k.tile + lane;
            const bool live = PHASE == 1 || nb < nb128;
            const float* src = PHASE == 1 ? f.s13 + (k.e * 2 * J + lane * J + k.j) * nkb + k.kb
                                          : f.s2 + (live ? (k.e * nb128 + nb) * J + k.j : 0);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&sh.wsc[it % SLOTS][lane])),
                         "l"(src), "r"(live ? 4 : 0)
                         : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[s]))
                         : "memory");
        }
        __syncwarp();
    };
    auto tokens = [&](const Walk<PHASE>& k, uint32_t it) {
        const int s = (int)(it % NS);
        if (lane == 0 && (it > 0 || f.withhold != PHASE)) {
            tma_load_2d(smem + s * stage_bytes(NB) + W_BYTES, tmX, &sh.full[s],
                        (int32_t)((PHASE == 1 ? k.kb : k.j) * BK), PHASE == 1 ? 0 : (int32_t)(k.a * f.Tp));
            bulk_load(sh.tok[it % SLOTS], (PHASE == 1 ? f.xs : f.as) + (int64_t)k.kb * f.Tp, (uint32_t)f.Tp * 4,
                      &sh.full[s]);
        }
        __syncwarp();
    };
    // the ring's first weights do not depend on the kernel before
    Walk<PHASE> k(f, sh.experts.id, r), ahead = k;
    uint32_t it = 0, n = 0;
    // (loops kept rolled: a CTA's first pass through code waits for instruction fetches)
#pragma unroll 1
    for (; n < NS && ahead.u < r.u1; ++n, ahead.next(r.u1)) weights(ahead, n);
    wait_previous();
    // The kernels behind may start from this kernel's triggers on, and read what k_few_prep wrote (expert list,
    // gate weights) before their own waits: no trigger may come before the wait above.
    bool triggered = false;
#pragma unroll 1
    for (; k.u < r.u1; ++it, k.next(r.u1)) {
        if (!triggered && r.u1 - k.u <= TRIGGER_UNITS) {
            launch_dependents();
            triggered = true;
        }
        if (it >= n) {
            const bool ok = mbar_wait(&sh.empty[it % NS], ((it / NS) & 1) ^ 1u, &sh.abort, f.timeout_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            weights(k, it);
        }
        tokens(k, it);
    }
    if (!triggered) launch_dependents();
    if (PHASE == 1 && lane == 0) {
        // While this kernel's last tiles are finished and the next one starts, HBM would idle: the
        // weights that this CTA's successor reads behind its ring's first ones go to L2.
        const Range r2 = few_range<2>(f, sh.experts.n, gridDim.x);
        Walk<2> w(f, sh.experts.id, r2);
#pragma unroll 1
        for (int i = 0; i < PREFETCH_UNITS && w.u < r2.u1; ++i, w.next(r2.u1)) {
            const int32_t r0 = (int32_t)(w.e * f.N + w.tile * 256);
            tma_prefetch_l2(tmNext, (int32_t)(w.j * BK), r0);
            if (w.tile * 256 + 128 < f.N) tma_prefetch_l2(tmNext, (int32_t)(w.j * BK), r0 + 128);
        }
    }
    // every copy issued lands before the CTA exits
    if (lane == 0)
        for (int s = 0; s < NS; ++s) {
            const uint32_t count = it > (uint32_t)s ? (it - s + NS - 1) / NS : 0;
            if (count) mbar_wait_drain(&sh.full[s], (count - 1) & 1, f.timeout_ns);
        }
}

template <int NB>
__device__ void few_mma(const Few& f, const Range& r, uint8_t* smem, FewShared<NB>& sh)
{
    constexpr int NS = num_stages(NB);
    const uint32_t base = smem_u32(smem);
    const uint32_t idesc = token_rows(NB) ? idesc_e4m3_f32(128, 256, 0) : idesc_e4m3_f32(128, (uint32_t)f.Tp, 0);
    const uint32_t units = r.u1 - r.u0;
#pragma unroll 1
    for (uint32_t it = 0; it < units; ++it) {
        const int s = (int)(it % NS);
        const uint32_t buf = it & 1;
        if (!mbar_wait(&sh.tempty[buf], ((it >> 1) & 1) ^ 1u, &sh.abort, f.timeout_ns) ||
            !mbar_wait(&sh.full[s], (it / NS) & 1, &sh.abort, f.timeout_ns))
            break;
        tc_fence_after();
        const uint32_t wa = base + s * stage_bytes(NB);
        const uint32_t d = sh.tmem_base + buf * 2 * NB;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {
            const uint64_t xd = smem_desc_sw128(wa + W_BYTES + k * 32, 16, 1024);
            const uint64_t wd = smem_desc_sw128(wa + k * 32, 16, 1024);
            if (token_rows(NB)) {       // the two row blocks are 256 adjacent rows
                mma_f8f6f4(d, xd, wd, idesc, k > 0);
            } else {
                mma_f8f6f4(d, wd, xd, idesc, k > 0);
                mma_f8f6f4(d + NB, smem_desc_sw128(wa + WBLK_BYTES + k * 32, 16, 1024), xd, idesc, k > 0);
            }
        }
        mma_commit(&sh.empty[s]);
        mma_commit(&sh.tfull[buf]);
    }
    mma_commit(&sh.drain);
    mbar_wait_drain(&sh.drain, 0, f.timeout_ns);
}

// The parts of a tile: CTAs c0..c1 hold one each, in slots of `stride` floats: two row
// blocks of [T][128], or, with tokens as rows, [128 / 4][T][4], as the promotion's threads can write whole
// lines.
struct Parts {
    const float* part;
    Range r;
    uint32_t c0, c1, tile_u0;
    int64_t stride;
    __device__ __forceinline__ Parts(const Few& f, const Range& range, uint32_t u0)
        : part(f.part), r(range), c0(range.owner(u0)), c1(range.owner(u0 + range.per - 1)), tile_u0(u0),
          stride((int64_t)2 * f.T * 128)
    {
    }
    __device__ __forceinline__ const float* at(uint32_t c) const
    {
        // a CTA whose range begins inside the tile left its part in slot 0
        return part + (2 * c + (r.begin(c) >= tile_u0 ? 0 : 1)) * stride;
    }
};

__device__ __forceinline__ void store_out(const Few& f, int t, int64_t n, float v)
{
    if (f.out_dtype == FP8_OUT_BF16)
        static_cast<__nv_bfloat16*>(f.out)[t * f.ldo + n] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(f.out)[t * f.ldo + n] = v;
}

// Eight adjacent outputs of a token (rows are 16-byte aligned).
__device__ __forceinline__ void store_out8(const Few& f, int t, int64_t n, const float* v)
{
    if (f.out_dtype == FP8_OUT_BF16) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.out) + t * f.ldo + n) = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(f.out) + t * f.ldo + n);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// The promotion with tokens as the accumulator's columns: thread = row of a block of the weights.
template <int PHASE, int NB>
__device__ void few_promotion(const Few& f, const Range& r, FewShared<NB>& sh)
{
    static_assert(NB <= 32, "a column's tokens are bits of one word");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = warp >> 2, row = tid & 127;
    const uint32_t tmem = sh.tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + blk * NB;
    uint32_t it = 0;
    int seg = 0;
    wait_previous();
    Walk<PHASE> k(f, sh.experts.id, r);
    for (; k.u < r.u1; ++seg) {
        const uint32_t tile = k.tile, tile_u0 = k.u - k.kb;
        // phase 1: which tokens were routed to the tile's expert (gate weight not 0)
        uint32_t routed = 0;
        if (PHASE == 1)
            routed = __ballot_sync(0xffffffffu, lane < f.T && __ldcg(f.gate + (int64_t)k.e * f.Tp + lane) != 0.0f);
        const uint32_t end = r.u1 < tile_u0 + r.per ? r.u1 : tile_u0 + r.per;
        float acc[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = 0.0f;
#pragma unroll 1
        for (; k.u < end; k.next(r.u1), ++it) {
            const uint32_t buf = it & 1;
            // the whole warp goes on or gives up (TMEM loads are warp-wide)
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.tfull[buf], (it >> 1) & 1, &sh.abort, f.timeout_ns))) return;
            tc_fence_after();
            const float* vec = sh.tok[it % SLOTS];
            const float sw = sh.wsc[it % SLOTS][blk];
            const uint32_t t = tmem + buf * 2 * NB;
            // phase 2: the columns that have a scale.  The others' products are not added, not even times
            // 0: an expert whose weights or scales hold a NaN or infinity spoils only its own tokens.
            uint32_t takes = 0;
            if (PHASE == 2) takes = __ballot_sync(0xffffffffu, lane < NB && vec[lane] != 0.0f);
            uint32_t p[NB];
            tmem_ld(t, p);
            tmem_ld_wait(p);
#pragma unroll
            for (int i = 0; i < NB; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(vec + i);
                if (PHASE == 1) {
                    float s0, s1, s2, s3;
                    fmul2(s0, s1, x.x, x.y, sw, sw);
                    fmul2(s2, s3, x.z, x.w, sw, sw);
                    ffma2(acc[i], acc[i + 1], __uint_as_float(p[i]), __uint_as_float(p[i + 1]), s0, s1);
                    ffma2(acc[i + 2], acc[i + 3], __uint_as_float(p[i + 2]), __uint_as_float(p[i + 3]), s2, s3);
                } else {
                    if ((takes >> i) & 1) acc[i] = fmaf(__uint_as_float(p[i]), x.x * sw, acc[i]);
                    if ((takes >> i) & 2) acc[i + 1] = fmaf(__uint_as_float(p[i + 1]), x.y * sw, acc[i + 1]);
                    if ((takes >> i) & 4) acc[i + 2] = fmaf(__uint_as_float(p[i + 2]), x.z * sw, acc[i + 2]);
                    if ((takes >> i) & 8) acc[i + 3] = fmaf(__uint_as_float(p[i + 3]), x.w * sw, acc[i + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.tempty[buf]);
        }

        // The sums, or this CTA's part of them: for k_few_act (phase 1), for k_few_out, or done.
        const Parts p(f, r, tile_u0);
        const bool shared = p.c1 > p.c0;
        if (PHASE == 1 || shared) {
            float* dst = (shared ? f.part + (2 * (int64_t)blockIdx.x + (seg ? 1 : 0)) * p.stride
                                 : f.whole + (int64_t)tile * p.stride) +
                         (int64_t)blk * f.T * 128 + row;
#pragma unroll
            for (int t = 0; t < NB; ++t)
                if (PHASE == 1 ? (routed >> t) & 1 : t < f.T) __stcg(dst + t * 128, acc[t]);
        } else if (tile * 256 + (int64_t)tid < f.N) {
#pragma unroll
            for (int t = 0; t < NB; ++t)
                if (t < f.T) store_out(f, t, tile * 256 + (int64_t)tid, acc[t]);
        }
    }
}

// The promotion with tokens as the accumulator's rows: thread = token, and row block of the weights.
template <int PHASE, int NB>
__device__ void few_promotion_rows(const Few& f, const Range& r, FewShared<NB>& sh)
{
    static_assert(NB == 128, "a thread's 128 accumulators are a row block's columns");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = warp >> 2, tok = tid & 127;
    const uint32_t tmem = sh.tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + blk * NB;
    uint32_t it = 0;
    int seg = 0;
    wait_previous();
    Walk<PHASE> k(f, sh.experts.id, r);
    for (; k.u < r.u1; ++seg) {
        const uint32_t tile = k.tile, tile_u0 = k.u - k.kb;
        // phase 1: only tokens routed to the tile's expert (gate weight not 0) matter, and their sums are
        // stored without gaps
        bool routed = tok < f.T;
        int at = tok;
        if (PHASE == 1) {
            uint32_t word[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 32 * i + lane;
                word[i] = __ballot_sync(0xffffffffu, t < f.T && __ldcg(f.gate + (int64_t)k.e * f.Tp + t) != 0.0f);
            }
            at = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i == (warp & 3)) {
                    routed = (word[i] >> lane) & 1;
                    at += __popc(word[i] & ((1u << lane) - 1));
                }
                if (i < (warp & 3)) at += __popc(word[i]);
            }
        }
        const uint32_t end = r.u1 < tile_u0 + r.per ? r.u1 : tile_u0 + r.per;
        float acc[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = 0.0f;
#pragma unroll 1
        for (; k.u < end; k.next(r.u1), ++it) {
            const uint32_t buf = it & 1;
            // the whole warp goes on or gives up (TMEM loads are warp-wide)
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.tfull[buf], (it >> 1) & 1, &sh.abort, f.timeout_ns))) return;
            tc_fence_after();
            const float x = sh.tok[it % SLOTS][tok], s = x * sh.wsc[it % SLOTS][blk];
            // Phase 2: a token that did not pick the unit's expert has scale 0 here.  Its products are not
            // added, not even times 0: an expert whose weights or scales hold a NaN or infinity spoils
            // only its own tokens.
            const bool on = routed && (PHASE == 1 || x != 0.0f);
            if (__any_sync(0xffffffffu, on)) {
                const uint32_t t = tmem + buf * 2 * NB;
                constexpr int CH = 32;
                uint32_t pa[CH], pb[CH];
                tmem_ld(t, pa);
#pragma unroll
                for (int c = 0; c < NB; c += CH) {
                    uint32_t (&p)[CH] = (c & CH) ? pb : pa;
                    uint32_t (&q)[CH] = (c & CH) ? pa : pb;
                    tmem_ld_wait(p);
                    if (c + CH < NB) tmem_ld(t + c + CH, q);
                    if (on)
#pragma unroll
                        for (int i = 0; i < CH; i += 2)
                            ffma2(acc[c + i], acc[c + i + 1], __uint_as_float(p[i]), __uint_as_float(p[i + 1]), s, s);
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.tempty[buf]);
        }

        const Parts p(f, r, tile_u0);
        const bool shared = p.c1 > p.c0;
        if (PHASE == 1 || shared) {
            if (!routed) continue;
            float* dst = (shared ? f.part + (2 * (int64_t)blockIdx.x + (seg ? 1 : 0)) * p.stride
                                 : f.whole + (int64_t)tile * p.stride) +
                         (int64_t)blk * f.T * 128 + at * 4;
#pragma unroll
            for (int i = 0; i < NB; i += 4)
                __stcg(reinterpret_cast<float4*>(dst + i * f.T),
                       make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]));
        } else if (tok < f.T && tile * 256 + (int64_t)blk * 128 < f.N) {
#pragma unroll
            for (int i = 0; i < NB; i += 8) store_out8(f, tok, tile * 256 + (int64_t)(blk * 128 + i), acc + i);
        }
    }
}

template <int PHASE, int NB>
__global__ void __launch_bounds__(num_threads(NB), NB <= 16 ? 2 : 1)
    k_few_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmNext, const Few f)
{
    // the ring first: its tiles need 1024-byte alignment (128-byte swizzle atoms)
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int NS = num_stages(NB);
    FewShared<NB>& sh = *reinterpret_cast<FewShared<NB>*>(smem + NS * stage_bytes(NB));
    constexpr uint32_t TMEM_COLS = 4 * NB;     // two buffers of two blocks' NB columns
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512 && NS >= 2 && NS + 2 <= SLOTS, "TMEM columns, ring depth");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 3);     // lane 0's bytes, two scales
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

    // Phase 1 lists the active experts itself, so that its first weights can be on their way while
    // k_few_prep still runs.  Phase 2 reads the list: phase 1 let the kernels behind it start only after
    // it had seen k_few_prep complete.
    if (PHASE == 1) {
        list_experts(f, sh.experts);
    } else {
        const int A = f.T * f.k < f.G ? f.T * f.k : f.G;
        if (threadIdx.x == 0) sh.experts.n = __ldcg(f.n_act);
        for (int i = threadIdx.x; i < A; i += blockDim.x) sh.experts.id[i] = (uint16_t)__ldcg(f.act + i);
        __syncthreads();
    }
    const Range r = few_range<PHASE>(f, sh.experts.n, gridDim.x);
    if (warp >= NUM_PROMO_WARPS) {
        if (num_threads(NB) == 384) regs_dec<CTRL_REGS>();
        if (warp == WARP_TMA) {
            few_producer<PHASE, NB>(&tmW, &tmX, &tmNext, f, r, smem, sh, lane);
        } else if (warp == WARP_MMA && lane == 0) {
            few_mma<NB>(f, r, smem, sh);
        }
        __syncwarp();
    } else {
        if (num_threads(NB) == 384) regs_inc<PROMO_REGS>();
        if constexpr (token_rows(NB))
            few_promotion_rows<PHASE, NB>(f, r, sh);
        else
            few_promotion<PHASE, NB>(f, r, sh);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
}

// Up to 32 tokens.  Block = (tile of phase 1, every gridDim.y-th 8 tokens): adds its parts for the tokens routed to its expert,
// thread = channel; SwiGLU and 1x128 quantization.  Tokens not routed here (gate weight 0)
// get scale 0, for which phase 2 adds nothing, whatever their codes are.  Everything but the parts is known (k_few_prep had completed before phase 1
// let this kernel start), and done, before phase 1 ends.
constexpr int ACT_TOKENS = 8;

__global__ void __launch_bounds__(128) k_few_act(const Few f, uint32_t ctas)
{
    __shared__ float wmax[4][ACT_TOKENS];
    __shared__ __align__(16) uint8_t codes[ACT_TOKENS][128];
    __shared__ uint8_t tcol[32];
    const int tid = threadIdx.x, lane = tid & 31, w4 = tid >> 5;
    launch_dependents();
    const uint32_t J = (uint32_t)(f.I / 128), tile = blockIdx.x, a = tile / J, j = tile - a * J;
    const int n_act = __ldcg(f.n_act);
    const bool live = (int)a < n_act;
    float gw = 0.0f;                          // gate weight of token `lane`
    if (live && lane < f.T) gw = __ldcg(f.gate + (int64_t)__ldcg(f.act + a) * f.Tp + lane);
    const uint32_t routed = __ballot_sync(0xffffffffu, gw != 0.0f);
    if (tid < 32 && gw != 0.0f) tcol[__popc(routed & ((1u << lane) - 1))] = (uint8_t)lane;
    const int n = __popc(routed);
    const Range r = few_range<1>(f, live ? n_act : 1, ctas);
    const Parts p(f, r, (live ? tile : 0) * r.per);
    __syncthreads();
    if (!live || (blockIdx.y > 0 && (int)blockIdx.y * ACT_TOKENS >= n)) {
        wait_previous();
        return;
    }
    const int64_t row0 = (int64_t)a * f.Tp;                          // of aq
    float* const as = f.as + (int64_t)tile * f.Tp;
    uint8_t* const aq = f.aq + row0 * f.I + j * 128;
    const int i8 = lane & (ACT_TOKENS - 1);
    // A rehearsal of one round while phase 1 still runs, on numbers that are not used, fetches the
    // instructions: cold, they took longer (3.5 us) than the loads.  (The compiler must not know the
    // first round's number: it would peel that round off, into code of its own.)
    int round = -1;
    asm volatile("" : "+r"(round));
#pragma unroll 1
    for (; round * ACT_TOKENS < n; round += round < 0 ? 1 + (int)blockIdx.y : (int)gridDim.y) {
        const bool real = round >= 0;
        const int c = real ? round * ACT_TOKENS : 0;
        if (round == (int)blockIdx.y) wait_previous();
        float g[ACT_TOKENS], u[ACT_TOKENS];
#pragma unroll
        for (int i = 0; i < ACT_TOKENS; ++i) g[i] = u[i] = 0.0f;
#pragma unroll 1
        for (uint32_t q = p.c0; q <= p.c1; ++q) {
            int now = round;                  // (hidden again, as is what follows from it: no second copy of this
                                              // loop or of its loads either, which costs 4 us)
            asm volatile("" : "+r"(now));
            const float* src = (p.c0 == p.c1 ? f.whole + (int64_t)tile * p.stride : p.at(q)) + tid;
            if (now < 0) src = f.gate;
            int up = now < 0 ? 0 : f.T * 128, mul = now < 0 ? 0 : 128;
            asm volatile("" : "+l"(src), "+r"(up), "+r"(mul));
            float x[2][ACT_TOKENS];           // all in flight at once; past the last column, one not used
#pragma unroll
            for (int i = 0; i < ACT_TOKENS; ++i) {
                const float* col = src + tcol[c + i < n ? c + i : 0] * mul;
                x[0][i] = __ldcg(col);
                x[1][i] = __ldcg(col + up);
            }
#pragma unroll
            for (int i = 0; i < ACT_TOKENS; ++i) {
                g[i] += x[0][i];
                u[i] += x[1][i];
            }
        }
#pragma unroll
        for (int i = 0; i < ACT_TOKENS; i += 2) {
            const F2 a = silu2<true>(f2(g[i], g[i + 1])) * f2(u[i], u[i + 1]);
            g[i] = lo(a);
            g[i + 1] = hi(a);
        }
#pragma unroll
        for (int i = 0; i < ACT_TOKENS; ++i) {
            const float m = warp_absmax(g[i]);
            if (lane == 0) wmax[w4][i] = m;
        }
        __syncthreads();
        // lane i derives the scale of column c + i
        const GroupScale gs =
            group_scale(fmaxf(fmaxf(wmax[0][i8], wmax[1][i8]), fmaxf(wmax[2][i8], wmax[3][i8])), f.mode);
        const int t = c + i8 < n ? tcol[c + i8] : 0;
        const float wt = __shfl_sync(0xffffffffu, gw, t);
        if (real && tid < ACT_TOKENS && c + i8 < n) as[t] = gs.s * wt;
#pragma unroll
        for (int k = 0; k < ACT_TOKENS; ++k)
            codes[k][tid] = (uint8_t)encode4(g[k], 0.f, 0.f, 0.f, __shfl_sync(0xffffffffu, gs.inv, k));
        __syncthreads();
        if (real && tid < ACT_TOKENS * 8 && c + (tid >> 3) < n)
            *reinterpret_cast<uint4*>(aq + (int64_t)tcol[c + (tid >> 3)] * f.I + (tid & 7) * 16) =
                *reinterpret_cast<const uint4*>(&codes[tid >> 3][(tid & 7) * 16]);
        // (the next round's writes of codes follow a barrier that these reads precede)
    }
    if (n == 0) wait_previous();
    if (blockIdx.y == 0 && tid < 32 && lane < f.T && gw == 0.0f) as[lane] = 0.0f;
}

// The same behind few_promotion_rows, whose sums lie [channel / 4][token][4]: block = (tile of phase 1,
// every gridDim.y-th 32 of the tokens routed to its expert), thread = token and 32 channels, so that all lanes work and a
// token's 64 values need no shuffle.  Codes of tokens not routed here are left as they are: phase 2 does
// not add what it makes of them.
__global__ void __launch_bounds__(128) k_few_act_rows(const Few f, uint32_t ctas)
{
    __shared__ float wmax[4][32], gcol[128];
    __shared__ uint32_t words[4];
    __shared__ uint8_t tcol[128];
    const int tid = threadIdx.x, lane = tid & 31, w4 = tid >> 5;
    launch_dependents();
    const uint32_t J = (uint32_t)(f.I / 128), tile = blockIdx.x, a = tile / J, j = tile - a * J;
    const int n_act = __ldcg(f.n_act), e = __ldcg(f.act + a);
    const bool live = (int)a < n_act;
    float gw = 0.0f;                          // gate weight of token tid
    if (live && tid < f.T) gw = __ldcg(f.gate + (int64_t)e * f.Tp + tid);
    const uint32_t word = __ballot_sync(0xffffffffu, gw != 0.0f);
    if (lane == 0) words[w4] = word;
    __syncthreads();
    int n = 0, rank = __popc(word & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < w4) rank += __popc(words[w]);
        n += __popc(words[w]);
    }
    if (gw != 0.0f) {
        tcol[rank] = (uint8_t)tid;
        gcol[rank] = gw;
    }
    __syncthreads();
    const Range r = few_range<1>(f, live ? n_act : 1, ctas);
    const Parts p(f, r, (live ? tile : 0) * r.per);
    wait_previous();
    if (live && blockIdx.y == 0 && tid < f.T && gw == 0.0f) f.as[(int64_t)tile * f.Tp + tid] = 0.0f;
#pragma unroll 1
    for (int c0 = 32 * blockIdx.y; c0 < n; c0 += 32 * gridDim.y) {
        const bool on = c0 + lane < n;
        const int at = on ? c0 + lane : c0, t = tcol[at];
        F2 g[16], u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = u[i] = f2(0.0f, 0.0f);
#pragma unroll 1
        for (uint32_t q = p.c0; q <= p.c1; ++q) {
            const float* src = (p.c0 == p.c1 ? f.whole + (int64_t)tile * p.stride : p.at(q)) + w4 * 32 * f.T + at * 4;
            float4 x[2][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[0][i] = __ldcg(reinterpret_cast<const float4*>(src + 4 * i * f.T));
                x[1][i] = __ldcg(reinterpret_cast<const float4*>(src + 4 * i * f.T + f.T * 128));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[2 * i] = g[2 * i] + f2(x[0][i].x, x[0][i].y);
                g[2 * i + 1] = g[2 * i + 1] + f2(x[0][i].z, x[0][i].w);
                u[2 * i] = u[2 * i] + f2(x[1][i].x, x[1][i].y);
                u[2 * i + 1] = u[2 * i + 1] + f2(x[1][i].z, x[1][i].w);
            }
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            g[i] = silu2<true>(g[i]) * u[i];
            m = absmax3(m, lo(g[i]), hi(g[i]));
        }
        __syncthreads();                      // (the round before has read wmax)
        wmax[w4][lane] = m;
        __syncthreads();
        const GroupScale gs =
            group_scale(fmaxf(absmax3(wmax[0][lane], wmax[1][lane], wmax[2][lane]), wmax[3][lane]), f.mode);
        if (!on) continue;
        if (w4 == 0) f.as[(int64_t)tile * f.Tp + t] = gs.s * gcol[at];
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = encode4(lo(g[2 * i]), hi(g[2 * i]), lo(g[2 * i + 1]), hi(g[2 * i + 1]), gs.inv);
        uint4* dst = reinterpret_cast<uint4*>(f.aq + ((int64_t)a * f.Tp + t) * f.I + j * 128 + w4 * 32);
        dst[0] = make_uint4(c[0], c[1], c[2], c[3]);
        dst[1] = make_uint4(c[4], c[5], c[6], c[7]);
    }
}

// Output columns whose sums are in parts (the whole tiles are written already): block =
// 256 columns x OUT_TOKENS tokens, a thread one column, with the loads of OUT_PARTS parts in flight
// at once.  With no valid expert at all, the sum over none.
constexpr int OUT_TOKENS = 2, OUT_PARTS = 8;

__global__ void __launch_bounds__(256) k_few_out(const Few f, uint32_t ctas)
{
    // k_few_prep had completed long before phase 2 let this kernel start
    const int n_act = __ldcg(f.n_act);
    const int t0 = blockIdx.y * OUT_TOKENS, blk = threadIdx.x >> 7, row = threadIdx.x & 127;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const Range r = few_range<2>(f, n_act ? n_act : 1, ctas);
    const Parts p(f, r, blockIdx.x * r.per);
    const int64_t at = (int64_t)blk * f.T * 128 + (int64_t)t0 * 128 + row;
    wait_previous();
    if (n >= f.N || (n_act && p.c0 == p.c1)) return;
    float v[OUT_TOKENS];
#pragma unroll
    for (int i = 0; i < OUT_TOKENS; ++i) v[i] = 0.0f;
    if (n_act) {
#pragma unroll 1
        for (uint32_t c = p.c0; c <= p.c1; c += OUT_PARTS) {
            float x[OUT_PARTS][OUT_TOKENS];
#pragma unroll
            for (int q = 0; q < OUT_PARTS; ++q) {
                const float* src = p.at(c + q <= p.c1 ? c + q : p.c1) + at;
#pragma unroll
                for (int i = 0; i < OUT_TOKENS; ++i) x[q][i] = __ldcg(src + (t0 + i < f.T ? i * 128 : 0));
            }
#pragma unroll
            for (int q = 0; q < OUT_PARTS; ++q)
#pragma unroll
                for (int i = 0; i < OUT_TOKENS; ++i) v[i] += c + q <= p.c1 ? x[q][i] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < OUT_TOKENS; ++i)
        if (t0 + i < f.T) store_out(f, t0 + i, n, v[i]);
}

// The same behind few_promotion_rows: block = (64 columns, 32 tokens), warp = 8 adjacent columns, thread = one
// token's 8.
constexpr int OUT_ROWS_PARTS = 4;

__global__ void __launch_bounds__(256) k_few_out_rows(const Few f, uint32_t ctas)
{
    const int n_act = __ldcg(f.n_act), lane = threadIdx.x & 31, t = 32 * blockIdx.y + lane;
    const uint32_t tile = blockIdx.x >> 2;
    const int col = (int)(blockIdx.x & 3) * 64 + (int)(threadIdx.x >> 5) * 8;         // of the tile
    const int64_t n = (int64_t)tile * 256 + col;
    const Range r = few_range<2>(f, n_act ? n_act : 1, ctas);
    const Parts p(f, r, tile * r.per);
    const int at = (col >> 7) * f.T * 128 + (col & 127) * f.T + (t < f.T ? t : 0) * 4;
    wait_previous();
    if (n >= f.N || t >= f.T || (n_act && p.c0 == p.c1)) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (n_act) {
#pragma unroll 1
        for (uint32_t c = p.c0; c <= p.c1; c += OUT_ROWS_PARTS) {
            float4 x[OUT_ROWS_PARTS][2];
#pragma unroll
            for (int q = 0; q < OUT_ROWS_PARTS; ++q) {
                const float* src = p.at(c + q <= p.c1 ? c + q : p.c1) + at;
                x[q][0] = __ldcg(reinterpret_cast<const float4*>(src));
                x[q][1] = __ldcg(reinterpret_cast<const float4*>(src + 4 * f.T));
            }
#pragma unroll
            for (int q = 0; q < OUT_ROWS_PARTS; ++q) {
                if (c + q > p.c1) break;
                v[0] += x[q][0].x, v[1] += x[q][0].y, v[2] += x[q][0].z, v[3] += x[q][0].w;
                v[4] += x[q][1].x, v[5] += x[q][1].y, v[6] += x[q][1].z, v[7] += x[q][1].w;
            }
        }
    }
    store_out8(f, t, n, v);
}

// ------------------------------------------------------------ host side

template <int NB>
int launch_few_gemms(const Few& f, const CUtensorMap& tmW13, const CUtensorMap& tmW2, const CUtensorMap& tmX,
                     const CUtensorMap& tmA, unsigned ctas, cudaStream_t st)
{
    constexpr uint32_t smem = num_stages(NB) * stage_bytes(NB) + (uint32_t)sizeof(FewShared<NB>);
    static_assert(smem <= (NB <= 16 ? 116736u - 1024u : 232448u), "shared memory of a CTA (two per SM up to 16 tokens)");
    if (allow_smem<k_few_gemm<1, NB>>((int)smem) != cudaSuccess || allow_smem<k_few_gemm<2, NB>>((int)smem) != cudaSuccess)
        return FP8_ERR_LAUNCH;
    // both may start while the kernel before them in the stream still runs
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(num_threads(NB), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_few_gemm<1, NB>, tmW13, tmX, tmW2, f) != cudaSuccess) return FP8_ERR_LAUNCH;
    const int64_t A = (int64_t)f.T * f.k < f.G ? (int64_t)f.T * f.k : f.G;
    cudaLaunchConfig_t act = cfg;
    // the tokens of a tile in several blocks where there are few tiles
    const unsigned tiles = (unsigned)(A * (f.I / 128)), spread = (2 * ctas + tiles - 1) / tiles;
    const unsigned most = token_rows(NB) ? 4 : (unsigned)(f.T + ACT_TOKENS - 1) / ACT_TOKENS;
    act.gridDim = dim3(tiles, max(token_rows(NB) ? 2u : 1u, min(spread, most)), 1);
    act.blockDim = dim3(128, 1, 1);
    act.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&act, token_rows(NB) ? k_few_act_rows : k_few_act, f, (uint32_t)ctas) != cudaSuccess)
        return FP8_ERR_LAUNCH;
    if (cudaLaunchKernelEx(&cfg, k_few_gemm<2, NB>, tmW2, tmA, tmW2, f) != cudaSuccess) return FP8_ERR_LAUNCH;
    const unsigned tiles2 = (unsigned)((f.N + 255) / 256);
    cfg.gridDim = token_rows(NB) ? dim3(4 * tiles2, (unsigned)((f.T + 31) / 32), 1)
                                 : dim3(tiles2, (unsigned)((f.T + OUT_TOKENS - 1) / OUT_TOKENS), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, token_rows(NB) ? k_few_out_rows : k_few_out, f, (uint32_t)ctas) == cudaSuccess
               ? FP8_OK
               : FP8_ERR_LAUNCH;
}

}  // namespace

int64_t moe_mlp_few_workspace_bytes(int64_t T, int k, int G, int64_t K, int64_t I, int64_t N)
{
    return few_layout(nullptr, nullptr, T, k, G, K, I, N);
}

int launch_moe_mlp_few(const void* x, int in_dtype, int64_t T, int64_t K, int64_t ldx, const int32_t* topk,
                       const float* weights, int k, int G, const uint8_t* W13, const float* s13,
                       const uint8_t* W2, const float* s2, int64_t I, int64_t N, void* out, int out_dtype,
                       int64_t ldo, void* workspace, int mode, cudaStream_t st, int withhold)
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
    f.withhold = withhold;
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
    if (f.Tp <= MAX_COLUMN_TOKENS) return launch_few_gemms<32>(f, tmW13, tmW2, tmX, tmA, ctas, st);
    return launch_few_gemms<128>(f, tmW13, tmW2, tmX, tmA, ctas, st);
}

int read_and_clear_few_status() { return read_and_clear_module_status(); }

}  // namespace fp8fg
