// swiglu.cu -- the gated activation between the two GEMMs of an MLP, fused
// with the FP8 quantizers on both sides of it (sm_100a).
//
//   forward   h = [g | u] (the first GEMM's output) -> a = silu(g) * u,
//             quantized 1x128 (the second GEMM's A operand), and h itself
//             quantized 1x128: the 8-bit checkpoint kept for backward
//   backward  checkpoint and dA -> dG = dA * u * s * (1 + g * (1 - s)),
//             dU = dA * silu(g), s = sigmoid(g), quantized 1x128 (the Dgrad
//             GEMM's operand) and 128x1 (the Wgrad GEMM's), and a recomputed
//             and quantized 128x1 (the other Wgrad's operand)
//
// The recipe keeps the SwiGLU's inputs in FP8 with the fine-grained grouping
// and recomputes its output in the backward pass ("5 Ways You can get More
// Deepseek While Spending Less": FP8 tiles cached for backward;
// gnrental.net post: activations stored in FP8 for backward).  All
// arithmetic is FP32; the only roundings to fewer bits are the E4M3 codes and
// the optional BF16 gradient, each once, from the FP32 value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "fp8fg_device.cuh"
#include "fp8fg_host.h"
#include "fp8fg_quant.cuh"
#include "fp8fg_swiglu.cuh"

namespace fp8fg {

namespace {

// Rows in use: all M, or the device-side count clamped to [0, M].
__device__ __forceinline__ int64_t live_rows(const int32_t* n_rows, int64_t M)
{
    if (!n_rows) return M;
    const int64_t n = __ldg(n_rows);
    return n < 0 ? 0 : (n < M ? n : M);
}

// max(|a|, |b|, |c|, |d|)
__device__ __forceinline__ float absmax4(float a, float b, float c, float d)
{
    return fmaxf(absmax3(a, b, c), fabsf(d));
}

// Four adjacent elements of a row, as raw bits until they are needed.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ void load_shared(const void* p) { r = *static_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(F2& a, F2& b) const
    {
        a = f2(bf16_lo(r.x), bf16_hi(r.x));
        b = f2(bf16_lo(r.y), bf16_hi(r.y));
    }
};
template <>
struct Quad<float> {
    uint4 r;
    __device__ __forceinline__ void load_shared(const void* p) { r = *static_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(F2& a, F2& b) const
    {
        a = f2(__uint_as_float(r.x), __uint_as_float(r.y));
        b = f2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
};

// Four scaled values -> four E4M3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ uint32_t scale_cvt4(F2 a, F2 b, float inv)
{
    const F2 s = f2(inv, inv), x = a * s, y = b * s;
    return cvt4(lo(x), hi(x), lo(y), hi(y));
}

__device__ __forceinline__ uint32_t pack_bf16(F2 v)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo(v), hi(v));
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------ forward

// Threads of a CTA, rows per lane, and CTAs per SM (which caps the registers at 80; with a checkpoint 8 bytes
// a thread spill).  BF16: 4096 x 9216 takes 46.4 us, 135168 x 2048 311.  Of 1 to 4 rows and 64 to 256
// threads these ran fastest over the range of sizes, at 45.3 and 305 us before the sigmoid was as exact as it is:
// 256 threads 46.8 and 315; 3 rows and 5 CTAs 45.5 and 300, but 3.8 us instead of 3.3 for
// 1000 x 2048; others 47 to 54 and 315 to 358.  FP32 rows hold twice the registers: 16384 x 2048 takes
// 58 us with one row, 69 with two, whose loads spill, 58 with two in 4 CTAs.
constexpr int kFwdThreads = 128;
constexpr int kFwdCtasPerSm = 6;
template <typename T>
constexpr int kFwdSteps = sizeof(T) == 2 ? 2 : 1;
template <typename T>
constexpr int kFwdRowsPerCta = kFwdThreads / 8 * kFwdSteps<T>;      // 8 lanes a row

// Lane l of a row's 8 lanes owns 16 of a group's 128 channels, in 16-byte pieces 128 bytes
// apart (so that the 8 lanes of a row read 128 contiguous bytes at a time): BF16 2 pieces of 8
// channels, FP32 4 of 4.
template <typename T>
struct Sixteen;
template <>
struct Sixteen<__nv_bfloat16> {
    static constexpr int kPieces = 2, kPer = 8;
    uint4 r[2];
    __device__ __forceinline__ void get(F2 (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = f2(bf16_lo(r[i].x), bf16_hi(r[i].x));
            v[4 * i + 1] = f2(bf16_lo(r[i].y), bf16_hi(r[i].y));
            v[4 * i + 2] = f2(bf16_lo(r[i].z), bf16_hi(r[i].z));
            v[4 * i + 3] = f2(bf16_lo(r[i].w), bf16_hi(r[i].w));
        }
    }
    static __device__ __forceinline__ void store(uint8_t* dst, const uint32_t (&c)[4])   // dst: channel 0 + 8 * lane
    {
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(dst + 64) = make_uint2(c[2], c[3]);
    }
    static __device__ __forceinline__ void load_codes(const uint8_t* src, uint32_t (&c)[4])
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                         : "=r"(c[2 * i]), "=r"(c[2 * i + 1])
                         : "l"(src + 64 * i));
    }
    static __device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const F2 (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(dst + 64 * i) =
                make_uint4(pack_bf16(v[4 * i]), pack_bf16(v[4 * i + 1]), pack_bf16(v[4 * i + 2]), pack_bf16(v[4 * i + 3]));
    }
};
template <>
struct Sixteen<float> {
    static constexpr int kPieces = 4, kPer = 4;
    uint4 r[4];
    __device__ __forceinline__ void get(F2 (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = f2(__uint_as_float(r[i].x), __uint_as_float(r[i].y));
            v[2 * i + 1] = f2(__uint_as_float(r[i].z), __uint_as_float(r[i].w));
        }
    }
    static __device__ __forceinline__ void store(uint8_t* dst, const uint32_t (&c)[4])   // dst: channel 0 + 4 * lane
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(dst + 32 * i) = c[i];
    }
    static __device__ __forceinline__ void load_codes(const uint8_t* src, uint32_t (&c)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(c[i]) : "l"(src + 32 * i));
    }
    static __device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const F2 (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint2*>(dst + 32 * i) = make_uint2(pack_bf16(v[2 * i]), pack_bf16(v[2 * i + 1]));
    }
};

__device__ __forceinline__ float absmax16(const F2 (&v)[8])
{
    float m = fmaxf(fabsf(lo(v[0])), fabsf(hi(v[0])));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = absmax3(m, lo(v[i]), hi(v[i]));
    return m;
}

// Max over the 8 lanes of a row.
__device__ __forceinline__ float row_max(float a)
{
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
}

__device__ __forceinline__ void encode16(const F2 (&v)[8], float inv, uint32_t (&c)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = scale_cvt4(v[2 * i], v[2 * i + 1], inv);
}

// CTA = 4 warps; 8 lanes own the 128 gate and the 128 up channels of one
// channel block of a row (16 + 16 a lane), so a warp works on 4 rows at once and each
// of a row's three groups (a, g, u) reduces its max-abs in three shuffles.  Lane 0 of
// the row then derives the scale of a, lane 1 that of g, lane 2 that of u, in the same
// instructions: the two correctly rounded divisions of a scale, three times over in
// all lanes, would cost more than the SwiGLU itself.
// Grid (1-D): channel block fastest, then row blocks, so adjacent CTAs read adjacent
// segments of the same rows.
template <typename Tin, bool KEEP>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtasPerSm) k_swiglu_quant(
    const Tin* __restrict__ h, int M, int I, int ldh, uint8_t* __restrict__ qa, int ldqa,
    float* __restrict__ sa, uint8_t* __restrict__ qh, int ldqh, float* __restrict__ sh,
    const int32_t* __restrict__ n_rows, int mode)
{
    using V = Sixteen<Tin>;
    const int l = threadIdx.x & 7;
    const uint32_t ncb = (uint32_t)I / 128, rb = blockIdx.x / ncb, cb = blockIdx.x - rb * ncb;
    const uint32_t m0 = rb * kFwdRowsPerCta<Tin> + (threadIdx.x >> 3);    // may pass 2^31 by less than a CTA's rows
    const uint32_t rows = (uint32_t)live_rows(n_rows, M);
    const int col = (int)cb * 128 + l * V::kPer;

    V rg[kFwdSteps<Tin>], ru[kFwdSteps<Tin>];
#pragma unroll
    for (int i = 0; i < kFwdSteps<Tin>; ++i) {
        const uint32_t m = m0 + kFwdThreads / 8 * i;
        const Tin* src = h + (int64_t)(int)(m < rows ? m : 0) * ldh + col;
#pragma unroll
        for (int j = 0; j < V::kPieces; ++j) {
            rg[i].r[j] = ru[i].r[j] = make_uint4(0, 0, 0, 0);
            if (m < rows) {
                rg[i].r[j] = ld_stream16(src + 8 * V::kPer * j);
                ru[i].r[j] = ld_stream16(src + I + 8 * V::kPer * j);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kFwdSteps<Tin>; ++i) {
        const uint32_t m = m0 + kFwdThreads / 8 * i;
        const bool live = m < rows;
        F2 g[8], u[8], a[8];
        rg[i].get(g);
        ru[i].get(u);
        const float gmax = absmax16(g);
        if (__any_sync(0xffffffffu, gmax > kNearGates)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = silu2<true>(g[j]) * u[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = silu2<false>(g[j]) * u[j];
        }
        float mine = row_max(absmax16(a));
        if (KEEP) {
            const float mg = row_max(gmax), mu = row_max(absmax16(u));
            mine = l == 1 ? mg : (l == 2 ? mu : mine);
        }
        const GroupScale gs = group_scale(mine, mode);
        if (live && l < (KEEP ? 3 : 1))
            (l == 0 ? sa + (int64_t)(int)cb * M : sh + (int64_t)(int)(l == 1 ? cb : ncb + cb) * M)[m] = gs.s;
        uint32_t c[4];
        encode16(a, __shfl_sync(0xffffffffu, gs.inv, 0, 8), c);
        if (live) V::store(qa + (int64_t)(int)m * ldqa + col, c);
        if (KEEP) {
            const float ig = __shfl_sync(0xffffffffu, gs.inv, 1, 8), iu = __shfl_sync(0xffffffffu, gs.inv, 2, 8);
            uint8_t* dst = qh + (int64_t)(int)m * ldqh + col;
            encode16(g, ig, c);
            if (live) V::store(dst, c);
            encode16(u, iu, c);
            if (live) V::store(dst + I, c);
        }
    }
}

// ------------------------------------------------------------ backward

struct BwdParams {
    const uint8_t* qh;
    const float* sh;
    const void* da;
    __nv_bfloat16* dh;      // any of the four outputs may be null
    uint8_t* qdh;
    float* sdh;
    uint8_t* qdhT;
    float* sdhT;
    uint8_t* qaT;
    float* saT;
    const int32_t* n_rows;
    int M, I, ldqh, ldda, lddh, ldqdh, ldqdhT, ldqaT;
    int mode;
    uint64_t timeout_ns;
};

constexpr int kBwdThreads = 512;
constexpr int kBwdWarps = kBwdThreads / 32;     // 16
constexpr int kBwdTok = 128 / kBwdWarps;        // 8 tokens per warp

// dG, dU and a of a pair of channels (FAR as in silu2).
template <bool FAR>
__device__ __forceinline__ void gradients(F2 g, F2 u, F2 da, F2& dg, F2& du, F2& a)
{
    const F2 one = f2(1.0f, 1.0f);
    F2 r, f;
    if (FAR)
        sigmoid2_far(g, r, f);
    else
        r = sigmoid2(g);
    const F2 rest = fma2(FAR ? r * f : r, f2(-1.0f, -1.0f), one);      // 1 - s
    F2 silu = g * r, slope = r * fma2(g, rest, one);
    if (FAR) {
        silu = silu * f;
        slope = slope * f;
    }
    dg = da * u * slope;
    du = da * silu;
    a = silu * u;
}

// Whether gates of checkpoints with these scales may lie beyond kNearGates (a code is at most 448).
__device__ __forceinline__ bool far_gates(float scale) { return !(fabsf(scale) <= kNearGates / 448.0f); }

// Backward without transposed outputs: no group spans rows, so the work is split as the forward's (8
// lanes own a row's channel block).  16384 x 2048, codes of dH alone: 37.9 us (FP32 dA 43.3), 46.6
// (60.5) by the tiles of k_swiglu_bwd; 128 x 512 3.4 and 5.1.  With 7 CTAs per SM 38.3 (47.8), with 6 39.0 (50.4),
// although 8 spill 48 bytes a thread of BF16; of other shapes, 10 CTAs of one row and 4 of three were 10 and 15 % slower.
constexpr int kBwdRowsCtasPerSm = 8;
template <typename Tda>
__global__ void __launch_bounds__(kFwdThreads, kBwdRowsCtasPerSm) k_swiglu_bwd_rows(const BwdParams p)
{
    using V = Sixteen<Tda>;
    const int l = threadIdx.x & 7;
    const uint32_t ncb = (uint32_t)p.I / 128, rb = blockIdx.x / ncb, cb = blockIdx.x - rb * ncb;
    const uint32_t m0 = rb * kFwdRowsPerCta<Tda> + (threadIdx.x >> 3);
    const uint32_t rows = (uint32_t)live_rows(p.n_rows, p.M);
    const int col = (int)cb * 128 + l * V::kPer;

    V rd[kFwdSteps<Tda>];
    uint32_t cg[kFwdSteps<Tda>][4], cu[kFwdSteps<Tda>][4];
    float sg[kFwdSteps<Tda>], su[kFwdSteps<Tda>];
#pragma unroll
    for (int i = 0; i < kFwdSteps<Tda>; ++i) {
        const uint32_t m = m0 + kFwdThreads / 8 * i;
        const int64_t r = (int64_t)(int)(m < rows ? m : 0);
        sg[i] = su[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) cg[i][j] = cu[i][j] = 0;
#pragma unroll
        for (int j = 0; j < V::kPieces; ++j) rd[i].r[j] = make_uint4(0, 0, 0, 0);
        if (m < rows) {
            V::load_codes(p.qh + r * p.ldqh + col, cg[i]);
            V::load_codes(p.qh + r * p.ldqh + col + p.I, cu[i]);
            const Tda* da = static_cast<const Tda*>(p.da) + r * p.ldda + col;
#pragma unroll
            for (int j = 0; j < V::kPieces; ++j) rd[i].r[j] = ld_stream16(da + 8 * V::kPer * j);
            sg[i] = __ldg(p.sh + (int64_t)(int)cb * p.M + r);
            su[i] = __ldg(p.sh + (int64_t)(int)(ncb + cb) * p.M + r);
        }
    }
#pragma unroll
    for (int i = 0; i < kFwdSteps<Tda>; ++i) {
        const uint32_t m = m0 + kFwdThreads / 8 * i;
        const bool live = m < rows;
        F2 da[8], dg[8], du[8];
        rd[i].get(da);
        const F2 s0 = f2(sg[i], sg[i]), s1 = f2(su[i], su[i]);
        auto all = [&](auto far) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float gf[4], uf[4];
                decode4_e4m3(cg[i][j], gf);
                decode4_e4m3(cu[i][j], uf);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    F2 a;
                    gradients<decltype(far)::value>(f2(gf[2 * k], gf[2 * k + 1]) * s0, f2(uf[2 * k], uf[2 * k + 1]) * s1,
                                                    da[2 * j + k], dg[2 * j + k], du[2 * j + k], a);
                }
            }
        };
        if (__any_sync(0xffffffffu, far_gates(sg[i])))
            all(std::true_type{});
        else
            all(std::false_type{});
        if (p.dh && live) {
            __nv_bfloat16* dst = p.dh + (int64_t)(int)m * p.lddh + col;
            V::store_bf16(dst, dg);
            V::store_bf16(dst + p.I, du);
        }
        if (!p.qdh) continue;
        const float mg = row_max(absmax16(dg)), mu = row_max(absmax16(du));
        const GroupScale gs = group_scale(l == 1 ? mu : mg, p.mode);
        if (live && l < 2) p.sdh[(int64_t)(int)(l ? ncb + cb : cb) * p.M + m] = gs.s;
        uint8_t* dst = p.qdh + (int64_t)(int)m * p.ldqdh + col;
        uint32_t c[4];
        encode16(dg, __shfl_sync(0xffffffffu, gs.inv, 0, 8), c);
        if (live) V::store(dst, c);
        encode16(du, __shfl_sync(0xffffffffu, gs.inv, 1, 8), c);
        if (live) V::store(dst + p.I, c);
    }
}

struct Tile {
    int32_t tb, cb;         // block of 128 tokens, block of 128 channels
};

// Inputs of one tile as they lie in shared memory.
template <typename Tda>
struct __align__(128) BwdStage {
    uint8_t g[128 * 128];                       // checkpoint codes of the gate and the up half
    uint8_t u[128 * 128];
    Tda da[128 * 128];
    float scale[2][128];                        // the checkpoint's, of both halves
};

// FP32 gradients leave room for one stage (96 KB) beside the transposed codes, BF16 ones for two.
template <typename Tda>
constexpr int kBwdStages = sizeof(Tda) == 2 ? 2 : 1;

template <typename Tda>
struct __align__(128) BwdShared {
    BwdStage<Tda> stage[kBwdStages<Tda>];
    uint8_t outT[3][128 * 128];                 // transposed codes of dG, dU, a
    float part[3][kBwdWarps][128];              // per-warp max-abs of each channel
    float inv[3 * 128];                         // per-channel encode factors
    float rmax[kBwdWarps][16];                  // a warp's 16 row maxima
    uint64_t full[2];                           // a stage has arrived
    uint64_t bPart, bInv, bOut;                 // all warps: part written, inv written, outT written
    int abort;
};

// 16 bytes global -> shared (its 32-bit address), asynchronously; zeros when `live` is false.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
// This thread's arrival on an mbarrier, once its copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Persistent CTAs of 512 threads over tiles of 128 tokens x 128 channels of I (channel
// block fastest), which arrive by cp.async while the tile before is worked on: into the other of two
// stages, or, with FP32 gradients, into the only one once its values are in registers.  (Three TMA
// boxes instead save a tenth of the instructions, yet took 645 us instead of 534, as the kernel was
// then, for 135168 x 2048.)
// Warp w owns tokens 8w .. 8w+7, lane l channels 4l .. 4l+3, so a warp holds whole 1x128
// groups (one warp reduction each; lane j derives the scale of group j of the warp's 16 once)
// and the 128x1 groups combine the warps' maxima through shared memory.  dG, dU and a stay in
// FP32 registers (96 a thread) from the one computation to both encodes.  Transposed codes go
// through shared memory (the 8-byte pieces of a channel's row XOR-swizzled by the channel's
// lane: two wavefronts per store) and leave as whole 128-byte rows.
// The 16 warps never stop at a common barrier: each of a tile's three hand-overs (part, inv,
// outT) is an mbarrier that a warp arrives on, does work that does not need it, and
// then waits for -- the 1x128 groups get their scales and the rows of the tile before go out
// between part and inv, the 1x128 groups are encoded between inv and outT.  (4096 x 9216 takes
// 73.8 us.  Measured at 70.4, before the sigmoid was as exact as it is: 71.1 with the 1x128 scales behind the
// channels', 75.5 with half of the 1x128 codes before them.  Waits that suspend instead of spinning cost 2 %
// more; the checkpoint's scales loaded into registers a tile ahead, 2 to 20 %, as the compiler lets them be
// waited for.)
// Tokens at or beyond the rows in use count as zero in the 128x1 groups.
// WITHHOLD (self-test): one warp never says that its part of the first tile's maxima is written.
template <typename Tda, bool WITHHOLD = false>
__global__ void __launch_bounds__(kBwdThreads, 1) k_swiglu_bwd(const BwdParams p)
{
    extern __shared__ __align__(128) uint8_t bwd_raw[];
    BwdShared<Tda>& s = *reinterpret_cast<BwdShared<Tda>*>(bwd_raw);
    constexpr int NST = kBwdStages<Tda>;
    const int w = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int32_t ncb = p.I / 128;
    const int rows = (int)live_rows(p.n_rows, p.M);
    const int32_t ntb = (int32_t)(((uint32_t)rows + 127) / 128);
    const bool wantH = p.qdhT != nullptr, wantA = p.qaT != nullptr;      // one of them at least

    if (threadIdx.x == 0) {
        mbar_init(&s.full[0], kBwdThreads);
        mbar_init(&s.full[1], kBwdThreads);
        mbar_init(&s.bPart, kBwdWarps);
        mbar_init(&s.bInv, kBwdWarps);
        mbar_init(&s.bOut, kBwdWarps);
        s.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();

    // A wait that runs out is reported, and what this launch writes from then on is worthless.
    auto wait = [&](uint64_t* bar, int parity) {
        mbar_wait_spin(bar, (uint32_t)parity & 1u, &s.abort, p.timeout_ns);
        __syncwarp();
    };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // A tile into a stage: thread i copies the 16-byte pieces i, i + 512, ... of each array in row
    // order.  Rows behind those in use become zeros.
    constexpr int kPer = 16 / (int)sizeof(Tda), kPerRow = 128 / kPer, kStepD = kBwdThreads / kPerRow;
    const int64_t offQ = (int64_t)(threadIdx.x >> 3) * p.ldqh + (threadIdx.x & 7) * 16;
    const int64_t offD = (int64_t)(threadIdx.x / kPerRow) * p.ldda + threadIdx.x % kPerRow * kPer;
    auto load = [&](Tile tile, int st) {
        const int t0 = tile.tb * 128;
        const uint8_t* q = p.qh + (int64_t)t0 * p.ldqh + tile.cb * 128 + offQ;
        const Tda* da = static_cast<const Tda*>(p.da) + (int64_t)t0 * p.ldda + tile.cb * 128 + offD;
        const uint32_t dst = smem_u32(&s.stage[st]) + threadIdx.x * 16;
        constexpr uint32_t kU = offsetof(BwdStage<Tda>, u), kD = offsetof(BwdStage<Tda>, da), kStep = kBwdThreads * 16;
        if (t0 <= rows - 128) {
            cp16(dst, q);
            cp16(dst + kU, q + p.I);
            q += (int64_t)64 * p.ldqh;
            cp16(dst + kStep, q);
            cp16(dst + kU + kStep, q + p.I);
#pragma unroll
            for (int i = 0; i < 128 / kStepD; ++i, da += (int64_t)kStepD * p.ldda) cp16(dst + kD + i * kStep, da);
        } else {
            for (int i = 0; i < 2; ++i) {
                const int r = (threadIdx.x >> 3) + 64 * i;
                const bool live = t0 < rows - r;
                const uint8_t* src = live ? q + (int64_t)(i * 64) * p.ldqh : p.qh;
                cp16(dst + i * kStep, src, live);
                cp16(dst + kU + i * kStep, src + p.I, live);
            }
            for (int i = 0; i < 128 / kStepD; ++i) {
                const bool live = t0 < rows - (int)(threadIdx.x / kPerRow) - i * kStepD;
                cp16(dst + kD + i * kStep, live ? da + (int64_t)(i * kStepD) * p.ldda : static_cast<const Tda*>(p.da), live);
            }
        }
        if (threadIdx.x < 256) {
            const int t = t0 + (threadIdx.x & 127), half = threadIdx.x >> 7;
            const bool live = t < rows;
            cp4(smem_u32(&s.stage[st].scale[0][0]) + threadIdx.x * 4,
                p.sh + (int64_t)(half * ncb + tile.cb) * p.M + (live ? t : 0), live);
        }
        cp_arrive(&s.full[st]);
    };
    // whole 128-byte rows of a tile's transposed codes: 8 threads a row, 64 channels a pass
    auto store_rows = [&](Tile tile) {
        const int t0 = tile.tb * 128;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (!(x < 2 ? wantH : wantA)) continue;
            const int ld = x < 2 ? p.ldqdhT : p.ldqaT;
            const int row = (x < 2 ? x * p.I : 0) + tile.cb * 128 + (int)(threadIdx.x >> 3);
            uint8_t* dst = (x < 2 ? p.qdhT : p.qaT) + (int64_t)row * ld + t0 + (threadIdx.x & 7) * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i, dst += (int64_t)64 * ld) {
                const int c = (threadIdx.x >> 3) + 64 * i;
                const int wl = c >> 2;                                // lane that wrote channel c
                uint4 q = *reinterpret_cast<const uint4*>(&s.outT[x][c * 128 + (((threadIdx.x & 7) ^ (wl & 7)) * 16)]);
                if (wl & 8) q = make_uint4(q.z, q.w, q.x, q.y);       // its halves swapped
                *reinterpret_cast<uint4*>(dst) = q;
            }
        }
    };

    // tiles in steps of the grid without divisions
    const int32_t step_tb = (int32_t)gridDim.x / ncb, step_cb = (int32_t)gridDim.x % ncb;
    Tile tile{(int32_t)blockIdx.x / ncb, (int32_t)blockIdx.x % ncb}, prev = tile, next = tile;
    if (tile.tb < ntb) load(tile, 0);
    int it = 0;
    for (; tile.tb < ntb; ++it, prev = tile, tile = next) {
        const int st = NST == 2 ? it & 1 : 0;
        next.tb += step_tb;
        next.cb += step_cb;
        if (next.cb >= ncb) {
            next.cb -= ncb;
            ++next.tb;
        }
        // two stages: all warps have read the other one, for this one has waited for the
        // previous tile's bPart
        if (NST == 2 && next.tb < ntb) load(next, st ^ 1);
        wait(&s.full[st], NST == 2 ? it >> 1 : it);

        // The tile's work of a warp; `far` says whether gates may lie beyond kNearGates (as in silu2), at compile
        // time or, as a bool, at run time.
        auto work = [&](auto far) {
            const int col = tile.cb * 128 + 4 * lane;
            const int tw = tile.tb * 128 + w * kBwdTok;
            const int nr = min((int64_t)rows - tw, (int64_t)kBwdTok);             // this warp's rows in use, may be <= 0
            F2 v[3][kBwdTok][2];      // dG, dU, a
            {
                const BwdStage<Tda>& d = s.stage[st];
                float sc[2][kBwdTok];
#pragma unroll
                for (int i = 0; i < 2 * kBwdTok; i += 4)
                    *reinterpret_cast<float4*>(&sc[0][0] + i) =
                        *reinterpret_cast<const float4*>(&d.scale[i / kBwdTok][w * kBwdTok + i % kBwdTok]);
                auto values = [&](auto far) {
#pragma unroll
                    for (int i = 0; i < kBwdTok; ++i) {
                        const int r = w * kBwdTok + i;
                        const float s0 = sc[0][i], s1 = sc[1][i];
                        float gf[4], uf[4];
                        decode4_e4m3(*reinterpret_cast<const uint32_t*>(d.g + r * 128 + 4 * lane), gf);
                        decode4_e4m3(*reinterpret_cast<const uint32_t*>(d.u + r * 128 + 4 * lane), uf);
                        Quad<Tda> q;
                        q.load_shared(d.da + r * 128 + 4 * lane);
                        F2 da[2];
                        q.get(da[0], da[1]);
                        const F2 sg = f2(s0, s0), su = f2(s1, s1);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            gradients<decltype(far)::value>(f2(gf[2 * k], gf[2 * k + 1]) * sg,
                                                            f2(uf[2 * k], uf[2 * k + 1]) * su, da[k], v[0][i][k], v[1][i][k],
                                                            v[2][i][k]);
                        }
                    }
                };
                if constexpr (!std::is_same_v<decltype(far), bool>)
                    values(far);
                else if (far)
                    values(std::true_type{});
                else
                    values(std::false_type{});
            }

            // per-warp column maxima for the 128x1 groups
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (!(x < 2 ? wantH : wantA)) continue;
                float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kBwdTok; i += 2)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[2 * k] = absmax3(a[2 * k], lo(v[x][i][k]), lo(v[x][i + 1][k]));
                        a[2 * k + 1] = absmax3(a[2 * k + 1], hi(v[x][i][k]), hi(v[x][i + 1][k]));
                    }
                *reinterpret_cast<float4*>(&s.part[x][w][4 * lane]) = make_float4(a[0], a[1], a[2], a[3]);
            }
            if (!WITHHOLD || it > 0 || w != 3) arrive(&s.bPart);
            // maxima and scales of the 1x128 groups (lane j: group j of the warp's 16)
            GroupScale gs{};
            if (p.qdh) {
#pragma unroll
                for (int i = 0; i < kBwdTok; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const F2 (&r)[2] = v[x][i];
                        const float m = warp_absmax(absmax4(lo(r[0]), hi(r[0]), lo(r[1]), hi(r[1])));
                        if (lane == 0) s.rmax[w][8 * x + i] = m;
                    }
                __syncwarp();
                gs = group_scale(s.rmax[w][lane & 15], p.mode);
                __syncwarp();
            }
            if (it > 0) {
                wait(&s.bOut, it - 1);
                store_rows(prev);
            }
            wait(&s.bPart, it);
            if (NST == 1 && next.tb < ntb) load(next, 0);
            // channel scales; a warp past the 384 channels arrives all the same: bInv also
            // says that every warp has stored the previous tile's rows
            if (threadIdx.x < 384 && (threadIdx.x < 256 ? wantH : wantA)) {
                const int x = threadIdx.x >> 7, c = threadIdx.x & 127;
                float a = s.part[x][0][c];
#pragma unroll
                for (int k = 1; k < kBwdWarps - 1; k += 2) a = absmax3(a, s.part[x][k][c], s.part[x][k + 1][c]);
                const GroupScale gs = group_scale(fmaxf(a, s.part[x][kBwdWarps - 1][c]), p.mode);
                s.inv[threadIdx.x] = gs.inv;
                const int ch = tile.cb * 128 + c;
                if (x < 2)
                    p.sdhT[(int64_t)tile.tb * (2 * p.I) + x * p.I + ch] = gs.s;
                else
                    p.saT[(int64_t)tile.tb * p.I + ch] = gs.s;
            }
            arrive(&s.bInv);

            // 1x128 groups and BF16 rows
            if (p.dh) {
                __nv_bfloat16* dst = p.dh + (int64_t)tw * p.lddh + col;
#pragma unroll
                for (int i = 0; i < kBwdTok; ++i, dst += p.lddh)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (i < nr)
                            *reinterpret_cast<uint2*>(dst + x * p.I) =
                                make_uint2(pack_bf16(v[x][i][0]), pack_bf16(v[x][i][1]));
            }
            if (p.qdh) {
                if (lane < 16 && (lane & 7) < nr)
                    p.sdh[(int64_t)((lane >> 3) * ncb + tile.cb) * p.M + tw + (lane & 7)] = gs.s;
                uint8_t* dst = p.qdh + (int64_t)tw * p.ldqdh + col;
#pragma unroll
                for (int i = 0; i < kBwdTok; ++i, dst += p.ldqdh)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float inv = __shfl_sync(0xffffffffu, gs.inv, 8 * x + i);
                        if (i < nr)
                            *reinterpret_cast<uint32_t*>(dst + x * p.I) = scale_cvt4(v[x][i][0], v[x][i][1], inv);
                    }
            }
            wait(&s.bInv, it);
            const int half = (w & 1) ^ ((lane >> 3) & 1);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (!(x < 2 ? wantH : wantA)) continue;
                const float4 i4 = *reinterpret_cast<const float4*>(&s.inv[x * 128 + 4 * lane]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const F2 inv = k ? f2(i4.z, i4.w) : f2(i4.x, i4.y);
                    F2 e[kBwdTok];
#pragma unroll
                    for (int i = 0; i < kBwdTok; ++i) e[i] = v[x][i][k] * inv;
                    const int c = 4 * lane + 2 * k;
                    uint8_t* dst = &s.outT[x][c * 128 + (((w >> 1) ^ (lane & 7)) * 16) + half * 8];
                    *reinterpret_cast<uint2*>(dst) = make_uint2(cvt4(lo(e[0]), lo(e[1]), lo(e[2]), lo(e[3])),
                                                                cvt4(lo(e[4]), lo(e[5]), lo(e[6]), lo(e[7])));
                    *reinterpret_cast<uint2*>(dst + 128) = make_uint2(cvt4(hi(e[0]), hi(e[1]), hi(e[2]), hi(e[3])),
                                                                      cvt4(hi(e[4]), hi(e[5]), hi(e[6]), hi(e[7])));
                }
            }
            arrive(&s.bOut);
        };
        // The branch around the values alone is the faster one for BF16 gradients (16384 x 2048: 65.5 us; 67.9 around all
        // of the work), and the slower for FP32 ones (90.7 and 86.8).
        const bool far = __any_sync(0xffffffffu, far_gates(s.stage[st].scale[0][w * kBwdTok + lane % kBwdTok]));
        if constexpr (sizeof(Tda) == 2)
            work(far);
        else if (far)
            work(std::true_type{});
        else
            work(std::false_type{});
        // part is written again only behind this tile's bInv, inv only behind the next tile's
        // bPart, which a warp arrives on after the reads of inv above.
    }
    if (it > 0) {
        wait(&s.bOut, it - 1);
        store_rows(prev);
    }
    // after a wait that ran out, no copy may still be on its way when the CTA exits
    if (threadIdx.x == 0 && s.abort)
        for (int st = 0; st < NST; ++st) {
            const int loads = (it - st + NST - 1) / NST;
            if (loads > 0) mbar_wait_drain(&s.full[st], (uint32_t)((loads - 1) & 1), p.timeout_ns);
        }
}

template <typename Tin>
cudaError_t fwd(const void* h, int64_t M, int64_t I, int64_t ldh, uint8_t* qa, int64_t ldqa, float* sa,
                uint8_t* qh, int64_t ldqh, float* sh, const int32_t* n_rows, int mode, cudaStream_t st)
{
    const unsigned grid = (unsigned)((M + kFwdRowsPerCta<Tin> - 1) / kFwdRowsPerCta<Tin> * (I / 128));
    const Tin* x = static_cast<const Tin*>(h);
    if (qh)
        k_swiglu_quant<Tin, true><<<grid, kFwdThreads, 0, st>>>(x, (int)M, (int)I, (int)ldh, qa, (int)ldqa, sa, qh, (int)ldqh, sh,
                                                         n_rows, mode);
    else
        k_swiglu_quant<Tin, false><<<grid, kFwdThreads, 0, st>>>(x, (int)M, (int)I, (int)ldh, qa, (int)ldqa, sa, qh, (int)ldqh, sh,
                                                          n_rows, mode);
    return cudaGetLastError();
}

template <typename Tda, bool WITHHOLD = false>
cudaError_t bwd(const BwdParams& p, cudaStream_t st)
{
    if (!p.qdhT && !p.qaT) {
        const int64_t blocks = ((int64_t)p.M + kFwdRowsPerCta<Tda> - 1) / kFwdRowsPerCta<Tda> * (p.I / 128);
        k_swiglu_bwd_rows<Tda><<<(unsigned)blocks, kFwdThreads, 0, st>>>(p);
        return cudaGetLastError();
    }
    static constexpr int kBytes = (int)sizeof(BwdShared<Tda>);
    const cudaError_t e = allow_smem<k_swiglu_bwd<Tda, WITHHOLD>>(kBytes);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((int64_t)p.M + 127) / 128 * (p.I / 128);
    const int64_t sms = device_sm_count();
    const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
    k_swiglu_bwd<Tda, WITHHOLD><<<grid, kBwdThreads, kBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swiglu_quant(const void* h, int in_dtype, int64_t M, int64_t I, int64_t ldh,
                                uint8_t* qa, int64_t ldqa, float* sa, uint8_t* qh, int64_t ldqh,
                                float* sh, const int32_t* n_rows, int mode, cudaStream_t st)
{
    return in_dtype == FP8_IN_BF16
               ? fwd<__nv_bfloat16>(h, M, I, ldh, qa, ldqa, sa, qh, ldqh, sh, n_rows, mode, st)
               : fwd<float>(h, M, I, ldh, qa, ldqa, sa, qh, ldqh, sh, n_rows, mode, st);
}

cudaError_t launch_swiglu_bwd(const uint8_t* qh, int64_t ldqh, const float* sh, const void* da,
                              int in_dtype, int64_t ldda, int64_t M, int64_t I, void* dh, int64_t lddh,
                              uint8_t* qdh, int64_t ldqdh, float* sdh, uint8_t* qdhT, int64_t ldqdhT,
                              float* sdhT, uint8_t* qaT, int64_t ldqaT, float* saT,
                              const int32_t* n_rows, int mode, cudaStream_t st, bool withhold)
{
    BwdParams p;
    p.qh = qh;
    p.sh = sh;
    p.da = da;
    p.ldqh = (int)ldqh;
    p.ldda = (int)ldda;
    p.dh = static_cast<__nv_bfloat16*>(dh);
    p.qdh = qdh;
    p.sdh = sdh;
    p.qdhT = qdhT;
    p.sdhT = sdhT;
    p.qaT = qaT;
    p.saT = saT;
    p.n_rows = n_rows;
    p.M = (int)M;
    p.I = (int)I;
    p.lddh = (int)lddh;
    p.ldqdh = (int)ldqdh;
    p.ldqdhT = (int)ldqdhT;
    p.ldqaT = (int)ldqaT;
    p.mode = mode;
    p.timeout_ns = wait_timeout_ns();
    if (withhold) return in_dtype == FP8_IN_BF16 ? bwd<__nv_bfloat16, true>(p, st) : bwd<float, true>(p, st);
    return in_dtype == FP8_IN_BF16 ? bwd<__nv_bfloat16>(p, st) : bwd<float>(p, st);
}

int read_and_clear_swiglu_status() { return read_and_clear_module_status(); }

}  // namespace fp8fg
