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

#include <cstdint>
#include <mutex>

#include "fp8fg_device.cuh"
#include "fp8fg_host.h"
#include "fp8fg_quant.cuh"

namespace fp8fg {

namespace {

// 1 / (1 + exp(-g)).  exp(-g) = inf (g < -88.7) gives 0, whose products
// with finite values are 0: the limit.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + expf(-g)); }

// Rows in use: all M, or the device-side count clamped to [0, M].
__device__ __forceinline__ int64_t live_rows(const int32_t* n_rows, int64_t M)
{
    if (!n_rows) return M;
    const int64_t n = __ldg(n_rows);
    return n < 0 ? 0 : (n < M ? n : M);
}

__device__ __forceinline__ float halfwarp_max(float a)
{
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
}

__device__ __forceinline__ float warp_max(float a)
{
    return halfwarp_max(fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16)));
}

// ------------------------------------------------------------ forward

constexpr int kFwdRowsPerHalfWarp = 4;
constexpr int kFwdRowsPerCta = 16 * kFwdRowsPerHalfWarp;   // 64

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv)
{
    return make_uint2(encode4(v[0], v[1], v[2], v[3], inv), encode4(v[4], v[5], v[6], v[7], inv));
}

// CTA = 256 threads = 16 half-warps; a half-warp owns the 128 gate and the 128
// up channels of one block of one row at a time (16 lanes x 8 + 8 elements),
// so each of the three groups (g, u, a) reduces over 16 lanes.  A thread has
// the loads of 4 rows (128 B of BF16) in flight before it uses any.
// Grid (1-D): channel block fastest, then 64-row blocks, so adjacent CTAs read
// adjacent segments of the same rows.
template <typename Tin, bool KEEP>
__global__ void __launch_bounds__(256) k_swiglu_quant(
    const Tin* __restrict__ h, int64_t M, int64_t I, int64_t ldh, uint8_t* __restrict__ qa,
    int64_t ldqa, float* __restrict__ sa, uint8_t* __restrict__ qh, int64_t ldqh,
    float* __restrict__ sh, const int32_t* __restrict__ n_rows, int mode)
{
    const int hw = threadIdx.x >> 4;
    const int l = threadIdx.x & 15;
    const int64_t ncb = I / 128;
    const int64_t cb = blockIdx.x % ncb;
    const int64_t m0 = (int64_t)(blockIdx.x / ncb) * kFwdRowsPerCta;
    const int64_t rows = live_rows(n_rows, M);
    if (m0 >= rows) return;
    const int64_t col = cb * 128 + l * 8;

    Chunk8<Tin> cg[kFwdRowsPerHalfWarp], cu[kFwdRowsPerHalfWarp];
#pragma unroll
    for (int i = 0; i < kFwdRowsPerHalfWarp; ++i) {
        const int64_t m = m0 + i * 16 + hw;
        if (m < rows) {
            cg[i].load(h + m * ldh + col);
            cu[i].load(h + m * ldh + I + col);
        } else {
            cg[i].zero();
            cu[i].zero();
        }
    }
#pragma unroll
    for (int i = 0; i < kFwdRowsPerHalfWarp; ++i) {
        const int64_t m = m0 + i * 16 + hw;
        const bool live = m < rows;
        float g[8], u[8], a[8];
        cg[i].get(g);
        cu[i].get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = g[j] * sigmoid(g[j]) * u[j];
        const GroupScale ga = group_scale(halfwarp_max(absmax8(a)), mode);
        if (live) {
            *reinterpret_cast<uint2*>(qa + m * ldqa + col) = encode8(a, ga.inv);
            if (l == 0) sa[cb * M + m] = ga.s;
        }
        if (KEEP) {
            const GroupScale gg = group_scale(halfwarp_max(absmax8(g)), mode);
            const GroupScale gu = group_scale(halfwarp_max(absmax8(u)), mode);
            if (live) {
                *reinterpret_cast<uint2*>(qh + m * ldqh + col) = encode8(g, gg.inv);
                *reinterpret_cast<uint2*>(qh + m * ldqh + I + col) = encode8(u, gu.inv);
                if (l == 0) {
                    sh[cb * M + m] = gg.s;
                    sh[(ncb + cb) * M + m] = gu.s;
                }
            }
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
    int64_t M, I, ldqh, ldda, lddh, ldqdh, ldqdhT, ldqaT;
    int mode;
};

constexpr int kBwdThreads = 512;
constexpr int kBwdWarps = kBwdThreads / 32;     // 16
constexpr int kBwdTok = 128 / kBwdWarps;        // 8 tokens per warp

struct __align__(16) BwdShared {
    uint8_t outT[3][128 * 128];                 // transposed codes of dG, dU, a
    float part[3][kBwdWarps][128];              // per-warp max-abs of each channel
    float inv[3][128];                          // per-channel encode factors
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename Tda>
__device__ __forceinline__ void load4(const Tda* p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[4])
{
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
}
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&v)[4])
{
    const float4 w = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

// CTA = 512 threads per tile of 128 tokens x 128 channels of I: warp w owns
// tokens 8w .. 8w+7, lane l channels 4l .. 4l+3, so a warp holds whole 1x128
// groups (max-abs by shuffles) and the 128x1 groups combine the warps' maxima
// through shared memory.  dG, dU and a stay in FP32 registers from the one
// computation to the encodes.  Transposed codes go through shared memory (the
// 8-byte pieces of a channel's row XOR-swizzled by the channel's lane, two
// wavefronts per store) and leave as whole 128-byte rows.
// Tokens at or beyond the rows in use count as zero in the 128x1 groups.
template <typename Tda>
__global__ void __launch_bounds__(kBwdThreads, 1) k_swiglu_bwd(const BwdParams p)
{
    extern __shared__ __align__(16) uint8_t bwd_raw[];
    BwdShared& s = *reinterpret_cast<BwdShared*>(bwd_raw);
    const int w = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t ncb = p.I / 128;
    const int64_t cb = blockIdx.x % ncb;
    const int64_t t0 = (int64_t)(blockIdx.x / ncb) * 128;
    const int64_t rows = live_rows(p.n_rows, p.M);
    if (t0 >= rows) return;
    const int64_t col = cb * 128 + 4 * lane;
    const Tda* da = static_cast<const Tda*>(p.da);

    float v[3][kBwdTok][4];       // dG, dU, a
#pragma unroll
    for (int i = 0; i < kBwdTok; ++i) {
        const int64_t t = t0 + w * kBwdTok + i;
        float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < rows) {
            const uint32_t qg = __ldg(reinterpret_cast<const uint32_t*>(p.qh + t * p.ldqh + col));
            const uint32_t qu = __ldg(reinterpret_cast<const uint32_t*>(p.qh + t * p.ldqh + p.I + col));
            const float sg = __ldg(p.sh + cb * p.M + t), su = __ldg(p.sh + (ncb + cb) * p.M + t);
            load4<Tda>(da + t * p.ldda + col, d);
            decode4_e4m3(qg, g);
            decode4_e4m3(qu, u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] *= sg;
                u[k] *= su;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float sig = sigmoid(g[k]);
            const float silu = g[k] * sig;
            v[0][i][k] = d[k] * u[k] * (sig * (1.0f + g[k] * (1.0f - sig)));
            v[1][i][k] = d[k] * silu;
            v[2][i][k] = silu * u[k];
        }
    }

#pragma unroll
    for (int i = 0; i < kBwdTok; ++i) {
        const int64_t t = t0 + w * kBwdTok + i;
        if (t >= rows) break;                                     // warp-uniform
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t c = x * p.I + col;
            const float (&r)[4] = v[x][i];
            if (p.dh)
                *reinterpret_cast<uint2*>(p.dh + t * p.lddh + c) =
                    make_uint2(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]));
            if (p.qdh) {
                const float m = fmaxf(fmaxf(fabsf(r[0]), fabsf(r[1])), fmaxf(fabsf(r[2]), fabsf(r[3])));
                const GroupScale gs = group_scale(warp_max(m), p.mode);
                *reinterpret_cast<uint32_t*>(p.qdh + t * p.ldqdh + c) = encode4(r[0], r[1], r[2], r[3], gs.inv);
                if (lane == 0) p.sdh[(x * ncb + cb) * p.M + t] = gs.s;
            }
        }
    }
    if (!p.qdhT && !p.qaT) return;

    const bool want[3] = {p.qdhT != nullptr, p.qdhT != nullptr, p.qaT != nullptr};
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (!want[x]) continue;
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kBwdTok; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = fmaxf(a[k], fabsf(v[x][i][k]));
        *reinterpret_cast<float4*>(&s.part[x][w][4 * lane]) = make_float4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    const int64_t tb = t0 / 128;
    if (threadIdx.x < 384) {
        const int x = threadIdx.x >> 7, c = threadIdx.x & 127;
        if (want[x]) {
            float a = s.part[x][0][c];
#pragma unroll
            for (int k = 1; k < kBwdWarps; ++k) a = fmaxf(a, s.part[x][k][c]);
            const GroupScale gs = group_scale(a, p.mode);
            s.inv[x][c] = gs.inv;
            if (x < 2)
                p.sdhT[tb * 2 * p.I + x * p.I + cb * 128 + c] = gs.s;
            else
                p.saT[tb * p.I + cb * 128 + c] = gs.s;
        }
    }
    __syncthreads();
    const int half = (w & 1) ^ ((lane >> 3) & 1);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (!want[x]) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float inv = s.inv[x][4 * lane + k];
            const uint2 o = make_uint2(encode4(v[x][0][k], v[x][1][k], v[x][2][k], v[x][3][k], inv),
                                       encode4(v[x][4][k], v[x][5][k], v[x][6][k], v[x][7][k], inv));
            const int c = 4 * lane + k;
            *reinterpret_cast<uint2*>(&s.outT[x][c * 128 + (((w >> 1) ^ (lane & 7)) * 16) + half * 8]) = o;
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (!want[x]) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int id = threadIdx.x + kBwdThreads * i;
            const int c = id >> 3, chunk = id & 7;
            const int wl = c >> 2;                                // lane that wrote channel c
            uint4 q = *reinterpret_cast<const uint4*>(&s.outT[x][c * 128 + ((chunk ^ (wl & 7)) * 16)]);
            if ((wl >> 3) & 1) q = make_uint4(q.z, q.w, q.x, q.y);
            uint8_t* dst = x < 2 ? p.qdhT + (x * p.I + cb * 128 + c) * p.ldqdhT
                                 : p.qaT + (cb * 128 + c) * p.ldqaT;
            *reinterpret_cast<uint4*>(dst + t0 + chunk * 16) = q;
        }
    }
}

// Once per kernel and device: opt into its dynamic shared memory.
template <auto kernel>
cudaError_t allow_smem(int bytes)
{
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (ready[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    ready[dev] = e == cudaSuccess;
    return e;
}

template <typename Tin>
cudaError_t fwd(const void* h, int64_t M, int64_t I, int64_t ldh, uint8_t* qa, int64_t ldqa, float* sa,
                uint8_t* qh, int64_t ldqh, float* sh, const int32_t* n_rows, int mode, cudaStream_t st)
{
    const unsigned grid = (unsigned)((M + kFwdRowsPerCta - 1) / kFwdRowsPerCta * (I / 128));
    const Tin* x = static_cast<const Tin*>(h);
    if (qh)
        k_swiglu_quant<Tin, true><<<grid, 256, 0, st>>>(x, M, I, ldh, qa, ldqa, sa, qh, ldqh, sh, n_rows, mode);
    else
        k_swiglu_quant<Tin, false><<<grid, 256, 0, st>>>(x, M, I, ldh, qa, ldqa, sa, qh, ldqh, sh, n_rows, mode);
    return cudaGetLastError();
}

template <typename Tda>
cudaError_t bwd(const BwdParams& p, cudaStream_t st)
{
    static constexpr int kBytes = (int)sizeof(BwdShared);
    const cudaError_t e = allow_smem<k_swiglu_bwd<Tda>>(kBytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((p.M + 127) / 128 * (p.I / 128));
    k_swiglu_bwd<Tda><<<grid, kBwdThreads, kBytes, st>>>(p);
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
                              const int32_t* n_rows, int mode, cudaStream_t st)
{
    BwdParams p;
    p.qh = qh;
    p.sh = sh;
    p.da = da;
    p.dh = static_cast<__nv_bfloat16*>(dh);
    p.qdh = qdh;
    p.sdh = sdh;
    p.qdhT = qdhT;
    p.sdhT = sdhT;
    p.qaT = qaT;
    p.saT = saT;
    p.n_rows = n_rows;
    p.M = M;
    p.I = I;
    p.ldqh = ldqh;
    p.ldda = ldda;
    p.lddh = lddh;
    p.ldqdh = ldqdh;
    p.ldqdhT = ldqdhT;
    p.ldqaT = ldqaT;
    p.mode = mode;
    return in_dtype == FP8_IN_BF16 ? bwd<__nv_bfloat16>(p, st) : bwd<float>(p, st);
}

}  // namespace fp8fg
