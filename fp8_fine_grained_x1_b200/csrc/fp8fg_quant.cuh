// fp8fg_quant.cuh -- device pieces every quantizer of libfp8fg shares: the
// group scale, the E4M3 encode and decode of four values, and the 16-byte
// streaming loads of the inputs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8fg_device.cuh"

namespace fp8fg {

namespace {

// ------------------------------------------------------------ group scale

struct GroupScale {
    float s;    // stored scale (dequantisation multiplier)
    float inv;  // factor applied before the E4M3 cast
};

// Scale of a group with max-abs `amax` (amax >= 0, finite).
//   FP32 mode: s = amax/448, inv = 448/amax, both correctly rounded; a zero
//              group gets s = inv = 1; when amax/448 would fall below the
//              smallest normal FP32 the scale saturates at 2^-126.
//   POW2 mode: s = 2^e, e least with amax <= 448*2^e, e >= -126; inv = 2^-e.
__device__ __forceinline__ GroupScale group_scale(float amax, int mode)
{
    GroupScale g;
    if (amax == 0.0f) {
        g.s = 1.0f;
        g.inv = 1.0f;
        return g;
    }
    if (mode == FP8_SCALE_POW2) {
        const uint32_t b = __float_as_uint(amax);
        const int ex = (int)((b >> 23) & 0xFF);
        int e = -126;
        if (ex != 0) {
            // amax = m * 2^(ex-127), m in [1,2).  448 = 1.75 * 2^8, so the
            // least e is ex-127-8 when m <= 1.75 and one more otherwise.
            e = ex - 127 - 8 + (((b & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
            if (e < -126) e = -126;
        }
        g.s = __uint_as_float((uint32_t)(e + 127) << 23);
        g.inv = __uint_as_float((uint32_t)(127 - e) << 23);
        return g;
    }
    if (amax < __uint_as_float(0x04E00000u)) {        // 1.75 * 2^-118
        g.s = __uint_as_float(0x00800000u);            // 2^-126
        g.inv = __uint_as_float(0x7E800000u);          // 2^126
        return g;
    }
    // Both quotients correctly rounded.  Where nothing can under- or overflow they come from the
    // correctly rounded reciprocals r of 448 and of amax: q = fl(x * r), the remainder x - q * y in one FMA,
    // and fl(q + remainder * r), the steps of Markstein's division ("Computation of elementary functions on
    // the IBM RISC System/6000 processor", 1990).  His theorem wants q within one unit in the last place, and q
    // is up to 1.4 off here; that the results are the correctly rounded quotients all the same is shown by
    // exhaustion, over all 2^23 significands (a power of two in amax changes no step).  About half the
    // instructions of two divisions.
    if (__float_as_uint(amax) - 0x0F800000u <= 0x60000000u) {      // 2^-96 <= amax <= 2^96
        constexpr float r448 = 1.0f / 448.0f;
        const float q = amax * r448;
        g.s = fmaf(fmaf(-448.0f, q, amax), r448, q);
        const float r = __frcp_rn(amax), p = 448.0f * r;
        g.inv = fmaf(fmaf(-amax, p, 448.0f), r, p);
        return g;
    }
    g.inv = __fdiv_rn(448.0f, amax);
    g.s = __fdiv_rn(amax, 448.0f);
    return g;
}

// Four scaled values -> four E4M3 codes packed little-endian in a uint32:
// byte i = E4M3(fl32(x_i * inv)), round to nearest even, saturating to
// +-448.  The products are two packed FP32x2 multiplies (each lane rounded
// to nearest like a scalar multiply); each cvt packs two codes, its first
// source going to the upper byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    float a2, b2, c2, d2;
    fmul2(a2, b2, a, b, inv, inv);
    fmul2(c2, d2, c, d, inv, inv);
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a2), "f"(b2), "f"(c2), "f"(d2));
    return r;
}

// ------------------------------------------------------------ vector loads

__device__ __forceinline__ uint4 ld_stream16(const void* p)
{
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight consecutive input elements held as raw bits (16 B of BF16 or 32 B of
// FP32) until they are needed as floats.
template <typename Tin>
struct Chunk8;

template <>
struct Chunk8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = ld_stream16(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
        v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
    }
};

template <>
struct Chunk8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = ld_stream16(p);
        b = ld_stream16(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
};

__device__ __forceinline__ float absmax8(const float (&v)[8])
{
    float a = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
    return a;
}

// ------------------------------------------------------------ decode

// Four E4M3 codes (little-endian in w) -> their exact values: each pair of
// codes widens to FP16x2 (exact: E4M3 is a subset of FP16), each FP16 to FP32.
__device__ __forceinline__ void decode4_e4m3(uint32_t w, float (&f)[4])
{
    asm("{\n\t.reg .b16 q0, q1, h0, h1, h2, h3;\n\t.reg .b32 p0, p1;\n\t"
        "mov.b32 {q0, q1}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 p0, q0;\n\t"
        "cvt.rn.f16x2.e4m3x2 p1, q1;\n\t"
        "mov.b32 {h0, h1}, p0;\n\t"
        "mov.b32 {h2, h3}, p1;\n\t"
        "cvt.f32.f16 %0, h0;\n\t"
        "cvt.f32.f16 %1, h1;\n\t"
        "cvt.f32.f16 %2, h2;\n\t"
        "cvt.f32.f16 %3, h3;\n\t}"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
        : "r"(w));
}

}  // namespace

}  // namespace fp8fg
