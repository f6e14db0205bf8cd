// fp8fg_swiglu.cuh -- the SwiGLU's arithmetic on two lanes at once (packed
// FP32x2 instructions), and the warp-wide max-abs its quantizers use.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fp8fg_device.cuh"

namespace fp8fg {

namespace {

// Two FP32 values in one 64-bit register pair, computed on together: each operation is
// one packed instruction, each lane rounded like the scalar one.  (The float2
// intrinsics for the same instructions made the kernels here 12 to 17 % slower.)
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo(F2 a)
{
    float x;
    asm("mov.b64 {%0, _}, %1;" : "=f"(x) : "l"(a.v));
    return x;
}
__device__ __forceinline__ float hi(F2 a)
{
    float y;
    asm("mov.b64 {_, %0}, %1;" : "=f"(y) : "l"(a.v));
    return y;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + exp(-g)).  exp(-g) is 2^t for t = -g * log2(e), rounded: that alone would cost |g| * 2^-23 of it
// (the product's rounding, and log2(e)'s).  What is lost, -g - t * ln(2), is exact in one FMA but for
// ln(2)'s rounding (2^-28.4 of it), and exp(-g) = 2^t * (1 + that) to FP32's precision.  The
// exponential and the reciprocal are the hardware's approximations, at most two and one units in the last
// place off.

// The reciprocal of 1 + e * (1 + what is lost), e = 2^t.
__device__ __forceinline__ F2 rcp_1p_exp(F2 e, F2 t, F2 g)
{
    const F2 minus = f2(-1.0f, -1.0f), d = fma2(t, f2(0.6931471805599453f, 0.6931471805599453f), g);
    const F2 y = fma2(e, d, fma2(e, minus, minus));      // negated, as d is minus what is lost
    return f2(rcp_approx(-lo(y)), rcp_approx(-hi(y)));
}

// For |g| <= kNearGates, where exp(-g) is below 2^126 and its reciprocal a normal number (ln(2^126) = 87.3).
constexpr float kNearGates = 87.0f;
__device__ __forceinline__ F2 sigmoid2(F2 g)
{
    const F2 t = g * f2(-1.4426950408889634f, -1.4426950408889634f);      // -log2(e)
    const F2 e = f2(ex2_approx(lo(t)), ex2_approx(hi(t)));
    return rcp_1p_exp(e, t, g);
}

// The sigmoid of any gates, as a product r * f: below about -86.6, r stays at 2^-125 and f is
// the rest, so that products with r first (g * r * f) are right down to FP32's smallest normal
// number, where the sigmoid itself no longer is one; above, f is 1 and r has sigmoid2's bits.  Beyond
// -340 and 138, where it is 0 and 1, the gate is taken for these: nothing overflows, not even an infinity.
__device__ __forceinline__ void sigmoid2_far(F2 g, F2& r, F2& f)
{
    const F2 c = f2(fminf(fmaxf(lo(g), -340.0f), 138.0f), fminf(fmaxf(hi(g), -340.0f), 138.0f));
    const F2 t = c * f2(-1.4426950408889634f, -1.4426950408889634f);
    r = rcp_1p_exp(f2(ex2_approx(fminf(lo(t), 125.0f)), ex2_approx(fminf(hi(t), 125.0f))), t, c);
    f = f2(ex2_approx(fminf(125.0f - lo(t), 0.0f)), ex2_approx(fminf(125.0f - hi(t), 0.0f)));
}

// silu(g) = g * sigmoid(g); FAR for any gates, else for |g| <= kNearGates (with the same bits there).
template <bool FAR>
__device__ __forceinline__ F2 silu2(F2 g)
{
    if (!FAR) return g * sigmoid2(g);
    F2 r, f;
    sigmoid2_far(g, r, f);
    return g * r * f;
}

// max(|a|, |b|, |c|): one three-input instruction.
__device__ __forceinline__ float absmax3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// Max of |a| over the warp, in every lane.
__device__ __forceinline__ float warp_absmax(float a)
{
    float r;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
    return r;
}

}  // namespace

}  // namespace fp8fg
