// The gated activation u g / (1 + exp(-g)) and the pair arithmetic of the quantizers that fuse it.
#pragma once

#include <stdint.h>

namespace q8 {

// Two fp32 values as one operand: the pair operations take one issue slot for two.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Two of u * g / (1 + exp(-g)) for |g| <= kGateFast. exp(-g) = 2^h e^-d with h = fl(-g log2 e) and d = g + h ln 2, which is
// under 2^-16, so that e^-d is 1 - d: without d the rounding of h would cost |g| half steps. Off by less than
// 2^-20 of the value: the fast exponential 2^-22, ln 2 in 24 bits times h 2^-22, 1 - d and the sum half a step each
// (2^-24), the fast reciprocal 2^-23, two products half a step each. (32768 x 2048 bf16: 53.7 us without d, 56.0 with it,
// 67.6 with fp32's own exponential for every gate.)
constexpr float kGateFast = 87.0f;   // the exponential and its reciprocal are normal numbers
__device__ __forceinline__ void silu_mul2(float& g0, float& g1, float u0, float u1) {
    const uint64_t g = pack2(g0, g1), one = pack2(1.0f, 1.0f);
    const uint64_t h = mul2(g, pack2(-1.4426950408889634f, -1.4426950408889634f));
    const uint64_t d = fma2(h, pack2(0.6931471805599453f, 0.6931471805599453f), g);
    float e0, e1, r0, r1;
    unpack2(h, e0, e1);
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e0) : "f"(e0));
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e1) : "f"(e1));
    unpack2(fma2(pack2(e0, e1), fma2(d, pack2(-1.0f, -1.0f), one), one), e0, e1);
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r0) : "f"(e0));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r1) : "f"(e1));
    unpack2(mul2(mul2(g, pack2(r0, r1)), pack2(u0, u1)), g0, g1);
}

// The same for any gate, from t = exp(-|g|), so that nothing overflows before the value does and the tail of a closed gate
// keeps its bits: u g / (1 + t) for g >= 0, u g t / (1 + t) below (the reciprocal is of a number between 1 and 2). Where t
// is subnormal (|g| > 87.3) two of its steps, 2^-148 |g u|, come on top.
__device__ __forceinline__ float silu_mul_far(float g, float u) {
    const float t = expf(-fabsf(g));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.0f + t));
    return (g < 0.0f ? g * t : g) * r * u;
}

// max(m, |a|, |b|), NaN if one is (its bits are then above those of inf).
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

}  // namespace q8
