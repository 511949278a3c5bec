// act.cuh -- the gated block's activations and their derivatives in fp32
// (include/syn_ffn.h).
#pragma once

#include "syn_ffn.h"
#include "window.cuh"

namespace syn {
namespace ffn {

__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float inverse(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / (1 + exp(-z)), to 2^-23 (8 + |z|) of itself: the exponential's argument is rounded, which
// counts with its size (1e-6 at 1, 1e-5 at -80)
__device__ __forceinline__ float sigmoid(float z) { return inverse(1.f + exp2_of(-1.4426950409f * z)); }

// The tanh form is g * sigmoid(2 sqrt(2/pi) (g + 0.044715 g^3)); g is held within
// 20, where the sigmoid is 0 or 1 in fp32, so that no power of it overflows.
__device__ __forceinline__ float tanh_gate(float g, float &slope) {
    const float t = fminf(fmaxf(g, -20.f), 20.f), t2 = t * t;
    const float s = sigmoid(t * fmaf(0.07135481283f, t2, 1.5957691216f));
    slope = s * (1.f - s) * fmaf(0.2140644385f, t2, 1.5957691216f);
    return s;
}
// Phi(g), and exp(-g^2 / 2).  Phi(-x) = exp(-x^2 / 2) t P(t) with t = 1 / (1 + 0.3 x) for
// x >= 0 (the form of Abramowitz and Stegun, 7.1.26), P fitted for the least relative error:
// 4.5e-7 at every x in fp32, and the exponential's 2^-24 g^2.  (The library's
// complementary error function takes 40 instructions more: 23 of 60 us for 19456
// tokens, 128 -> 1280.)
__device__ constexpr float kNormal[8] = {0.11963193864f, 0.12071329355f, 0.1001686975f,  0.12771588564f,
                                         -0.05207988992f, 0.20460686088f, -0.15618763864f, 0.03543076664f};
__device__ __forceinline__ float normal_gate(float g, float &bell) {
    const float t = inverse(fmaf(fabsf(g), 0.3f, 1.f));
    bell = exp2_of(g * (g * -0.7213475204f));
    float s = fmaf(t, kNormal[7], kNormal[6]);
#pragma unroll
    for (int i = 5; i >= 0; --i) s = fmaf(t, s, kNormal[i]);
    s = s * (t * bell);
    return g > 0.f ? 1.f - s : s;
}

// act(g), and its derivative
template <int ACT> __device__ __forceinline__ float act_grad(float g, float &d) {
    if (ACT == SYN_ACT_SILU) {
        const float s = sigmoid(g);
        d = s * fmaf(g, 1.f - s, 1.f);
        return g * s;
    }
    if (ACT == SYN_ACT_GELU) {
        float bell;
        const float s = normal_gate(g, bell);
        d = fmaf(g * 0.3989422804f, bell, s);
        return g * s;
    }
    float slope;
    const float s = tanh_gate(g, slope);
    d = fmaf(g, slope, s);
    return g * s;
}

// act(g) u of two values at once, with one instruction for both where there is one (19456
// tokens, 128 -> 1280: GELU 28.4 -> 26.9 us, tanh form 25.6 -> 22.9, SiLU level)
using window::add2;
using window::f2;
using window::fma2;
using window::mul2;
using window::unf2;
__device__ __forceinline__ uint64_t twice(float v) { return f2(v, v); }
template <float (*F)(float)> __device__ __forceinline__ uint64_t each(uint64_t v) {
    float a, b;
    unf2(v, a, b);
    return f2(F(a), F(b));
}
__device__ __forceinline__ float within20(float g) { return fminf(fmaxf(g, -20.f), 20.f); }
__device__ __forceinline__ float size_of(float g) { return fabsf(g); }
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
    return each<inverse>(add2(each<exp2_of>(mul2(z, twice(-1.4426950409f))), twice(1.f)));
}
template <int ACT> __device__ __forceinline__ uint64_t act_of(uint64_t g) {
    if (ACT == SYN_ACT_SILU) return mul2(g, sigmoid2(g));
    if (ACT == SYN_ACT_GELU) {
        const uint64_t t = each<inverse>(fma2(each<size_of>(g), twice(0.3f), twice(1.f)));
        const uint64_t bell = each<exp2_of>(mul2(g, mul2(g, twice(-0.7213475204f))));
        uint64_t s = fma2(t, twice(kNormal[7]), twice(kNormal[6]));
#pragma unroll
        for (int i = 5; i >= 0; --i) s = fma2(t, s, twice(kNormal[i]));
        s = mul2(s, mul2(t, bell));
        float a, b, p, q, v, w;
        unf2(s, a, b);
        unf2(fma2(s, twice(-1.f), twice(1.f)), p, q);
        unf2(g, v, w);
        return mul2(g, f2(v > 0.f ? p : a, w > 0.f ? q : b));
    }
    const uint64_t t = each<within20>(g);
    return mul2(g, sigmoid2(mul2(t, fma2(twice(0.07135481283f), mul2(t, t), twice(1.5957691216f)))));
}

template <int ACT> __device__ __forceinline__ void gated(float &g0, float &g1, float u0, float u1) {
    unf2(mul2(act_of<ACT>(f2(g0, g1)), f2(u0, u1)), g0, g1);
}

}  // namespace ffn
}  // namespace syn
