// act.cuh -- the activations of the gated form and their slopes, in float32.
//
// sigmoid(x) = 1 / (1 + e^-x) with the approximate base-2 exponential and
// reciprocal instructions, subnormals flushed: e^-x overflows to infinity for x
// below about -88, where the reciprocal is 0, and results below 2^-126 are 0.
// Relative error a few units in the last place (and |x| 2^-23 from the argument),
// well below the rounding of the tensor-core sums that go in.  The forms that keep
// subnormals (__expf, __fdividef) take three more instructions each, and an
// epilogue warp, alone on its scheduler, is bound by its instructions: with them
// the activation took 32 of 104 us (FP4, 4096 x 14336 x 512).
#pragma once

#include <stdint.h>

namespace tcg {

// (the values of gemm_act_t)
enum : int32_t { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActRelu = 3, kActSigmoid = 4 };

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, and 1 / x
__device__ __forceinline__ float exp2_approx(float x)
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

__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_approx(1.f + exp2_approx(-kLog2e * x)); }

// gelu_tanh: 0.5 g (1 + tanh(y)) = g sigmoid(2 y), y = sqrt(2 / pi) (g + 0.044715 g^3)
constexpr float kGeluTanh1 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluTanh3 = 0.07135481282720802f;  // 0.044715 of that
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// Phi(g), the normal distribution function, and e = exp(-g^2 / 2): the rational
// approximation 7.1.26 of Abramowitz and Stegun's Handbook of Mathematical
// Functions, erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2) with t = 1 / (1 + p x) for x
// = |g| / sqrt(2), within 1.5e-7 (7.5e-8 of Phi).  One exponential, which the
// slope needs anyway, and no branch; for g < 0 nothing cancels.
__device__ __forceinline__ float normal_cdf(float g, float &e)
{
    const float x = fabsf(g) * kSqrtHalf;
    const float t = rcp_approx(1.f + 0.3275911f * x);
    e = exp2_approx(-0.5f * kLog2e * g * g);
    const float q = 0.5f * e * t *
                    (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    return g < 0.f ? q : 1.f - q;  // (a NaN stays one)
}

template <int ACT>
__device__ __forceinline__ float act_value(float g)
{
    if (ACT == kActSilu)
        return g * sigmoid_f32(g);
    if (ACT == kActGelu) {
        float e;
        return g * normal_cdf(g, e);
    }
    if (ACT == kActGeluTanh)
        return g * sigmoid_f32(g * (kGeluTanh1 + kGeluTanh3 * g * g));
    if (ACT == kActRelu)
        return g <= 0.f ? 0.f : g;  // (a NaN stays one)
    return sigmoid_f32(g);
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void act_value_slope(float g, float &a, float &s)
{
    if (ACT == kActSilu) {
        const float p = sigmoid_f32(g);
        a = g * p;
        s = p * (1.f + g * (1.f - p));
    } else if (ACT == kActGelu) {
        float e;
        const float c = normal_cdf(g, e);
        a = g * c;
        s = c + g * kInvSqrt2Pi * e;
    } else if (ACT == kActGeluTanh) {
        const float p = sigmoid_f32(g * (kGeluTanh1 + kGeluTanh3 * g * g));
        a = g * p;
        // (past |g| = 30, p is 0 or 1 and the second term 0: keep g^3 finite there)
        const float c = fminf(fmaxf(g, -30.f), 30.f);
        s = p + c * p * (1.f - p) * (kGeluTanh1 + 3.f * kGeluTanh3 * c * c);
    } else if (ACT == kActRelu) {
        a = g <= 0.f ? 0.f : g;
        s = g <= 0.f ? 0.f : (g > 0.f ? 1.f : g);
    } else {
        const float p = sigmoid_f32(g);
        a = p;
        s = p * (1.f - p);
    }
}

// Call f with the activation as a compile-time constant (decltype(tag)::value).
template <int ACT>
struct ActTag {
    static constexpr int value = ACT;
};

template <typename F>
__device__ __forceinline__ void with_act(int32_t act, F f)
{
    switch (act) {
    case kActSilu: f(ActTag<kActSilu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    case kActRelu: f(ActTag<kActRelu>{}); break;
    default: f(ActTag<kActSigmoid>{}); break;
    }
}

}  // namespace tcg
