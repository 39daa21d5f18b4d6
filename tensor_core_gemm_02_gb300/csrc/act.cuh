// act.cuh -- the activations of the gated form and their slopes, in float32.
//
// sigmoid(x) = 1 / (1 + e^-x) with the approximate base-2 exponential and
// reciprocal instructions, subnormals flushed: e^-x overflows to infinity for x
// below about -88, where the reciprocal is 0, and results below 2^-126 are 0.
// Relative error a few units in the last place and 0.75 |x| 2^-23 from the argument
// (gelu: 1.25 g^2 / 2 of them), also where the result is small.  The forms that keep
// subnormals (__expf, __fdividef) take three more instructions each, and an
// epilogue warp, alone on its scheduler, is bound by its instructions (FP4, 4096 x
// 14336 x 512, with them 132 us, 115 without, one epilogue group at the time).
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
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// Phi(g), the normal distribution function, and e = exp(-g^2 / 2).  With x = |g| /
// sqrt(2), erfc(x) = e^(-x^2) t P(t), t = 1 / (1 + 0.33 x): P of degree 7 was fitted
// for the smallest largest relative error over 0 <= x <= 10 (Lawson's reweighted least
// squares on Chebyshev polynomials; past that e is 0), which is 9.4e-8, and 4.5e-7 with
// float32's roundings.  Relative, because the left tail is small: 7.1.26 of Abramowitz
// and Stegun's Handbook, three terms shorter and within 7.5e-8 of Phi, is off by 5e-5 of
// Phi at g = -3 and 5e-4 at -4.  One exponential, which the slope needs anyway, and
// no branch; for g < 0 nothing cancels.  (The three terms more: FP4 8192 x 14336 x 4096 359 ->
// 374 us, 4096 x 14336 x 512 84 -> 87, bf16 98 -> 100; the gradients' elementwise part
// 8192 x 14336 191 -> 195.)
__device__ __forceinline__ float normal_cdf(float g, float &e)
{
    const float t = rcp_approx(1.f + 0.23334524f * fabsf(g));  // (0.33 / sqrt(2))
    e = exp2_approx(-0.5f * kLog2e * g * g);
    const float p = 0.091478062f +
                    t * (0.1006113605f +
                         t * (0.02361230475f +
                              t * (0.2042461265f + t * (-0.1755704975f + t * (0.2301159335f + t * -0.0676721895f)))));
    const float q = e * t * (0.093178896f + t * p);  // (P / 2)
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
