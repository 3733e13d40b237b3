// fp8mm_act.cuh -- activations and their slopes, fp32 in and out.
//
//   relu       max(x, 0)
//   gelu       x Phi(x), Phi the normal distribution function
//   gelu_tanh  x (1 + tanh u) / 2 = x s(2u), u = sqrt(2/pi) (x + 0.044715 x^3),
//              s the logistic function: no cancellation for negative x
//   silu       x s(x)
//
// All go through one exponential and one reciprocal (ex2.approx and
// rcp.approx, relative errors of about 2^-22 and 2^-23), which the products'
// epilogues can afford: 10 to 16 instructions per element.
//
// Phi: for a = |x|, Phi(-a) = exp(-a^2/2) h(a), where h is half the scaled
// complementary error function of a/sqrt(2). h falls like 1/a, so it is a
// polynomial in t = 1/(1 + p a) without constant term (the form of
// C. Hastings, "Approximations for Digital Computers", 1955). The seven
// coefficients and p are a least-maximum fit of the relative error over
// 0 <= a <= 20 against scipy's erfcx: at most 1.3e-6 of h, so Phi keeps that
// relative accuracy in its tail, where 1 + erf(x) has none left.
//
// Limits: NaN gives NaN; -inf gives -0 or +0 (relu: 0), +inf gives +inf;
// slopes are 0 and 1 there. The arguments are clamped where the function has
// reached its limit in fp32, so that inf never meets 0.
#pragma once

#include <cuda_runtime.h>

namespace fp8mm {

// activation codes of the C ABI
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// min and max that return NaN when either argument is NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float clamp_nan(float x, float lim) { return min_nan(max_nan(x, -lim), lim); }

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-x)); 0 where exp(-x) overflows.
__device__ __forceinline__ float logistic(float x) { return rcp_approx(1.0f + ex2_approx(-kLog2e * x)); }

// Phi(-a) and exp(-a^2/2) for 0 <= a <= 20.
__device__ __forceinline__ float normal_tail(float a, float &e)
{
    const float t = rcp_approx(fmaf(0.36864640577302416f, a, 1.0f));
    e = ex2_approx((a * a) * (-0.5f * kLog2e));
    float h = 0.04837304787388369f;
    h = fmaf(h, t, -0.17252712897935096f);
    h = fmaf(h, t, 0.15209262775945798f);
    h = fmaf(h, t, 0.0424434924047982f);
    h = fmaf(h, t, 0.13644234400211985f);
    h = fmaf(h, t, 0.14606507133564497f);
    h = fmaf(h, t, 0.1471111567833028f);
    return h * (t * e);
}

__device__ __forceinline__ float act_relu(float x) { return max_nan(x, 0.0f); }

// x Phi(x) = max(x, 0) - |x| Phi(-|x|); Phi(-20) is 0 in fp32.
__device__ __forceinline__ float act_gelu(float x)
{
    const float a = fminf(fabsf(x), 20.0f);
    float e;
    const float q = normal_tail(a, e);
    return fmaf(-a, q, max_nan(x, 0.0f));
}

constexpr float kGeluTanhC0 = 1.5957691216057308f;               // 2 sqrt(2/pi)
constexpr float kGeluTanhC1 = 1.5957691216057308f * 0.044715f;

__device__ __forceinline__ float act_gelu_tanh(float x)
{
    x = max_nan(x, -20.0f);                                       // s(2u) is 0 there
    return x * logistic(x * fmaf(kGeluTanhC1, x * x, kGeluTanhC0));
}

__device__ __forceinline__ float act_silu(float x)
{
    x = max_nan(x, -110.0f);                                      // x s(x) is 0 there
    return x * logistic(x);
}

// ------------------------------------------------------------- slopes ---

__device__ __forceinline__ float slope_relu(float x) { return x > 0.0f ? 1.0f : (x != x ? x : 0.0f); }

// Phi(x) + x exp(-x^2/2) / sqrt(2 pi)
__device__ __forceinline__ float slope_gelu(float x)
{
    x = clamp_nan(x, 20.0f);
    float e;
    const float q = normal_tail(fabsf(x), e);
    return fmaf(x * 0.3989422804014327f, e, x > 0.0f ? 1.0f - q : q);
}

// s + x s (1 - s) (2u)'
__device__ __forceinline__ float slope_gelu_tanh(float x)
{
    x = clamp_nan(x, 20.0f);
    const float x2 = x * x;
    const float s = logistic(x * fmaf(kGeluTanhC1, x2, kGeluTanhC0));
    const float d = fmaf(3.0f * kGeluTanhC1, x2, kGeluTanhC0);
    return fmaf(s * (1.0f - s), x * d, s);
}

// s (1 + x (1 - s))
__device__ __forceinline__ float slope_silu(float x)
{
    x = clamp_nan(x, 110.0f);
    const float s = logistic(x);
    return s * fmaf(x, 1.0f - s, 1.0f);
}

// One switch for a whole array, so that the unrolled loops hold no branches.
template <int CH>
__device__ __forceinline__ void apply_act(int act, float (&v)[CH])
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = act_relu(v[j]);
        break;
    case kActGelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = act_gelu(v[j]);
        break;
    case kActGeluTanh:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = act_gelu_tanh(v[j]);
        break;
    case kActSilu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = act_silu(v[j]);
        break;
    default: break;
    }
}

// v *= slope(z)
template <int CH>
__device__ __forceinline__ void apply_slope(int act, float (&v)[CH], const float (&z)[CH])
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = z[j] <= 0.0f ? 0.0f : v[j] * slope_relu(z[j]);   // 0 below the kink, also for an infinite v
        break;
    case kActGelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] *= slope_gelu(z[j]);
        break;
    case kActGeluTanh:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] *= slope_gelu_tanh(z[j]);
        break;
    case kActSilu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] *= slope_silu(z[j]);
        break;
    default: break;
    }
}

}  // namespace fp8mm
