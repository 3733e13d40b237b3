// fp8mm_act.cuh -- activations and their slopes, fp32 in and out.
//
//   relu       max(x, 0)
//   gelu       x Phi(x), Phi the normal distribution function
//   gelu_tanh  x (1 + tanh u) / 2 = x s(2u), u = sqrt(2/pi) (x + 0.044715 x^3),
//              s the logistic function: no cancellation for negative x
//   silu       x s(x)
//
// All go through one exponential and one reciprocal (ex2.approx and
// rcp.approx, relative errors of about 2^-22 and 2^-23), two elements at a
// time (f32x2): 5 to 14 instructions per element, so that the products'
// epilogues stay hidden behind the matrix instructions of the next tile.
//
// Phi: for a = |x|, Phi(-a) = exp(-a^2/2) h(a), where h is half the scaled
// complementary error function of a/sqrt(2). h falls like 1/a, so it is a
// polynomial in t = 1/(1 + p a) without constant term (the form of
// C. Hastings, "Approximations for Digital Computers", 1955). The seven
// coefficients and p are a least-maximum fit of the relative error over
// 0 <= a <= 20 against scipy's erfcx: at most 1.3e-6 of h, so Phi keeps its
// relative accuracy in the tail (with the rounding of the exponent's argument
// 8e-6 at x = -13), where 1 + erf(x) has none left.
//
// Limits: NaN gives NaN; -inf gives -0 or +0 (relu: 0), +inf gives +inf;
// slopes are 0 and 1 there. The arguments are clamped where the function has
// reached its limit in fp32, so that inf never meets 0.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

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

// ------------------------------------------------------ pairs of values ---

struct Pair {
    float lo, hi;
};

__device__ __forceinline__ uint64_t pack(Pair p) { return ptx::f32x2(p.lo, p.hi); }
__device__ __forceinline__ uint64_t both(float c) { return ptx::f32x2(c, c); }
__device__ __forceinline__ Pair unpack(uint64_t v)
{
    Pair p;
    ptx::unpack_f32x2(v, p.lo, p.hi);
    return p;
}
__device__ __forceinline__ uint64_t ex2_pair(uint64_t v)
{
    const Pair p = unpack(v);
    return ptx::f32x2(ex2_approx(p.lo), ex2_approx(p.hi));
}
__device__ __forceinline__ uint64_t rcp_pair(uint64_t v)
{
    const Pair p = unpack(v);
    return ptx::f32x2(rcp_approx(p.lo), rcp_approx(p.hi));
}

// 1 / (1 + 2^v)
__device__ __forceinline__ uint64_t rcp_1p_ex2(uint64_t v) { return rcp_pair(ptx::add_f32x2(ex2_pair(v), both(1.0f))); }

// Phi(-a) for 0 <= a <= 20, given -a; e receives exp(-a^2/2).
__device__ __forceinline__ uint64_t normal_tail(uint64_t neg_a, uint64_t &e)
{
    const uint64_t t = rcp_pair(ptx::fma_f32x2(both(-0.36864640577302416f), neg_a, both(1.0f)));
    e = ex2_pair(ptx::mul_f32x2(ptx::mul_f32x2(neg_a, neg_a), both(-0.5f * kLog2e)));
    uint64_t h = both(0.04837304787388369f);
    h = ptx::fma_f32x2(h, t, both(-0.17252712897935096f));
    h = ptx::fma_f32x2(h, t, both(0.15209262775945798f));
    h = ptx::fma_f32x2(h, t, both(0.0424434924047982f));
    h = ptx::fma_f32x2(h, t, both(0.13644234400211985f));
    h = ptx::fma_f32x2(h, t, both(0.14606507133564497f));
    h = ptx::fma_f32x2(h, t, both(0.1471111567833028f));
    return ptx::mul_f32x2(h, ptx::mul_f32x2(t, e));
}

// x Phi(x) = max(x, 0) - |x| Phi(-|x|); Phi(-20) is 0 in fp32.
__device__ __forceinline__ Pair act_gelu(Pair x)
{
    const uint64_t na = ptx::f32x2(fmaxf(-fabsf(x.lo), -20.0f), fmaxf(-fabsf(x.hi), -20.0f));
    uint64_t e;
    const uint64_t q = normal_tail(na, e);
    return unpack(ptx::fma_f32x2(na, q, ptx::f32x2(max_nan(x.lo, 0.0f), max_nan(x.hi, 0.0f))));
}

constexpr float kGeluTanhC0 = 1.5957691216057308f;               // 2 sqrt(2/pi)
constexpr float kGeluTanhC1 = 1.5957691216057308f * 0.044715f;

// s(2u) is 0 in fp32 at x = -20
__device__ __forceinline__ Pair act_gelu_tanh(Pair x)
{
    const uint64_t v = ptx::f32x2(max_nan(x.lo, -20.0f), max_nan(x.hi, -20.0f));
    const uint64_t k = ptx::fma_f32x2(both(-kLog2e * kGeluTanhC1), ptx::mul_f32x2(v, v), both(-kLog2e * kGeluTanhC0));
    return unpack(ptx::mul_f32x2(v, rcp_1p_ex2(ptx::mul_f32x2(v, k))));
}

// x s(x) is 0 in fp32 at x = -110
__device__ __forceinline__ Pair act_silu(Pair x)
{
    const uint64_t v = ptx::f32x2(max_nan(x.lo, -110.0f), max_nan(x.hi, -110.0f));
    return unpack(ptx::mul_f32x2(v, rcp_1p_ex2(ptx::mul_f32x2(v, both(-kLog2e)))));
}

// ------------------------------------------------------------- slopes ---

// v where x > 0, 0 elsewhere (also for an infinite v), NaN for a NaN x
__device__ __forceinline__ float times_slope_relu(float v, float x) { return x > 0.0f ? v : (x != x ? x : 0.0f); }

// Phi(x) + x exp(-x^2/2) / sqrt(2 pi)
__device__ __forceinline__ uint64_t slope_gelu(Pair x)
{
    x.lo = clamp_nan(x.lo, 20.0f);
    x.hi = clamp_nan(x.hi, 20.0f);
    uint64_t e;
    const uint64_t q2 = normal_tail(ptx::f32x2(-fabsf(x.lo), -fabsf(x.hi)), e);
    const Pair q = unpack(q2), p = unpack(ptx::fma_f32x2(q2, both(-1.0f), both(1.0f)));
    const uint64_t phi = ptx::f32x2(x.lo > 0.0f ? p.lo : q.lo, x.hi > 0.0f ? p.hi : q.hi);
    return ptx::fma_f32x2(ptx::mul_f32x2(pack(x), both(0.3989422804014327f)), e, phi);
}

// s + x s (1 - s) (2u)'
__device__ __forceinline__ uint64_t slope_gelu_tanh(Pair x)
{
    const uint64_t v = ptx::f32x2(clamp_nan(x.lo, 20.0f), clamp_nan(x.hi, 20.0f));
    const uint64_t v2 = ptx::mul_f32x2(v, v);
    const uint64_t k = ptx::fma_f32x2(both(-kLog2e * kGeluTanhC1), v2, both(-kLog2e * kGeluTanhC0));
    const uint64_t s = rcp_1p_ex2(ptx::mul_f32x2(v, k));
    const uint64_t d = ptx::fma_f32x2(both(3.0f * kGeluTanhC1), v2, both(kGeluTanhC0));
    const uint64_t r = ptx::mul_f32x2(s, ptx::fma_f32x2(s, both(-1.0f), both(1.0f)));
    return ptx::fma_f32x2(r, ptx::mul_f32x2(v, d), s);
}

// s (1 + x (1 - s))
__device__ __forceinline__ uint64_t slope_silu(Pair x)
{
    const uint64_t v = ptx::f32x2(clamp_nan(x.lo, 110.0f), clamp_nan(x.hi, 110.0f));
    const uint64_t s = rcp_1p_ex2(ptx::mul_f32x2(v, both(-kLog2e)));
    return ptx::mul_f32x2(s, ptx::fma_f32x2(v, ptx::fma_f32x2(s, both(-1.0f), both(1.0f)), both(1.0f)));
}

// One switch for a whole array, so that the unrolled loops hold no branches.
template <int CH>
__device__ __forceinline__ void apply_act(int act, float (&v)[CH])
{
    static_assert(CH % 2 == 0, "pairs");
#define FP8MM_EACH_PAIR(expr)                      \
    _Pragma("unroll") for (int j = 0; j < CH; j += 2) \
    {                                              \
        const Pair r = expr(Pair{v[j], v[j + 1]}); \
        v[j] = r.lo;                               \
        v[j + 1] = r.hi;                           \
    }
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = max_nan(v[j], 0.0f);
        break;
    case kActGelu: FP8MM_EACH_PAIR(act_gelu) break;
    case kActGeluTanh: FP8MM_EACH_PAIR(act_gelu_tanh) break;
    case kActSilu: FP8MM_EACH_PAIR(act_silu) break;
    default: break;
    }
#undef FP8MM_EACH_PAIR
}

// v *= slope(z)
template <int CH>
__device__ __forceinline__ void apply_slope(int act, float (&v)[CH], const float (&z)[CH])
{
    static_assert(CH % 2 == 0, "pairs");
#define FP8MM_EACH_PAIR(expr)                                                                       \
    _Pragma("unroll") for (int j = 0; j < CH; j += 2)                                               \
    {                                                                                               \
        const Pair r = unpack(ptx::mul_f32x2(ptx::f32x2(v[j], v[j + 1]), expr(Pair{z[j], z[j + 1]}))); \
        v[j] = r.lo;                                                                                \
        v[j + 1] = r.hi;                                                                            \
    }
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int j = 0; j < CH; ++j)
            v[j] = times_slope_relu(v[j], z[j]);
        break;
    case kActGelu: FP8MM_EACH_PAIR(slope_gelu) break;
    case kActGeluTanh: FP8MM_EACH_PAIR(slope_gelu_tanh) break;
    case kActSilu: FP8MM_EACH_PAIR(slope_silu) break;
    default: break;
    }
#undef FP8MM_EACH_PAIR
}

}  // namespace fp8mm
