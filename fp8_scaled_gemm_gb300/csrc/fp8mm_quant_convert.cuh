// fp8mm_quant_convert.cuh -- from a value and a scale to an fp8 code.
//
// Division: x / scale must be the correctly rounded fp32 quotient, because
// the quotient decides an fp8 code. For scales in [2^-80, 2^100) the kernels
// use r = RN(1/scale), q0 = RN(x r), e = RN(q0 scale - x) (one FMA, exact)
// and q1 = RN(q0 - e r) (one FMA): Markstein's correction of a quotient by
// its residual (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990), which gives
// RN(x / scale) for every bf16 x and every scale this recipe produces while
// the residual stays a normal number, i.e. for |x| >= 2^-100. Smaller |x|
// have |x / scale| < 2^-20, below half the smallest fp8 subnormal, and q1
// is then within a few fp32 ulps of the quotient: the code is +-0 either
// way. The signs of the FMA operands are chosen so that x = -0 gives -0.
// Scales outside that range, zero, inf or NaN take the IEEE division
// __fdiv_rn.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8q {

__device__ __forceinline__ float qmax_of(int q_type) { return q_type == 0 ? 448.0f : 57344.0f; }

__device__ __forceinline__ bool in_reciprocal_range(float s) { return s >= 0x1p-80f && s < 0x1p100f; }

// amax / qmax, correctly rounded: in the reciprocal's range as a quotient by 7 x
// 2^n through the rounded reciprocal and one correction, which was compared with
// the division for every mantissa.
__device__ __forceinline__ float row_scale(float amax, int q_type)
{
    const float qmax = qmax_of(q_type), c = q_type == 0 ? 1.0f / 448.0f : 1.0f / 57344.0f;
    const float s0 = __fmul_rn(amax, c), s = __fmaf_rn(__fmaf_rn(s0, -qmax, amax), c, s0);
    return in_reciprocal_range(s) ? s : __fdiv_rn(amax, qmax);
}

struct Divider {
    float s, r;
    int mode;   // 0: zero scale, 1: reciprocal + one correction, 2: IEEE division
};

__device__ __forceinline__ Divider make_divider(float s)
{
    Divider d;
    d.s = s;
    d.r = 0.0f;
    if (s == 0.0f) {
        d.mode = 0;
    } else if (in_reciprocal_range(s)) {
        d.r = __frcp_rn(s);
        d.mode = 1;
    } else {
        d.mode = 2;
    }
    return d;
}

// x / scale for the reciprocal path (mode 1); x is finite there.
__device__ __forceinline__ float div_fast(const Divider &d, float x)
{
    const float q0 = __fmul_rn(x, d.r);
    const float e = __fmaf_rn(q0, d.s, -x);
    return __fmaf_rn(-e, d.r, q0);
}

// x / scale for the other modes.
__device__ __forceinline__ float div_slow(const Divider &d, float x)
{
    if (d.mode == 0)
        return x;                                           // +-0 stays +-0
    const float v = __fdiv_rn(x, d.s);
    return v != v ? __uint_as_float(0x7FFFFFFFu) : v;       // one NaN code
}

// Two fp32 values to two fp8 codes (lo in the low byte), round to nearest even,
// saturating at +-qmax: the same as clamping to [-qmax, qmax] and rounding.
__device__ __forceinline__ uint32_t cvt_pair(float lo, float hi, int q_type)
{
    uint16_t r;
    if (q_type == 0)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fp8q
