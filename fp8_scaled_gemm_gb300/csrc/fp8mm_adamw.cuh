// fp8mm_adamw.cuh -- one AdamW step over many tensors.
//
//   g  = grad * grad_scale
//   m' = b1 m + (1 - b1) g          v' = b2 v + (1 - b2) g^2
//   w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// in fp32, every operation rounded by itself (no contraction), so that a step
// gives the same bits as its formula written out in single operations.
//
// States in 8 bits: e4m3 codes in blocks of 256 elements with an fp32 scale
// each (largest magnitude / 448), m as itself and v as its root: the root
// halves the exponents v spans, and e4m3 with the block's scale then reaches
// 2^-18 of the block's largest. Codes are 6 to 12 % apart (the smallest ones up to
// twice), and a step moves the root of v by less than 0.05 % of itself with b2 =
// 0.999, m by (1 - b1) of its distance to g: where that is under half of the codes'
// distance, the nearest code is the old one for ever. The root of v is therefore rounded
// up or down with the probabilities that keep its mean, by a hash of the element's place
// and of the step; it does not become zero unless it is, since it divides. m likewise with
// `stochastic`, which is how the states follow the ones in 32 bits over many steps.
// Without it m goes to the nearest code, but for an element whose gradient is zero. There
// the nearest code would hold m while v goes to its floor, and the weight would move for
// ever: with b1, b2 = 0.9, 0.95 by 0.7 lr a step, 2000 steps after its gradient ended;
// so it still does where a gradient is not zero but falls to a millionth.
//
// Bound by memory: with bf16 weights and gradients, fp32 originals and 8-bit
// states 16 bytes an element. A warp takes a block of 256 elements, 8
// consecutive ones a lane (16-byte accesses), so that a block's scale needs
// shuffles only. The tensors' addresses come in the kernel's parameters: no
// copy to the device, nothing kept, and a captured launch holds its own table.
#pragma once

#include "fp8mm_quant_convert.cuh"
#include "fp8mm_rows.cuh"

namespace fp8adam {

namespace ptx = fp8mm::ptx;

constexpr int kBlock = 256;            // elements of a block, of one warp
constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;          // 64 registers a thread; with 3 the loads' latency showed

struct Tensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *m_scale, *v_scale;
    long long count;
    int vec;                           // 16-byte accesses allowed (codes: 8)
};

struct Hyper {
    // 1 - lr wd, b1, 1 - b1, b2, 1 - b2, eps, lr / (1 - b1^t), 1 / sqrt(1 - b2^t);
    // made anew on the device where it holds lr or the step
    float keep, b1, b1c, b2, b2c, eps, step_size, root;
    double lr, rest1, beta1, beta2, weight_decay;      // rest1 = 1 - b1^t
    const float *lr_device;
    const int64_t *step_device;
    uint32_t step;                     // low bits, for the rounding
    int stochastic;                    // m's codes too
    const float *grad_scale;
};

// T tensors by value: few, some, or as many as 32 KB of parameters hold.
template <int T>
struct Params {
    Hyper h;
    int tensors, param_type, grad_type;
    long long blocks;
    long long first[T];                // a tensor's first block in the launch's order
    Tensor t[T];
};

constexpr int kFew = 32, kSome = 96, kMany = 400;
static_assert(sizeof(Params<kMany>) <= 32764, "kernel parameters");

// Eight elements of a lane as loaded, 2 or 4 bytes each.
struct Eight {
    uint32_t w[8];
};

__device__ __forceinline__ void load8(Eight &r, const void *base, int type, long long e)
{
    if (type == fp8rows::kF32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + e);
        const uint4 a = __ldcs(p), b = __ldcs(p + 1);
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    } else {
        const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(base) + e));
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    }
}

__device__ __forceinline__ void floats8(const Eight &r, int type, float (&v)[8])
{
    if (type == fp8rows::kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(r.w[i]);
    } else {
        fp8rows::Raw<2, 8> raw;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            raw.w[i] = r.w[i];
        fp8rows::to_float<2, 8>(raw, type == fp8rows::kF16, v);
    }
}

__device__ __forceinline__ float load1(const void *base, int type, long long e)
{
    return type == fp8rows::kF32 ? static_cast<const float *>(base)[e]
                                 : fp8rows::half_bits(static_cast<const unsigned short *>(base)[e], type == fp8rows::kF16);
}

__device__ __forceinline__ void store8(void *base, int type, long long e, const float (&v)[8])
{
    if (type == fp8rows::kF32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + e);
        __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
        __stcs(reinterpret_cast<uint4 *>(static_cast<unsigned short *>(base) + e),
               make_uint4(fp8rows::pack2(v[0], v[1], type), fp8rows::pack2(v[2], v[3], type),
                          fp8rows::pack2(v[4], v[5], type), fp8rows::pack2(v[6], v[7], type)));
    }
}

// Two e4m3 codes (low half first) to fp32.
__device__ __forceinline__ float2 decode2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float decode1(uint8_t code) { return decode2(code).x; }

// 32 bits for the rounding of element e at a step, of which v's root takes the upper 20 and m
// those of another product.
__device__ __forceinline__ uint32_t hash(uint32_t e, uint32_t step)
{
    uint32_t x = e * 0x9E3779B1u + step * 0x85EBCA77u;
    x = (x ^ (x >> 15)) * 0x2C1B3C6Du;
    x = (x ^ (x >> 13)) * 0x297A2D39u;
    return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t root_bits(uint32_t hash) { return hash >> 12; }
__device__ __forceinline__ uint32_t moment_bits(uint32_t hash) { return hash * 0x9E3779B1u >> 12; }

// q >= 0 (or NaN) to a value that e4m3 holds, up or down by u. Codes are 2^-3 of
// the power of two apart, 20 bits of an fp32 mantissa, and 2^-9 below 2^-6.
__device__ __forceinline__ float round_by(float q, uint32_t u)
{
    q = q > 448.0f ? 448.0f : q;
    if (q < 0x1p-6f)
        return q > 0.0f ? fmaxf(floorf(__fadd_rn(q * 512.0f, static_cast<float>(u) * 0x1p-20f)) * 0x1p-9f, 0x1p-9f) : q;
    return q == q ? __uint_as_float((__float_as_uint(q) + u) & ~0xFFFFFu) : q;
}

// The same for a finite q of either sign, and to zero as well: what is under 2^-6 with
// 2^-6 added, between which and 2^-5 codes are 2^-9 apart too. (Beyond 448 the conversion
// saturates. With round_by's conversions instead of these sums a step of 470 M elements
// took 1685 us, so 1459; to the nearest code 1293.)
__device__ __forceinline__ float round_signed(float q, uint32_t u)
{
    const float more = fabsf(q) < 0x1p-6f ? copysignf(0x1p-6f, q) : 0.0f;
    return __fsub_rn(__uint_as_float((__float_as_uint(__fadd_rn(q, more)) + u) & ~0xFFFFFu), more);
}

// ------------------------------------------- roots and quotients of pairs ---
// Correctly rounded, by P. Markstein's iterations ("Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990), on
// two values at once: a root from an approximate reciprocal root refined together with
// it, then corrected by its residual; a quotient from a refined reciprocal, corrected
// by its residual. CUDA's __fsqrt_rn and __fdiv_rn take 12 and 18 issue slots a value,
// these 5 and 4, and with the former the step with 8-bit states was bound by issue
// (470 M elements 1950 us). Compared with them for every mantissa (roots, reciprocals)
// in the operator's tests; a lane with a value outside their ranges takes CUDA's.
constexpr float kRootFrom = 0x1p-96f, kRootTo = 0x1p96f;

__device__ __forceinline__ uint64_t both(float v) { return ptx::f32x2(v, v); }
__device__ __forceinline__ float rsqrt_approx(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of three, NaN if one is; the least of three.
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float y;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Sums of pairs one value at a time: ptxas contracts a packed product and the packed
// sum behind it (also with -fmad=false), which would round once.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    float a0, a1, b0, b1;
    ptx::unpack_f32x2(a, a0, a1);
    ptx::unpack_f32x2(b, b0, b1);
    return ptx::f32x2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

// x in [kRootFrom, kRootTo]. (The signs are such that no operand has to be negated:
// h is minus half the reciprocal root, the residual is g^2 - x.)
__device__ __forceinline__ uint64_t root2(uint64_t x)
{
    float x0, x1;
    ptx::unpack_f32x2(x, x0, x1);
    const uint64_t y = ptx::f32x2(rsqrt_approx(x0), rsqrt_approx(x1));
    uint64_t g = ptx::mul_f32x2(x, y), h = ptx::mul_f32x2(y, both(-0.5f));
    const uint64_t e = ptx::fma_f32x2(h, g, both(0.5f));
    g = ptx::fma_f32x2(g, e, g);
    h = ptx::fma_f32x2(h, e, h);
    return ptx::fma_f32x2(ptx::fma_f32x2(g, g, ptx::mul_f32x2(x, both(-1.0f))), h, g);
}

// The rounded reciprocal of d in [2^-60, 2^60], from minus d.
__device__ __forceinline__ uint64_t reciprocal2(uint64_t d, uint64_t minus_d)
{
    float d0, d1;
    ptx::unpack_f32x2(d, d0, d1);
    const uint64_t y = ptx::f32x2(rcp_approx(d0), rcp_approx(d1));
    return ptx::fma_f32x2(y, ptx::fma_f32x2(minus_d, y, both(1.0f)), y);
}

// x / d from minus d and the rounded reciprocal y of d: |x| <= 2^60 (under 2^-90 the
// last bit may be another)
__device__ __forceinline__ uint64_t divide2(uint64_t x, uint64_t minus_d, uint64_t y)
{
    const uint64_t q = ptx::mul_f32x2(x, y);
    return ptx::fma_f32x2(ptx::fma_f32x2(q, minus_d, x), y, q);
}

// A scale, largest value / 448, with what a quotient by it needs.
struct Scale {
    float s, r;                        // r: its reciprocal, where `fast`
    bool fast;                         // see fp8q::Divider's mode 1
};

// The scales of a warp's block from every lane's largest |m| and v. The lower half of
// the warp works on m, the upper one on v and its root, on one value a lane.
__device__ __forceinline__ void block_scales(float most_m, float most_v, int lane, Scale &m, Scale &v)
{
    const bool upper = lane & 16;
    float x = fp8mm::max_nan(upper ? most_v : most_m, __shfl_xor_sync(0xFFFFFFFFu, upper ? most_m : most_v, 16));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        x = fp8mm::max_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    if (upper) {
        // (the largest root is the largest value's)
        float r, other;
        ptx::unpack_f32x2(root2(both(x)), r, other);
        x = x >= kRootFrom && x <= kRootTo ? r : __fsqrt_rn(x);
    }
    const float s = fp8q::row_scale(x, 0);
    float r = 0.0f;
    const bool fast = s >= 0x1p-59f && s <= 0x1p59f;
    if (fast) {
        float other;
        ptx::unpack_f32x2(reciprocal2(both(s), both(-s)), r, other);
    }
    m.s = __shfl_sync(0xFFFFFFFFu, s, 0);
    m.r = __shfl_sync(0xFFFFFFFFu, r, 0);
    v.s = __shfl_sync(0xFFFFFFFFu, s, 16);
    v.r = __shfl_sync(0xFFFFFFFFu, r, 16);
    m.fast = m.r != 0.0f;
    v.fast = v.r != 0.0f;
}

// The step's constants and a tensor's scales, as the elements' arithmetic takes them.
struct Factors {
    float keep, step_size, root, gs, ms, vs;
    uint32_t step;
    bool scaled_grad, stochastic;
    bool pairs;                        // eps and the root's factor allow roots and quotients of pairs
};

// ------------------------------------------------------- the step of one lane ---
// Eight elements: w, m and v (codes' values with BITS = 8) become the new ones, r the root of v; two at a time, in
// single operations each rounded by itself. Gives the largest |m| and v and the least
// v, of which the last is 0 where the pairs' range was left, and (BITS = 8) the elements
// whose m is to be rounded up or down, a bit each.
template <int BITS>
__device__ __forceinline__ void update(float (&w)[8], const float (&g)[8], float (&m)[8], float (&v)[8], float (&r)[8],
                                       const Hyper &h, const Factors &f, float &most_m, float &most_v, float &least, uint32_t &by_chance)
{
    uint64_t m2[4], v2[4];
    float least_g = INFINITY;
    least = kRootTo;
    most_m = most_v = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t gi = ptx::f32x2(g[2 * i], g[2 * i + 1]);
        m2[i] = ptx::f32x2(m[2 * i], m[2 * i + 1]);
        v2[i] = ptx::f32x2(v[2 * i], v[2 * i + 1]);
        if (f.scaled_grad)
            gi = ptx::mul_f32x2(gi, both(f.gs));
        if constexpr (BITS == 8) {
            float g0, g1;
            ptx::unpack_f32x2(gi, g0, g1);
            least_g = min3(least_g, fabsf(g0), fabsf(g1));
            m2[i] = ptx::mul_f32x2(m2[i], both(f.ms));
            v2[i] = ptx::mul_f32x2(v2[i], both(f.vs));
            v2[i] = ptx::mul_f32x2(v2[i], v2[i]);
        }
        m2[i] = add2(ptx::mul_f32x2(m2[i], both(h.b1)), ptx::mul_f32x2(gi, both(h.b1c)));
        v2[i] = add2(ptx::mul_f32x2(v2[i], both(h.b2)), ptx::mul_f32x2(ptx::mul_f32x2(gi, gi), both(h.b2c)));
        ptx::unpack_f32x2(m2[i], m[2 * i], m[2 * i + 1]);
        ptx::unpack_f32x2(v2[i], v[2 * i], v[2 * i + 1]);
        least = min3(least, v[2 * i], v[2 * i + 1]);
        most_v = max3_nan(most_v, v[2 * i], v[2 * i + 1]);
        most_m = max3_nan(most_m, fabsf(m[2 * i]), fabsf(m[2 * i + 1]));
    }
    by_chance = BITS == 8 && f.stochastic ? 0xFFu : 0u;
    if (BITS == 8 && least_g == 0.0f && !f.stochastic) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            by_chance |= (f.scaled_grad ? g[i] * f.gs : g[i]) == 0.0f ? 1u << i : 0u;
    }
    // v and |m| at most 2^59: the root, the denominator and m are in the quotient's range
    // when eps and the root's factor are (a NaN is not)
    if (least >= kRootFrom && most_m <= 0x1p59f && most_v <= 0x1p59f && f.pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t r2 = root2(v2[i]);
            const uint64_t d = add2(ptx::mul_f32x2(r2, both(f.root)), both(h.eps)), minus_d = ptx::mul_f32x2(d, both(-1.0f));
            const uint64_t q = divide2(m2[i], minus_d, reciprocal2(d, minus_d));
            const uint64_t w2 = add2(ptx::mul_f32x2(ptx::f32x2(w[2 * i], w[2 * i + 1]), both(f.keep)),
                                     ptx::mul_f32x2(q, both(-f.step_size)));
            ptx::unpack_f32x2(r2, r[2 * i], r[2 * i + 1]);
            ptx::unpack_f32x2(w2, w[2 * i], w[2 * i + 1]);
        }
    } else {
        least = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = __fsqrt_rn(v[i]);
            w[i] = __fsub_rn(__fmul_rn(w[i], f.keep),
                             __fmul_rn(__fdiv_rn(m[i], __fadd_rn(__fmul_rn(r[i], f.root), h.eps)), f.step_size));
        }
    }
}

// Codes of a lane's eight m (in place: their quotients by the new scale, which a
// conversion rounds, those of `by_chance` to values that e4m3 holds) and r (to values that
// e4m3 holds). `least`: of the r's squares, or 0.
__device__ __forceinline__ void encode(float (&m)[8], float (&r)[8], const Scale &ms, const Scale &vs, float least, uint32_t e0,
                                       int stride, uint32_t step, uint32_t by_chance)
{
    if (ms.fast && vs.fast) {
        // (the block's values are finite and at most 448 scales: the reciprocal's way,
        // and no clamp but the conversion's)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            ptx::unpack_f32x2(divide2(ptx::f32x2(m[i], m[i + 1]), both(-ms.s), both(ms.r)), m[i], m[i + 1]);
            ptx::unpack_f32x2(divide2(ptx::f32x2(r[i], r[i + 1]), both(-vs.s), both(vs.r)), r[i], r[i + 1]);
        }
        if (least >= 0x1.01p-12f * vs.s * vs.s) {
            // no root under 2^-6: see round_by
            if (by_chance == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = __uint_as_float((__float_as_uint(r[i]) + root_bits(hash(e0 + static_cast<uint32_t>(stride * i), step))) & ~0xFFFFFu);
                return;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = hash(e0 + static_cast<uint32_t>(stride * i), step);
                r[i] = __uint_as_float((__float_as_uint(r[i]) + root_bits(x)) & ~0xFFFFFu);
                if (by_chance >> i & 1)
                    m[i] = round_signed(m[i], moment_bits(x));
            }
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = ms.s == 0.0f ? 0.0f : __fdiv_rn(m[i], ms.s);
            r[i] = vs.s == 0.0f ? 0.0f : __fdiv_rn(r[i], vs.s);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t x = hash(e0 + static_cast<uint32_t>(stride * i), step);
        r[i] = round_by(r[i], root_bits(x));
        if ((by_chance >> i & 1) && fabsf(m[i]) <= 512.0f)      // (neither infinite nor NaN)
            m[i] = round_signed(m[i], moment_bits(x));
    }
}

// -------------------------------------------------------------- blocks ---
// W32: w is read as fp32 (from the master or an fp32 parameter), MASTER: there are
// masters, G32: gradients are fp32; else 16-bit types, of which only the conversions
// differ.

// Asks for a whole block's inputs in L2 (their scales beside them gave nothing), while the
// warp's block before it is worked on: from the 16 bytes that hold the first one, since codes
// may be aligned to 8.
__device__ __forceinline__ void fetch_l2(const void *p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(p) & ~15ull), "r"(bytes) : "memory");
}

template <int BITS, bool W32, bool MASTER, bool G32>
__device__ __forceinline__ void fetch_block(const Tensor &t, long long block)
{
    const long long at = block * kBlock;
    const void *w = MASTER ? static_cast<const void *>(t.master) : t.param;
    fetch_l2(static_cast<const char *>(w) + at * (W32 ? 4 : 2), kBlock * (W32 ? 4 : 2));
    fetch_l2(static_cast<const char *>(t.grad) + at * (G32 ? 4 : 2), kBlock * (G32 ? 4 : 2));
    fetch_l2(static_cast<const char *>(t.m) + at * (BITS / 8), kBlock * (BITS / 8));
    fetch_l2(static_cast<const char *>(t.v) + at * (BITS / 8), kBlock * (BITS / 8));
}

// A whole block in 16-byte words, 8 neighbours a lane.
template <int BITS, bool W32, bool MASTER, bool G32>
__device__ __forceinline__ void whole_block(const Tensor &t, long long block, int param_type, int grad_type, const Hyper &h, Factors &f,
                                            int lane)
{
    const long long at = block * kBlock + lane * 8;
    const int w_type = W32 ? fp8rows::kF32 : param_type, g_type = G32 ? fp8rows::kF32 : grad_type;
    Eight rw, rg, rm, rv;
    load8(rw, MASTER ? static_cast<const void *>(t.master) : t.param, w_type, at);
    load8(rg, t.grad, g_type, at);
    if constexpr (BITS == 32) {
        load8(rm, t.m, fp8rows::kF32, at);
        load8(rv, t.v, fp8rows::kF32, at);
    } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.m) + at));
        const uint2 c = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.v) + at));
        rm.w[0] = a.x; rm.w[1] = a.y;
        rv.w[0] = c.x; rv.w[1] = c.y;
        f.ms = __ldcg(t.m_scale + block);
        f.vs = __ldcg(t.v_scale + block);
    }
    float w[8], g[8], m[8], v[8];
    floats8(rw, w_type, w);
    floats8(rg, g_type, g);
    if constexpr (BITS == 32) {
        floats8(rm, fp8rows::kF32, m);
        floats8(rv, fp8rows::kF32, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = decode2(rm.w[i / 2] >> (16 * (i % 2))), y = decode2(rv.w[i / 2] >> (16 * (i % 2)));
            m[2 * i] = x.x;
            m[2 * i + 1] = x.y;
            v[2 * i] = y.x;
            v[2 * i + 1] = y.y;
        }
    }
    float r[8], most_m, most_v, least;
    uint32_t by_chance;
    update<BITS>(w, g, m, v, r, h, f, most_m, most_v, least, by_chance);
    if constexpr (MASTER)
        store8(t.master, fp8rows::kF32, at, w);
    store8(t.param, W32 && !MASTER ? fp8rows::kF32 : param_type, at, w);
    if constexpr (BITS == 32) {
        store8(t.m, fp8rows::kF32, at, m);
        store8(t.v, fp8rows::kF32, at, v);
    } else {
        Scale ms, vs;
        block_scales(most_m, most_v, lane, ms, vs);
        if (lane == 0) {
            t.m_scale[block] = ms.s;
            t.v_scale[block] = vs.s;
        }
        encode(m, r, ms, vs, least, static_cast<uint32_t>(at), 1, f.step, by_chance);
        uint32_t cm[4], cv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cm[i] = fp8q::cvt_pair(m[2 * i], m[2 * i + 1], 0);
            cv[i] = fp8q::cvt_pair(r[2 * i], r[2 * i + 1], 0);
        }
        __stcs(reinterpret_cast<uint2 *>(static_cast<uint8_t *>(t.m) + at), make_uint2(cm[0] | cm[1] << 16, cm[2] | cm[3] << 16));
        __stcs(reinterpret_cast<uint2 *>(static_cast<uint8_t *>(t.v) + at), make_uint2(cv[0] | cv[1] << 16, cv[2] | cv[3] << 16));
    }
}

// A tensor's last block, or one of a tensor without that alignment: single elements,
// every 32nd of the block a lane. What is behind the end counts as zeros.
template <int BITS>
__device__ __noinline__ void any_block(const Tensor &t, long long block, int param_type, int grad_type, bool master, const Hyper &h,
                                       Factors f, int lane)
{
    const long long at = block * kBlock + lane;
    const int n = static_cast<int>(min(8ll, (t.count - at + 31) / 32));    // (<= 0: none)
    float w[8], g[8], m[8], v[8], r[8];
    if constexpr (BITS == 8) {
        f.ms = __ldcg(t.m_scale + block);
        f.vs = __ldcg(t.v_scale + block);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long e = at + 32 * i;
        const bool in = i < n;
        w[i] = in ? (master ? t.master[e] : load1(t.param, param_type, e)) : 0.0f;
        g[i] = in ? load1(t.grad, grad_type, e) : 0.0f;
        m[i] = !in ? 0.0f : BITS == 32 ? static_cast<const float *>(t.m)[e] : decode1(static_cast<const uint8_t *>(t.m)[e]);
        v[i] = !in ? 0.0f : BITS == 32 ? static_cast<const float *>(t.v)[e] : decode1(static_cast<const uint8_t *>(t.v)[e]);
    }
    float most_m, most_v, least;
    uint32_t by_chance;
    update<BITS>(w, g, m, v, r, h, f, most_m, most_v, least, by_chance);
    if constexpr (BITS == 8) {
        most_m = most_v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {               // (behind the end, 0 times a NaN scale)
                most_m = fp8mm::max_nan(most_m, fabsf(m[i]));
                most_v = fp8mm::max_nan(most_v, v[i]);
            }
        __syncwarp();
        Scale ms, vs;
        block_scales(most_m, most_v, lane, ms, vs);
        if (lane == 0) {
            t.m_scale[block] = ms.s;
            t.v_scale[block] = vs.s;
        }
        encode(m, r, ms, vs, least, static_cast<uint32_t>(at), 32, f.step, by_chance);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long e = at + 32 * i;
        if (i >= n)
            break;
        const float one[1] = {w[i]};
        if (master)
            t.master[e] = w[i];
        fp8rows::store_group<1>(t.param, param_type, e, one);
        if constexpr (BITS == 32) {
            static_cast<float *>(t.m)[e] = m[i];
            static_cast<float *>(t.v)[e] = v[i];
        } else {
            static_cast<uint8_t *>(t.m)[e] = static_cast<uint8_t>(fp8q::cvt_pair(m[i], 0.0f, 0));
            static_cast<uint8_t *>(t.v)[e] = static_cast<uint8_t>(fp8q::cvt_pair(r[i], 0.0f, 0));
        }
    }
}

template <int BITS, bool W32, bool MASTER, bool G32, int T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) adamw_kernel(const __grid_constant__ Params<T> p)
{
    __shared__ float shared_hyper[3];
    __shared__ uint32_t shared_step;
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    float keep = p.h.keep, step_size = p.h.step_size, root = p.h.root;
    uint32_t step = p.h.step;
    if (p.h.step_device || p.h.lr_device) {
        // (the same for every CTA; in double, as the host does it)
        if (threadIdx.x == 0) {
            double lr = p.h.lr, rest1 = p.h.rest1;
            shared_hyper[2] = root;
            shared_step = step;
            if (p.h.lr_device)
                lr = static_cast<double>(__ldcg(p.h.lr_device));
            if (p.h.step_device) {
                const long long t = __ldcg(reinterpret_cast<const long long *>(p.h.step_device));
                rest1 = 1.0 - pow(p.h.beta1, static_cast<double>(t));
                shared_hyper[2] = static_cast<float>(1.0 / sqrt(1.0 - pow(p.h.beta2, static_cast<double>(t))));
                shared_step = static_cast<uint32_t>(t);
            }
            shared_hyper[0] = static_cast<float>(1.0 - lr * p.h.weight_decay);
            shared_hyper[1] = static_cast<float>(lr / rest1);
        }
        __syncthreads();
        keep = shared_hyper[0];
        step_size = shared_hyper[1];
        root = shared_hyper[2];
        step = shared_step;
    }
    Factors f{keep, step_size, root, p.h.grad_scale ? __ldcg(p.h.grad_scale) : 1.0f, 0.0f, 0.0f, step,
              p.h.grad_scale != nullptr, p.h.stochastic != 0, p.h.eps >= 0x1p-60f && p.h.eps <= 0x1p59f && root <= 0x1p29f};
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    // With 8-bit states a block takes arithmetic for as long as its loads' wait, which its being
    // in L2 shortens from 2 us to a third (470 M elements 1430 to 1280 us). With 32-bit ones
    // memory is the bound (268 M 1260 us, with it 1268), with 16-bit weights and no fp32 ones the
    // instructions (268 M 717, 724).
    constexpr bool kAhead = BITS == 8 && W32;
    // (a warp's number that is known to be the same in its lanes: what follows from it is kept
    // and computed once a warp, 470 M 1441 to 1430 us, 268 M of 32 bits 1281 to 1260)
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    int k = 0;
    for (long long b = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp; b < p.blocks; b += warps) {
        if (k + 1 < p.tensors && b >= p.first[k + 1]) {
            // the last tensor that begins at b or before it, by halves: one after another, cold
            // lines of the table took longer than the blocks of 48 small tensors
            int end = p.tensors;
            for (++k; end - k > 1;) {
                const int middle = (k + end) / 2;
                if (b >= p.first[middle])
                    k = middle;
                else
                    end = middle;
            }
        }
        const Tensor &t = p.t[k];
        const long long block = b - p.first[k];
        if (kAhead && t.vec && (block + warps + 1) * kBlock <= t.count && lane == 0)
            fetch_block<BITS, W32, MASTER, G32>(t, block + warps);
        if (t.vec && (block + 1) * kBlock <= t.count)
            whole_block<BITS, W32, MASTER, G32>(t, block, p.param_type, p.grad_type, p.h, f, lane);
        else
            any_block<BITS>(t, block, p.param_type, p.grad_type, MASTER, p.h, f, lane);
    }
}

}  // namespace fp8adam
