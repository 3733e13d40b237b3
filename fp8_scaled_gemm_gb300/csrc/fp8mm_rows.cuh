// fp8mm_rows.cuh -- what the row kernels (layer norm, activation gradient)
// share: element groups, conversions, team reductions, and the sum of
// per-CTA column partials.
//
// Element types are the C ABI's output codes 0 bf16, 1 fp16, 2 fp32. Kernels
// are compiled per element size; bf16 and fp16 differ only in a uniform
// branch at the conversion.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8mm_act.cuh"
#include "sm103_ptx.cuh"

namespace fp8rows {

namespace ptx = fp8mm::ptx;

constexpr int kBF16 = 0, kF16 = 1, kF32 = 2;

// G consecutive elements of ES bytes as loaded: 16-byte words for G = 8
// (16-byte aligned), one word for a pair of 16-bit elements (G = 2, 4-byte
// aligned), one element for G = 1.
template <int ES, int G>
struct Raw {
    static_assert((ES == 2 || ES == 4) && (G == 8 || G == 1 || (G == 2 && ES == 2)), "element group");
    static constexpr int kWords = G == 1 ? 1 : G * ES / 4;
    uint32_t w[kWords];
};

template <int ES, int G>
__device__ __forceinline__ void load_raw(Raw<ES, G> &r, const void *base, long long elem)
{
    const uint8_t *p = static_cast<const uint8_t *>(base) + elem * ES;
    if constexpr (G == 1) {
        if constexpr (ES == 2) {
            asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=r"(r.w[0]) : "l"(p));   // zero-extends
        } else {
            asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
        }
    } else if constexpr (G == 2) {
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < Raw<ES, G>::kWords; i += 4)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3])
                         : "l"(p + i * 4));
    }
}

template <int ES, int G>
__device__ __forceinline__ void clear_raw(Raw<ES, G> &r)
{
#pragma unroll
    for (int i = 0; i < Raw<ES, G>::kWords; ++i)
        r.w[i] = 0;
}

__device__ __forceinline__ float half_bits(uint32_t h, bool f16)
{
    return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(h))) : __uint_as_float(h << 16);
}

template <int ES, int G>
__device__ __forceinline__ void to_float(const Raw<ES, G> &r, bool f16, float (&v)[G])
{
    if constexpr (ES == 4) {
#pragma unroll
        for (int i = 0; i < G; ++i)
            v[i] = __uint_as_float(r.w[i]);
    } else if constexpr (G == 1) {
        v[0] = half_bits(r.w[0], f16);
    } else if (f16) {
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type)
{
    if (type == kF16) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// G values to element `elem` of an array of `type`, one rounding.
template <int G>
__device__ __forceinline__ void store_group(void *base, int type, long long elem, const float (&v)[G])
{
    if constexpr (G == 1) {
        if (type == kF32)
            static_cast<float *>(base)[elem] = v[0];
        else
            static_cast<unsigned short *>(base)[elem] = static_cast<unsigned short>(pack2(v[0], 0.0f, type) & 0xFFFFu);
    } else if (type == kF32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + elem);
#pragma unroll
        for (int i = 0; i < G; i += 4)
            p[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        uint4 w;
        w.x = pack2(v[0], v[1], type);
        w.y = pack2(v[2], v[3], type);
        w.z = pack2(v[4], v[5], type);
        w.w = pack2(v[6], v[7], type);
        *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(base) + elem) = w;
    }
}

// G values of a parameter vector (weight, bias) of any type; `fill` without one.
template <int G>
__device__ __forceinline__ void load_param(const void *base, int type, long long elem, float fill, float (&v)[G])
{
    if (base == nullptr) {
#pragma unroll
        for (int i = 0; i < G; ++i)
            v[i] = fill;
    } else if (type == kF32) {
        if constexpr (G == 1) {
            v[0] = __ldg(static_cast<const float *>(base) + elem);
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
#pragma unroll
            for (int i = 0; i < G; i += 4) {
                const float4 x = __ldg(p + i / 4);
                v[i] = x.x;
                v[i + 1] = x.y;
                v[i + 2] = x.z;
                v[i + 3] = x.w;
            }
        }
    } else {
        Raw<2, G> r;
        if constexpr (G == 1) {
            r.w[0] = __ldg(static_cast<const unsigned short *>(base) + elem);
        } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(base) + elem));
            r.w[0] = x.x;
            r.w[1] = x.y;
            r.w[2] = x.z;
            r.w[3] = x.w;
        }
        to_float<2, G>(r, type == kF16, v);
    }
}

// Sums of NV values over a team of LANES x WARPS threads, the same value in
// every thread. `red`: one float per warp and value, of the whole CTA; the
// caller alternates between two such arrays from call to call, so one barrier
// per call is enough. Every thread of the CTA calls it.
template <int LANES, int WARPS, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float *red)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o, LANES);
    if constexpr (WARPS > 1) {
        const int warp = static_cast<int>(threadIdx.x) >> 5;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                red[warp * NV + i] = v[i];
        }
        __syncthreads();
        const int first = warp / WARPS * WARPS;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] += red[(first + w) * NV + i];
    }
}

// The largest value over a team; NaN if any is NaN.
template <int LANES, int WARPS>
__device__ __forceinline__ float team_max(float v, float *red)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        v = fp8mm::max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o, LANES));
    if constexpr (WARPS > 1) {
        const int warp = static_cast<int>(threadIdx.x) >> 5;
        if ((threadIdx.x & 31) == 0)
            red[warp] = v;
        __syncthreads();
        const int first = warp / WARPS * WARPS;
        v = red[first];
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            v = fp8mm::max_nan(v, red[first + w]);
    }
    return v;
}

// ------------------------------------------------- sums of column partials ---
// out_k[c] = sum over p < P of partial[(p * K + k) * C + c], k = blockIdx.y
// < K <= 2. One CTA per 32 columns: warp w adds partials w, w + 32, ..., then
// the 32 sums of a column are added over the lanes of one warp: the order
// depends on P only.

struct PartialSumParams {
    const float *partial;
    float *out0, *out1;
    long long C;
    int P, K;
};

constexpr int kSumThreads = 1024;

static __global__ void __launch_bounds__(kSumThreads) partial_sum_kernel(const PartialSumParams p)
{
    __shared__ float part[32][33];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < p.C) {
        const float *src = p.partial + (static_cast<long long>(warp) * p.K + k) * p.C + c;
        const long long step = 32ll * p.K * p.C;
#pragma unroll 8
        for (int i = warp; i < p.P; i += 32, src += step)
            s += __ldcg(src);
    }
    part[warp][lane] = s;
    __syncthreads();
    s = part[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const long long mine = static_cast<long long>(blockIdx.x) * 32 + warp;
    if (lane == 0 && mine < p.C)
        (k == 0 ? p.out0 : p.out1)[mine] = s;
}

}  // namespace fp8rows
