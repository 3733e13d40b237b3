// fp8mm_norm.cuh -- layer norm, forward and backward.
//
// Forward, per row of C elements (fp32 arithmetic):
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd gamma + beta
// and on request the row's fp8 codes, quantised from the unrounded y:
//   scale = max |y| / qmax,  q = fp8(y / scale)
// The variance is summed from the centred values, which the row's threads
// still hold in registers, so an offset of the row costs no precision.
//
// Backward, with xhat = (x - mean) rstd and w = dy gamma:
//   dx = rstd (w - sum w / C - xhat sum(w xhat) / C) [+ dres]
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
//
// Both are bound by HBM, if the instructions and the waits between a row's
// reductions are kept out of the way:
//  - A team of threads takes a row and goes on to other rows with the same
//    columns, E = 8 CH per thread, so that backward's column sums stay in
//    registers and the next row's loads are issued before the present row's
//    reductions. A team is 4 to 32 lanes of a warp, a CTA, or (wide rows) the
//    CTAs of a cluster, each with a slice of the columns, that exchange their
//    sums through distributed shared memory.
//  - E is as large as the registers allow: a reduction costs a warp about 30
//    instructions whatever E is (with E = 8, 43 instructions per element ran
//    the forward pass at 47 % of HBM; with 32 it is about 12).
//  - Arithmetic goes two columns at a time (f32x2).
//  - Every warp covers 32 E neighbouring columns, so a thread's addresses
//    differ by constants. Rows that start on 16 bytes take 16-byte loads of
//    8 elements; others single elements or, 16-bit ones of even width that
//    start on 4 bytes, pairs, neighbouring lanes neighbouring ones.
// Rows of more than 131072 columns (backward: of a cluster's eight CTAs) go
// through the long kernels, which read the row again from L2 for each pass.
#pragma once

#include "fp8mm_act.cuh"
#include "fp8mm_quant_convert.cuh"
#include "fp8mm_rows.cuh"

namespace fp8norm {

using namespace fp8rows;

// ------------------------------------------------------------------ teams ---

constexpr int kMaxCluster = 8;       // CTAs that share a row
constexpr int kStatusTimeout = 0x10b;

// Kinds of team: LANES 4 .. 32 lanes of a warp; kCta all threads of a CTA;
// kCluster all threads of a cluster's CTAs. (Several teams in a CTA, each
// with a named barrier, were slower: a barrier number that is not a constant
// makes a CTA hold all 16 of its barriers, so 4 CTAs fill an SM.)
constexpr int kCta = 0, kCluster = -1;

// A thread's columns: E = 8 CH of them from c0 on. G = 8: groups of 8
// neighbours, 8 x (lanes) apart; G = 2 and 1: pairs and single columns, lane by
// lane (pairs: an even number of columns). `left`
// columns lie between c0 and the end of the row (of the CTA's slice).
template <int G, int KIND, int CH>
struct Place {
    static constexpr int E = 8 * CH;
    static constexpr int kLanes = KIND > 0 ? KIND : 32;
    static constexpr int kStep = G * kLanes;   // between a thread's groups
    long long c0;
    int left;

    __device__ __forceinline__ Place(long long begin, long long end, int t)
    {
        c0 = begin + static_cast<long long>(t / kLanes) * (kLanes * E) + (t % kLanes) * G;
        left = static_cast<int>(max(0ll, min(end - c0, 1ll << 30)));
    }
    // whether the thread's group k (of E / G) lies inside
    __device__ __forceinline__ bool in(int k) const { return k * kStep < left; }
};

template <int ES, int G, int CH>
struct RawE {
    Raw<ES, G> r[8 * CH / G];
};

// The thread's elements of the row at `p` (its first element).
template <int ES, int G, int KIND, int CH>
__device__ __forceinline__ void load_e(RawE<ES, G, CH> &r, const uint8_t *p, const Place<G, KIND, CH> &pl)
{
    constexpr int N = 8 * CH / G;
    constexpr int step = Place<G, KIND, CH>::kStep;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (pl.in(k))
            load_raw<ES, G>(r.r[k], p, k * step);
        else
            clear_raw<ES, G>(r.r[k]);
    }
}

template <int ES, int G, int CH>
__device__ __forceinline__ void clear_e(RawE<ES, G, CH> &r)
{
#pragma unroll
    for (int k = 0; k < 8 * CH / G; ++k)
        clear_raw<ES, G>(r.r[k]);
}

// As fp32 pairs.
template <int ES, int G, int CH>
__device__ __forceinline__ void to_pairs(const RawE<ES, G, CH> &r, bool f16, uint64_t (&v)[4 * CH])
{
    if constexpr (ES == 2) {
        // one branch for all elements
        if (f16) {
#pragma unroll
            for (int i = 0; i < 4 * CH; ++i) {
                float lo, hi;
                if constexpr (G > 1) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.r[2 * i / G].w[i % (G / 2)]));
                    lo = f.x;
                    hi = f.y;
                } else {
                    lo = half_bits(r.r[2 * i].w[0], true);
                    hi = half_bits(r.r[2 * i + 1].w[0], true);
                }
                v[i] = ptx::f32x2(lo, hi);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * CH; ++i) {
                if constexpr (G > 1)
                    v[i] = ptx::f32x2(__uint_as_float(r.r[2 * i / G].w[i % (G / 2)] << 16),
                                      __uint_as_float(r.r[2 * i / G].w[i % (G / 2)] & 0xFFFF0000u));
                else
                    v[i] = ptx::f32x2(__uint_as_float(r.r[2 * i].w[0] << 16), __uint_as_float(r.r[2 * i + 1].w[0] << 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
            if constexpr (G == 8)
                v[i] = ptx::f32x2(__uint_as_float(r.r[i / 4].w[2 * (i % 4)]), __uint_as_float(r.r[i / 4].w[2 * (i % 4) + 1]));
            else
                v[i] = ptx::f32x2(__uint_as_float(r.r[2 * i].w[0]), __uint_as_float(r.r[2 * i + 1].w[0]));
        }
    }
}

// Pairs to memory in `type`, one rounding; p: the thread's first element.
template <int G, int KIND, int CH>
__device__ __forceinline__ void store_e(uint8_t *p, int type, const Place<G, KIND, CH> &pl, const uint64_t (&v)[4 * CH])
{
    constexpr int step = Place<G, KIND, CH>::kStep;
    if (type == kF32) {
        float *o = reinterpret_cast<float *>(p);
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
            if constexpr (G == 8) {
                if (i % 2 == 0 && pl.in(i / 4)) {
                    float a, b, c, d;
                    ptx::unpack_f32x2(v[i], a, b);
                    ptx::unpack_f32x2(v[i + 1], c, d);
                    *reinterpret_cast<float4 *>(o + (i / 4) * step + 2 * (i % 4)) = make_float4(a, b, c, d);
                }
            } else {
                float a, b;
                ptx::unpack_f32x2(v[i], a, b);
                if (pl.in(2 * i / G))
                    o[2 * i / G * step] = a;
                if (pl.in((2 * i + 1) / G))
                    o[(2 * i + 1) / G * step + (G == 2)] = b;
            }
        }
        return;
    }
    uint32_t w[4 * CH];
    if (type == kF16) {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i)
            w[i] = ptx::cvt_16x2<true>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i)
            w[i] = ptx::cvt_16x2<false>(v[i]);
    }
    unsigned short *o = reinterpret_cast<unsigned short *>(p);
    if constexpr (G == 8) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
            if (pl.in(k))
                *reinterpret_cast<uint4 *>(o + k * step) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else if constexpr (G == 2) {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i)
            if (pl.in(i))
                *reinterpret_cast<uint32_t *>(o + i * step) = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
            if (pl.in(2 * i))
                o[2 * i * step] = static_cast<unsigned short>(w[i] & 0xFFFFu);
            if (pl.in(2 * i + 1))
                o[(2 * i + 1) * step] = static_cast<unsigned short>(w[i] >> 16);
        }
    }
}

// The thread's parameters; `fill` without a vector, 0 outside the row.
template <int G, int KIND, int CH>
__device__ __forceinline__ void param_e(const void *base, int type, const Place<G, KIND, CH> &pl, float fill,
                                        uint64_t (&v)[4 * CH])
{
    constexpr int step = Place<G, KIND, CH>::kStep;
    if (base == nullptr) {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i)
            v[i] = ptx::f32x2(fill, fill);
    } else if (type == kF32) {
        const float *p = static_cast<const float *>(base) + pl.c0;
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
            if constexpr (G == 8) {
                if (i % 2 == 0) {
                    const float4 f = pl.in(i / 4) ? __ldg(reinterpret_cast<const float4 *>(p + (i / 4) * step + 2 * (i % 4)))
                                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[i] = ptx::f32x2(f.x, f.y);
                    v[i + 1] = ptx::f32x2(f.z, f.w);
                }
            } else {
                v[i] = ptx::f32x2(pl.in(2 * i / G) ? __ldg(p + 2 * i / G * step) : 0.0f,
                                  pl.in((2 * i + 1) / G) ? __ldg(p + (2 * i + 1) / G * step + (G == 2)) : 0.0f);
            }
        }
    } else {
        RawE<2, G, CH> r;
        load_e<2, G, KIND, CH>(r, static_cast<const uint8_t *>(base) + pl.c0 * 2, pl);
        to_pairs<2, G, CH>(r, type == kF16, v);
    }
}

// A thread's parameters in shared memory, fp32: float4 j of them at
// slots[j * threads], so that a warp's accesses are free of bank conflicts.
template <int CH>
__device__ __forceinline__ void keep_params(float4 *slots, int threads, const uint64_t (&v)[4 * CH])
{
#pragma unroll
    for (int j = 0; j < 2 * CH; ++j) {
        float4 f;
        ptx::unpack_f32x2(v[2 * j], f.x, f.y);
        ptx::unpack_f32x2(v[2 * j + 1], f.z, f.w);
        slots[j * threads] = f;
    }
}

// v with the columns outside the row set to 0.
template <int G, int KIND, int CH>
__device__ __forceinline__ void mask_e(uint64_t (&v)[4 * CH], const Place<G, KIND, CH> &pl)
{
#pragma unroll
    for (int i = 0; i < 4 * CH; ++i) {
        if constexpr (G > 1) {
            v[i] = pl.in(2 * i / G) ? v[i] : 0ull;
        } else {
            float a, b;
            ptx::unpack_f32x2(v[i], a, b);
            v[i] = ptx::f32x2(pl.in(2 * i) ? a : 0.0f, pl.in(2 * i + 1) ? b : 0.0f);
        }
    }
}

template <int N>
__device__ __forceinline__ float sum_pairs(const uint64_t (&v)[N])
{
    uint64_t s0 = v[0], s1 = v[1];
#pragma unroll
    for (int i = 2; i < N; i += 2) {
        s0 = ptx::add_f32x2(s0, v[i]);
        s1 = ptx::add_f32x2(s1, v[i + 1]);
    }
    s0 = ptx::add_f32x2(s0, s1);
    float lo, hi;
    ptx::unpack_f32x2(s0, lo, hi);
    return lo + hi;
}

// What bounds a wait: clocks, and the word that says that one ran out.
struct Limit {
    int *status;
    unsigned long long clocks;
};

struct Team {
    int T, warps;        // threads and warps of the team in this CTA
    int id;              // team within the CTA
    uint32_t rank, ctas; // place in the cluster
    uint32_t bar;        // kCluster: mbarriers of its exchanges, 8 bytes each
    Limit limit;
};

// Exchanges of a cluster's team: every warp's values go to all its CTAs, into
// the slot of the warp in their buffer `red`, and are counted there on mbarrier
// k. (A cluster barrier per exchange waits for the row's global stores as well:
// forward 4096 x 32768 bf16 with codes 290 us, then 194; backward 8192 x 8192
// fp32 268, now 177.)
template <int NV>
__device__ __forceinline__ void cluster_send(const float (&v)[NV], const Team &tm, float *red, int k)
{
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    const uint32_t bar = tm.bar + 8u * k;
    if (threadIdx.x == 0)
        ptx::mbar_arrive_expect_tx(bar, tm.ctas * tm.warps * NV * 4u);
    if (lane < static_cast<int>(tm.ctas)) {
        const uint32_t at = ptx::mapa_shared(ptx::smem_addr(red + (tm.rank * tm.warps + warp) * NV),
                                             static_cast<uint32_t>(lane)),
                       there = ptx::mapa_shared(bar, static_cast<uint32_t>(lane));
        if constexpr (NV == 2)
            ptx::st_async_f32x2(at, v[0], v[1], there);
        else
            ptx::st_async_f32(at, v[0], there);
    }
    __syncwarp();
}

// False when the wait ran out.
__device__ __forceinline__ bool cluster_wait(const Team &tm, int k, uint32_t parity)
{
    const uint32_t bar = tm.bar + 8u * k;
    bool here = ptx::mbar_try_wait_cluster(bar, parity);
    if (!here) {
        const unsigned long long t0 = static_cast<unsigned long long>(clock64());
        while (!(here = ptx::mbar_try_wait_cluster(bar, parity))) {
            if (static_cast<unsigned long long>(clock64()) - t0 > tm.limit.clocks) {
                atomicCAS(tm.limit.status, 0, kStatusTimeout);
                break;
            }
        }
    }
    return __all_sync(0xFFFFFFFFu, here);   // the warp stays together
}

// Both. An exchange's buffer is free for the one after next: a warp sends for
// the next one after it has read this one, and this CTA passes the next one
// with all warps' values.
template <int NV>
__device__ __forceinline__ bool cluster_exchange(const float (&v)[NV], const Team &tm, float *red, int k, uint32_t parity)
{
    cluster_send<NV>(v, tm, red, k);
    return cluster_wait(tm, k, parity);
}

// Words of one reduction's exchange buffer for NV values.
template <int KIND, int NV>
constexpr int kRedWords = KIND == kCluster ? kMaxCluster * 32 * NV : 32 * NV;

// Sums of NV values over the team, the same bits in every thread. The caller
// alternates between buffers so that two barriers lie between uses of one.
// (k, parity: cluster_exchange's; false when its wait ran out.)
template <int KIND, int NV>
__device__ __forceinline__ bool team_sum8(float (&v)[NV], const Team &tm, float *red, int k, uint32_t parity)
{
    constexpr int L = KIND > 0 ? KIND : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o, L);
    if constexpr (KIND <= 0) {
        const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
        int n = tm.warps;
        const float *mine = red;
        if constexpr (KIND == kCluster) {
            if (!cluster_exchange<NV>(v, tm, red, k, parity))
                return false;
            n *= static_cast<int>(tm.ctas);
        } else {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    red[warp * NV + i] = v[i];
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = 0.0f;
        for (int e = lane; e < n; e += 32)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] += mine[e * NV + i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    }
    return true;
}

// Largest of NV magnitudes over the team, on their bit patterns: unsigned
// order is the order of |v| with NaN above infinity.
template <int KIND, int NV>
__device__ __forceinline__ bool team_amax8(float (&v)[NV], const Team &tm, float *red, int k, uint32_t parity)
{
    uint32_t u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        u[i] = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    if constexpr (KIND > 0 && KIND < 32) {
#pragma unroll
        for (int o = KIND / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                u[i] = max(u[i], __shfl_xor_sync(0xFFFFFFFFu, u[i], o, KIND));
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            u[i] = __reduce_max_sync(0xFFFFFFFFu, u[i]);
    }
    if constexpr (KIND <= 0) {
        const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
        int n = tm.warps;
        const float *mine = red;
        if constexpr (KIND == kCluster) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] = __uint_as_float(u[i]);
            if (!cluster_exchange<NV>(v, tm, red, k, parity))
                return false;
            n *= static_cast<int>(tm.ctas);
        } else {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    red[warp * NV + i] = __uint_as_float(u[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            u[i] = 0;
        for (int e = lane; e < n; e += 32)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                u[i] = max(u[i], __float_as_uint(mine[e * NV + i]));
#pragma unroll
        for (int i = 0; i < NV; ++i)
            u[i] = __reduce_max_sync(0xFFFFFFFFu, u[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i] = __uint_as_float(u[i]);
    return true;
}

// The team this thread belongs to, and which of all teams it is. bars: room for
// a cluster's mbarriers.
template <int KIND, int BARS>
__device__ __forceinline__ Team this_team(int &t, long long &first, long long &stride, uint64_t *bars, const Limit &limit)
{
    Team tm{};
    if constexpr (KIND > 0) {
        tm.T = KIND;
        tm.warps = 1;
        const int per_cta = static_cast<int>(blockDim.x) / KIND;
        tm.id = static_cast<int>(threadIdx.x) / KIND;
        t = static_cast<int>(threadIdx.x) % KIND;
        first = static_cast<long long>(blockIdx.x) * per_cta + tm.id;
        stride = static_cast<long long>(gridDim.x) * per_cta;
    } else if constexpr (KIND == kCta) {
        tm.T = static_cast<int>(blockDim.x);
        tm.warps = tm.T >> 5;
        t = static_cast<int>(threadIdx.x);
        first = blockIdx.x;
        stride = gridDim.x;
    } else {
        tm.T = static_cast<int>(blockDim.x);
        tm.warps = tm.T >> 5;
        tm.rank = ptx::cluster_ctarank();
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(tm.ctas));
        t = static_cast<int>(threadIdx.x);
        first = blockIdx.x / tm.ctas;
        stride = gridDim.x / tm.ctas;
        tm.bar = ptx::smem_addr(bars);
        tm.limit = limit;
        if (t == 0) {
#pragma unroll
            for (int i = 0; i < BARS; ++i)
                ptx::mbar_init(tm.bar + 8 * i, 1);
            ptx::fence_mbar_init();
        }
        ptx::cluster_sync();             // no remote store before every CTA runs
    }
    return tm;
}

// ---------------------------------------------------------------- forward ---

struct NormParams {
    const void *x;
    long long ldx;
    int x_f16;                 // 16-bit x: fp16 (else bf16)
    const void *gamma, *beta;  // nullptr: 1 and 0
    int param_type;
    float eps;
    void *y;                   // nullptr: not wanted
    int y_type;
    long long ldy;
    float *mean, *rstd;        // nullptr: not wanted
    uint8_t *q;                // fp8 codes [R, C], or nullptr
    int q_type;
    float *q_scale;
    long long R, C;
    long long groups;          // long kernel: element groups per row
    long long slice_cols;      // kCluster: columns of each CTA
    Limit limit;               // kCluster
};

// The fp8 codes of G values of a row, C ABI semantics of fp8_quantize.
template <int G>
__device__ __forceinline__ void store_codes(uint8_t *dst, const fp8q::Divider &d, const float (&v)[G], int q_type)
{
    float z[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        z[i] = d.mode == 1 ? fp8q::div_fast(d, v[i]) : fp8q::div_slow(d, v[i]);
    if constexpr (G == 1) {
        *dst = static_cast<uint8_t>(fp8q::cvt_pair(z[0], 0.0f, q_type) & 0xFFu);
    } else {
        uint2 w;
        w.x = fp8q::cvt_pair(z[0], z[1], q_type) | (fp8q::cvt_pair(z[2], z[3], q_type) << 16);
        w.y = fp8q::cvt_pair(z[4], z[5], q_type) | (fp8q::cvt_pair(z[6], z[7], q_type) << 16);
        *reinterpret_cast<uint2 *>(dst) = w;
    }
}

// The codes of the thread's values, two from each pair by `code`.
template <int G, int KIND, int CH, typename Code>
__device__ __forceinline__ void put_codes(uint8_t *p, const Place<G, KIND, CH> &pl, const uint64_t (&v)[4 * CH],
                                          const Code &code)
{
    constexpr int step = Place<G, KIND, CH>::kStep;
    if constexpr (G == 8) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const uint2 w = make_uint2(code(v[4 * k]) | (code(v[4 * k + 1]) << 16),
                                       code(v[4 * k + 2]) | (code(v[4 * k + 3]) << 16));
            if (pl.in(k))
                *reinterpret_cast<uint2 *>(p + k * step) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i) {
            const uint32_t c = code(v[i]);
            if constexpr (G == 2) {
                if (pl.in(i))
                    *reinterpret_cast<unsigned short *>(p + i * step) = static_cast<unsigned short>(c);
            } else {
                if (pl.in(2 * i))
                    p[2 * i * step] = static_cast<uint8_t>(c & 0xFFu);
                if (pl.in(2 * i + 1))
                    p[(2 * i + 1) * step] = static_cast<uint8_t>(c >> 8);
            }
        }
    }
}

// The codes of the thread's values, those of fp8_quantize (a y of -0 may give +0).
// With a scale in the reciprocal's range the quotients come from the reciprocal in
// two parts: r, the nearest fp32 value to 1 / scale (rcp.approx and one step of
// Newton's iteration, which gave __frcp_rn's for every mantissa), and rl, what is
// left of 1 / scale, so that v r + v rl is rounded once but for 2^-46 of it. On a CPU
// every mantissa of the scale, with every value within 12 units of its product with
// every tie between two codes, gave the code of the correctly rounded quotient.
// (16384 x 8192 bf16: the reciprocal alone, which is on the wrong side of some
// ties, with a scale of one product 116 us; this 121, with all codes made before
// the first is stored 123, with div_fast's correction instead 127.)
template <int G, int KIND, int CH>
__device__ __forceinline__ void store_codes_e(uint8_t *p, const Place<G, KIND, CH> &pl, float scale,
                                              const uint64_t (&v)[4 * CH], int q_type)
{
    if (fp8q::in_reciprocal_range(scale)) {
        const float r0 = fp8mm::rcp_approx(scale), r = fmaf(fmaf(-scale, r0, 1.0f), r0, r0);
        const float e = fmaf(-scale, r, 1.0f), rl = fmaf(e, e, e) * r;
        const uint64_t r2 = ptx::f32x2(r, r), l2 = ptx::f32x2(rl, rl);
        auto quotient = [&](uint64_t x, float &lo, float &hi) {
            ptx::unpack_f32x2(ptx::fma_f32x2(x, r2, ptx::mul_f32x2(x, l2)), lo, hi);
        };
        // one branch for all
        if (q_type == 0)
            put_codes<G, KIND, CH>(p, pl, v, [&](uint64_t x) {
                float lo, hi;
                quotient(x, lo, hi);
                return fp8q::cvt_pair(lo, hi, 0);
            });
        else
            put_codes<G, KIND, CH>(p, pl, v, [&](uint64_t x) {
                float lo, hi;
                quotient(x, lo, hi);
                return fp8q::cvt_pair(lo, hi, 1);
            });
        return;
    }
    const fp8q::Divider d = fp8q::make_divider(scale);
    put_codes<G, KIND, CH>(p, pl, v, [&](uint64_t x) {
        float lo, hi;
        ptx::unpack_f32x2(x, lo, hi);
        return fp8q::cvt_pair(fp8q::div_slow(d, lo), fp8q::div_slow(d, hi), q_type);
    });
}

// One row per CTA at a time (KIND > 0: per team of lanes), 64 registers, and
// as many CTAs on an SM as make 1024 threads: they hide each other's barriers.
// 16 columns per thread. 16384 x 8192 bf16 with codes takes 121 us, 5.5 TB/s (83 %
// of a copy; 22 instructions per element, issue slots 62 % busy; 113 to 116 us and
// 20 before the codes were made of correctly rounded quotients, which the next
// figures are without). Measured there against 121 us of an earlier form: 8 columns 177; 32 columns and 768 threads
// 150; the next two rows in shared memory (cp.async) instead of the next one in
// registers 119 to 121; several rows' teams in one CTA 155; gamma and beta from
// global memory (L1) for every row 174 (they are kept in shared memory,
// keep_params); against 113: the warps' own means and differences joined in one
// exchange instead of two 116. Rows of 16-bit elements without 16-byte groups:
// 16384 x 4998 bf16 in pairs 90 us (68 %; single elements 121), 16384 x 4999 in
// single elements (34 instructions each) 123 us (50 %), against 80 at 5000
// columns. For odd widths, pairs with single elements at the edges took 134 to
// 158, accesses without bounds tests in all but the last warp 118 (35 instead
// of 26 at 1001 columns).
template <int ES, int G, int KIND, int CH>
__global__ void __launch_bounds__(KIND > 0 ? 256 : 1024, KIND > 0 ? (CH == 4 ? 3 : 4) : 1)
    norm_kernel(const NormParams p)
{
    __shared__ float red[3][kRedWords<KIND, 1>];
    __shared__ uint64_t bars[3];
    extern __shared__ float4 params[];
    ptx::grid_launch_dependents();
    int t;
    long long first, stride;
    const Team tm = this_team<KIND, 3>(t, first, stride, bars, p.limit);
    long long begin = 0, end = p.C;
    if constexpr (KIND == kCluster) {
        begin = min(p.C, tm.rank * p.slice_cols);
        end = min(p.C, begin + p.slice_cols);
    }
    const Place<G, KIND, CH> pl(begin, end, t);
    const bool speaks = t == 0 && (KIND != kCluster || tm.rank == 0);   // for the team
    float4 *const my_gamma = params + t, *const my_beta = my_gamma + 2 * CH * tm.T;
    ptx::grid_dependency_wait();

    const float inv_c = 1.0f / static_cast<float>(p.C);
    const uint8_t *x = static_cast<const uint8_t *>(p.x) + (first * p.ldx + pl.c0) * ES;
    const long long x_step = stride * p.ldx * ES;
    RawE<ES, G, CH> raw;
    clear_e<ES, G, CH>(raw);
    if (first < p.R)
        load_e<ES, G, KIND, CH>(raw, x, pl);
    if (tm.id == 0) {
        uint64_t v[4 * CH];
        param_e<G, KIND, CH>(p.gamma, p.param_type, pl, 1.0f, v);
        keep_params<CH>(my_gamma, tm.T, v);
        param_e<G, KIND, CH>(p.beta, p.param_type, pl, 0.0f, v);
        keep_params<CH>(my_beta, tm.T, v);
    }
    if constexpr (KIND > 0)
        __syncthreads();                 // several teams read the first one's copy

    // every thread of a CTA makes the same number of turns
    const long long first0 = KIND > 0 ? first - tm.id : first;
    for (long long turn = 0; first0 + turn * stride < p.R; ++turn) {
        const long long row = first + turn * stride;
        const uint32_t parity = static_cast<uint32_t>(turn) & 1u;
        uint64_t v[4 * CH];
        to_pairs<ES, G, CH>(raw, p.x_f16, v);
        x += x_step;
        if (row + stride < p.R)
            load_e<ES, G, KIND, CH>(raw, x, pl);
        float s[1] = {sum_pairs(v)};
        if (!team_sum8<KIND, 1>(s, tm, red[0], 0, parity))
            break;                       // the results are void
        const float mean = s[0] * inv_c;
        const uint64_t m2 = ptx::f32x2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < 4 * CH; ++i)
            v[i] = ptx::add_f32x2(v[i], m2);
        if (!pl.in(8 * CH / G - 1))
            mask_e<G, KIND, CH>(v, pl);
        uint64_t q0 = 0, q1 = 0;
#pragma unroll
        for (int i = 0; i < 4 * CH; i += 2) {
            q0 = ptx::fma_f32x2(v[i], v[i], q0);
            q1 = ptx::fma_f32x2(v[i + 1], v[i + 1], q1);
        }
        const uint64_t q2[2] = {q0, q1};
        s[0] = sum_pairs(q2);
        if (!team_sum8<KIND, 1>(s, tm, red[1], 1, parity))
            break;
        const float rstd = rsqrtf(fmaf(s[0], inv_c, p.eps));
        const uint64_t r2 = ptx::f32x2(rstd, rstd);
#pragma unroll
        for (int j = 0; j < 2 * CH; ++j) {
            const float4 ga = my_gamma[j * tm.T], be = my_beta[j * tm.T];
            v[2 * j] = ptx::fma_f32x2(ptx::mul_f32x2(v[2 * j], r2), ptx::f32x2(ga.x, ga.y), ptx::f32x2(be.x, be.y));
            v[2 * j + 1] =
                ptx::fma_f32x2(ptx::mul_f32x2(v[2 * j + 1], r2), ptx::f32x2(ga.z, ga.w), ptx::f32x2(be.z, be.w));
        }
        const bool valid = row < p.R;
        if (valid) {
            if (speaks) {
                if (p.mean)
                    p.mean[row] = mean;
                if (p.rstd)
                    p.rstd[row] = rstd;
            }
            if (p.y)
                store_e<G, KIND, CH>(static_cast<uint8_t *>(p.y) + (row * p.ldy + pl.c0) * (p.y_type == kF32 ? 4 : 2),
                                     p.y_type, pl, v);
        }
        if (p.q) {
            float amax[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < 4 * CH; ++i) {
                float a, b;
                ptx::unpack_f32x2(v[i], a, b);
                amax[0] = fp8mm::max_nan(amax[0], fabsf(a));
                amax[0] = fp8mm::max_nan(amax[0], fabsf(b));
            }
            if (!team_amax8<KIND, 1>(amax, tm, red[2], 2, parity))
                break;
            const float scale = fp8q::row_scale(amax[0], p.q_type);
            if (valid) {
                if (speaks)
                    p.q_scale[row] = scale;
                store_codes_e<G, KIND, CH>(p.q + row * p.C + pl.c0, pl, scale, v, p.q_type);
            }
        }
    }
    if constexpr (KIND == kCluster)
        ptx::cluster_sync();             // no CTA leaves while a peer's stores may reach it
}

// Rows of any length: one CTA per row, one pass over the row per quantity.
constexpr int kLongThreads = 1024;

template <int ES, int G>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const NormParams p)
{
    __shared__ float red[3][32];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float c_f = static_cast<float>(p.C);
    for (long long row = blockIdx.x; row < p.R; row += gridDim.x) {
        float s[1] = {0.0f};
        for (long long g = threadIdx.x; g < p.groups; g += kLongThreads) {
            Raw<ES, G> raw;
            load_raw<ES, G>(raw, p.x, row * p.ldx + g * G);
            float v[G];
            to_float<ES, G>(raw, p.x_f16, v);
#pragma unroll
            for (int i = 0; i < G; ++i)
                s[0] += v[i];
        }
        team_sum<32, 32, 1>(s, red[0]);
        const float mean = s[0] / c_f;
        s[0] = 0.0f;
        for (long long g = threadIdx.x; g < p.groups; g += kLongThreads) {
            Raw<ES, G> raw;
            load_raw<ES, G>(raw, p.x, row * p.ldx + g * G);
            float v[G];
            to_float<ES, G>(raw, p.x_f16, v);
#pragma unroll
            for (int i = 0; i < G; ++i)
                s[0] = fmaf(v[i] - mean, v[i] - mean, s[0]);
        }
        team_sum<32, 32, 1>(s, red[1]);
        const float rstd = 1.0f / sqrtf(s[0] / c_f + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
        float amax = 0.0f;
        fp8q::Divider d{};
        // first y and its maximum, then (with q) the codes of the same values
        for (int pass = 0; pass < (p.q ? 2 : 1); ++pass) {
            for (long long g = threadIdx.x; g < p.groups; g += kLongThreads) {
                Raw<ES, G> raw;
                load_raw<ES, G>(raw, p.x, row * p.ldx + g * G);
                float v[G], ga[G], be[G];
                to_float<ES, G>(raw, p.x_f16, v);
                load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
                load_param<G>(p.beta, p.param_type, g * G, 0.0f, be);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    v[i] = fmaf((v[i] - mean) * rstd, ga[i], be[i]);
                    amax = fp8mm::max_nan(amax, fabsf(v[i]));
                }
                if (pass == 1)
                    store_codes<G>(p.q + row * p.C + g * G, d, v, p.q_type);
                else if (p.y)
                    store_group<G>(p.y, p.y_type, row * p.ldy + g * G, v);
            }
            if (pass == 0 && p.q) {
                amax = team_max<32, 32>(amax, red[2]);
                const float scale = __fdiv_rn(amax, fp8q::qmax_of(p.q_type));
                if (threadIdx.x == 0)
                    p.q_scale[row] = scale;
                d = fp8q::make_divider(scale);
            }
        }
    }
}

// ------------------------------------------------------------- backward ---

struct NormGradParams {
    const void *dy, *x;
    long long lddy, ldx;
    int dy_f16, x_f16;
    const void *gamma;
    int param_type;
    const float *mean, *rstd;
    const void *dres;          // added to dx, or nullptr
    long long lddres;
    void *dx;                  // nullptr: not wanted
    long long lddx;
    int x_type;
    float *partial, *partial1; // dgamma and dbeta sums of CTA's or cluster's i rows at [i * partial_step], or nullptr
    long long partial_step;    // (a single one: the results themselves)
    long long R, C;
    long long groups;          // long kernels: element groups per row
    long long slice_cols;      // kCluster: columns of each CTA
    Limit limit;               // kCluster
};

// Columns per thread over 8 (CH) and threads of a CTA: two 16-bit operands in
// 16-byte groups leave room for 16 columns.
constexpr int kGradThreads = 512;
template <int ES, int DES, int G, int KIND>
constexpr int kGradCh = (ES == 2 && DES == 2 && G > 1 && KIND <= 0) ? 2 : 1;

// Each thread keeps the dgamma and dbeta sums of its columns in registers over
// all its rows; teams of lanes then add theirs in order through shared memory.
// 16384 x 8192 bf16 with a residual gradient takes 177 us, 6.1 TB/s (91 % of a
// copy), 8192 x 8192 fp32 178 (91 %). Registers (128 per thread) hold one row at
// work, one on its way and the sums, so an SM has 512 threads and wide rows one
// or two teams: 8192 x 16384 bf16 runs at 70 %, 4096 x 32768 at 41 %, waiting for
// exchanges. In pairs 16384 x 4094 takes 116 us (70 %), 12782 x 10500 361 (45 %;
// single elements 728). Single elements leave registers for 8 columns per thread
// (16384 x 4095 bf16 135 us, 60 %; over 4096 columns, in clusters, 19 to 39 %).
// Teams of lanes: CTAs of 256 threads, 4 on an SM (3 where registers hold fp32 rows).
constexpr int kGradLaneThreads = 256;
template <int ES, int DES>
constexpr int kGradLaneCtas = ES == 2 && DES == 2 ? 4 : 3;

// The team's column sums to its slot of the partial sums (cols: shared memory
// of kGradLaneThreads x 8 floats).
template <int G, int KIND, int CH>
__device__ __forceinline__ void store_column_sums(const NormGradParams &p, long long slot, int t,
                                                  const Place<G, KIND, CH> &pl, const uint64_t (&dga)[4 * CH],
                                                  const uint64_t (&dbe)[4 * CH], float *cols)
{
    constexpr int P = 4 * CH;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float f[2 * P];
#pragma unroll
        for (int i = 0; i < P; ++i)
            ptx::unpack_f32x2(k == 0 ? dga[i] : dbe[i], f[2 * i], f[2 * i + 1]);
        if constexpr (KIND > 0 && KIND < 32) {
            // teams of one warp first
#pragma unroll
            for (int o = KIND; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 2 * P; ++i)
                    f[i] += __shfl_xor_sync(0xFFFFFFFFu, f[i], o);
        }
        bool writes = true;
        if constexpr (KIND > 0) {
            // then the warps in order
            const int warps = static_cast<int>(blockDim.x) / 32, warp = static_cast<int>(threadIdx.x) >> 5;
            const bool speaks = static_cast<int>(threadIdx.x & 31) < KIND;
            writes = speaks && warp == warps - 1;
            for (int m = 0; m + 1 < warps; ++m) {
                __syncthreads();
                if (warp == m && speaks) {
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) {
                        const int at = i * KIND + t;
                        cols[at] = m == 0 ? f[i] : cols[at] + f[i];
                    }
                }
            }
            __syncthreads();
            if (writes && warps > 1) {
#pragma unroll
                for (int i = 0; i < 2 * P; ++i)
                    f[i] += cols[i * KIND + t];
            }
        }
        if (writes) {
            uint64_t v[P];
#pragma unroll
            for (int i = 0; i < P; ++i)
                v[i] = ptx::f32x2(f[2 * i], f[2 * i + 1]);
            store_e<G, KIND, CH>(
                reinterpret_cast<uint8_t *>((k == 0 ? p.partial : p.partial1) + slot * p.partial_step + pl.c0), kF32, pl,
                v);
        }
        __syncthreads();
    }
}

// Whether a thread has several groups of columns: some can lie in the row and others not.
template <int G, int CH>
constexpr bool kMixed = 8 * CH / G > 1;

// A row's terms of the column sums, and its two sums: s1 of w = dy gamma, s2 of
// w xhat. h: x, then xhat; w: dy, then w. m2, r2: -mean and rstd twice. Outside
// the row w is 0, but xhat would be -mean rstd, which can leave fp32's range and
// make w xhat NaN. So a thread of one group takes 0 for both outside the row
// (the callers see to it), and one of several sets xhat to 0 there (1 to 3 % of
// those kernels).
template <int G, int KIND, int CH>
__device__ __forceinline__ void grad_terms(uint64_t (&h)[4 * CH], uint64_t (&w)[4 * CH], uint64_t m2, uint64_t r2,
                                           const float4 *my_gamma, int threads, const Place<G, KIND, CH> &pl,
                                           uint64_t (&dga)[4 * CH], uint64_t (&dbe)[4 * CH], float (&s)[2])
{
    constexpr int P = 4 * CH;
    uint64_t s1 = 0, s2 = 0;
    if constexpr (kMixed<G, CH>) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            h[i] = ptx::mul_f32x2(ptx::add_f32x2(h[i], m2), r2);
        if (!pl.in(8 * CH / G - 1))
            mask_e<G, KIND, CH>(h, pl);
    }
#pragma unroll
    for (int j = 0; j < P / 2; ++j) {
        const float4 g4 = my_gamma[j * threads];
#pragma unroll
        for (int i = 2 * j; i < 2 * j + 2; ++i) {
            if constexpr (!kMixed<G, CH>)
                h[i] = ptx::mul_f32x2(ptx::add_f32x2(h[i], m2), r2);
            dga[i] = ptx::fma_f32x2(w[i], h[i], dga[i]);
            dbe[i] = ptx::add_f32x2(dbe[i], w[i]);
            w[i] = ptx::mul_f32x2(w[i], i == 2 * j ? ptx::f32x2(g4.x, g4.y) : ptx::f32x2(g4.z, g4.w));
            s1 = ptx::add_f32x2(s1, w[i]);
            s2 = ptx::fma_f32x2(w[i], h[i], s2);
        }
    }
    float lo, hi;
    ptx::unpack_f32x2(s1, lo, hi);
    s[0] = lo + hi;
    ptx::unpack_f32x2(s2, lo, hi);
    s[1] = lo + hi;
}

template <int ES, int DES, int G, int KIND, int CH>
__global__ void __launch_bounds__(KIND > 0 ? kGradLaneThreads : kGradThreads, KIND > 0 ? kGradLaneCtas<ES, DES> : 1)
    norm_grad_kernel(const NormGradParams p)
{
    constexpr int P = 4 * CH;
    __shared__ __align__(8) float red[2][kRedWords<KIND, 2>];
    __shared__ uint64_t bars[2];
    // gamma (keep_params: 2 CH float4s per thread); after the rows, the teams' sums meet here
    extern __shared__ float4 params[];
    float *const cols = reinterpret_cast<float *>(params);
    ptx::grid_launch_dependents();
    int t;
    long long first, stride, begin = 0, end = p.C;
    const Team tm = this_team<KIND, 2>(t, first, stride, bars, p.limit);
    if constexpr (KIND == kCluster) {
        begin = min(p.C, tm.rank * p.slice_cols);
        end = min(p.C, begin + p.slice_cols);
    }
    const Place<G, KIND, CH> pl(begin, end, t);
    ptx::grid_dependency_wait();

    const float inv_c = 1.0f / static_cast<float>(p.C);
    const uint8_t *px = static_cast<const uint8_t *>(p.x) + (first * p.ldx + pl.c0) * ES;
    const uint8_t *pd = static_cast<const uint8_t *>(p.dy) + (first * p.lddy + pl.c0) * DES;
    const uint8_t *pr = static_cast<const uint8_t *>(p.dres) + (first * p.lddres + pl.c0) * ES;
    uint8_t *po = static_cast<uint8_t *>(p.dx) + (first * p.lddx + pl.c0) * ES;
    const long long x_step = stride * p.ldx * ES, d_step = stride * p.lddy * DES, r_step = stride * p.lddres * ES,
                    o_step = stride * p.lddx * ES;
    RawE<ES, G, CH> nx;
    RawE<DES, G, CH> nd;
    clear_e<ES, G, CH>(nx);
    clear_e<DES, G, CH>(nd);
    float nmean = 0.0f, nrstd = 0.0f;
    if (first < p.R) {
        load_e<ES, G, KIND, CH>(nx, px, pl);
        load_e<DES, G, KIND, CH>(nd, pd, pl);
        if (kMixed<G, CH> || pl.in(0)) {
            nmean = __ldg(p.mean + first);
            nrstd = __ldg(p.rstd + first);
        }
    }
    uint64_t dga[P] = {}, dbe[P] = {};
    const int threads = static_cast<int>(blockDim.x);
    float4 *const my_gamma = params + threadIdx.x;
    {
        uint64_t ga[P];
        param_e<G, KIND, CH>(p.gamma, p.param_type, pl, 1.0f, ga);
        keep_params<CH>(my_gamma, threads, ga);
    }

    int flip = 0;
    const long long first0 = KIND > 0 ? first - tm.id : first;
    for (long long turn = 0; first0 + turn * stride < p.R; ++turn) {
        const long long row = first + turn * stride;
        const bool valid = row < p.R;
        RawE<ES, G, CH> rr;
        if (valid && p.dres)
            load_e<ES, G, KIND, CH>(rr, pr, pl);
        else
            clear_e<ES, G, CH>(rr);
        const float mean = nmean, rstd = nrstd;
        const uint64_t m2 = ptx::f32x2(-mean, -mean), r2 = ptx::f32x2(rstd, rstd);
        uint64_t h[P], w[P];
        to_pairs<ES, G, CH>(nx, p.x_f16, h);
        to_pairs<DES, G, CH>(nd, p.dy_f16, w);
        px += x_step;
        pd += d_step;
        if (row + stride < p.R) {
            load_e<ES, G, KIND, CH>(nx, px, pl);
            load_e<DES, G, KIND, CH>(nd, pd, pl);
            if (kMixed<G, CH> || pl.in(0)) {
                nmean = __ldg(p.mean + row + stride);
                nrstd = __ldg(p.rstd + row + stride);
            }
        }
        float s[2] = {0.0f, 0.0f};
        if (valid)
            grad_terms<G, KIND, CH>(h, w, m2, r2, my_gamma, threads, pl, dga, dbe, s);
        if (p.dx == nullptr)
            continue;                    // parameter sums only
        if (!team_sum8<KIND, 2>(s, tm, red[flip], flip, static_cast<uint32_t>(turn >> 1) & 1u))
            break;                       // the results are void
        flip ^= 1;
        const float a = -s[0] * inv_c, b = -s[1] * inv_c;
        const uint64_t a2 = ptx::f32x2(a, a), b2 = ptx::f32x2(b, b);
        if (valid) {
            uint64_t r[P];
            to_pairs<ES, G, CH>(rr, p.x_f16, r);
#pragma unroll
            for (int i = 0; i < P; ++i)
                w[i] = ptx::fma_f32x2(ptx::fma_f32x2(h[i], b2, ptx::add_f32x2(w[i], a2)), r2, r[i]);
            store_e<G, KIND, CH>(po, p.x_type, pl, w);
        }
        pr += r_step;
        po += o_step;
    }
    if (p.partial != nullptr)
        store_column_sums<G, KIND, CH>(p, KIND == kCluster ? blockIdx.x / tm.ctas : blockIdx.x, t, pl, dga, dbe, cols);
    if constexpr (KIND == kCluster)
        ptx::cluster_sync();             // no CTA leaves while a peer's stores may reach it
}

// The same for a cluster's CTAs and 16-byte groups of 16-bit elements: a row's
// sums are sent before the row before it is finished, so that an exchange has a
// row's work to hide behind; until then the row is kept as loaded, and it is
// converted twice. bf16 with a residual gradient, norm_grad_kernel and this one:
// 8192 x 16384 250 and 221 us (228 since columns past the row's end are left out of
// its sums), 12000 x 12288 324 and 278 (287), 4096 x 32768 441 and 383 (388).
// Other operands lost with it (16384 x 9132 unaligned 653 and 762, 4096 x 16384
// fp32 284 and 303: 8 columns per thread leave less work to hide behind, and more
// of the second conversion's). Four buffers: a warp sends for row n after it has
// passed row n - 2's exchange, and every warp sent for that after it had read row
// n - 4's.
template <int ES, int DES, int G, int CH>
__global__ void __launch_bounds__(kGradThreads) norm_grad_cluster_kernel(const NormGradParams p)
{
    constexpr int P = 4 * CH, KIND = kCluster;
    __shared__ __align__(8) float red[4][kMaxCluster * (kGradThreads / 32) * 2];
    __shared__ uint64_t bars[4];
    extern __shared__ float4 params[];           // gamma (keep_params: 2 CH float4s per thread)
    ptx::grid_launch_dependents();
    int t;
    long long row, stride;
    const Team tm = this_team<KIND, 4>(t, row, stride, bars, p.limit);
    const long long begin = min(p.C, tm.rank * p.slice_cols), end = min(p.C, begin + p.slice_cols);
    const Place<G, KIND, CH> pl(begin, end, t);
    ptx::grid_dependency_wait();

    const float inv_c = 1.0f / static_cast<float>(p.C);
    const uint8_t *px = static_cast<const uint8_t *>(p.x) + (row * p.ldx + pl.c0) * ES;
    const uint8_t *pd = static_cast<const uint8_t *>(p.dy) + (row * p.lddy + pl.c0) * DES;
    const uint8_t *pr = static_cast<const uint8_t *>(p.dres) + (row * p.lddres + pl.c0) * ES;
    uint8_t *po = static_cast<uint8_t *>(p.dx) + (row * p.lddx + pl.c0) * ES;
    RawE<ES, G, CH> lx, cx;                      // on its way; sent for, to be finished
    RawE<DES, G, CH> ld, cd;
    float lmean = 0.0f, lrstd = 0.0f, cmean = 0.0f, crstd = 0.0f;
    clear_e<ES, G, CH>(lx);
    clear_e<DES, G, CH>(ld);
    auto load = [&](long long r) {
        load_e<ES, G, KIND, CH>(lx, px, pl);
        load_e<DES, G, KIND, CH>(ld, pd, pl);
        lmean = __ldg(p.mean + r);
        lrstd = __ldg(p.rstd + r);
        px += stride * p.ldx * ES;
        pd += stride * p.lddy * DES;
    };
    if (row < p.R)
        load(row);
    uint64_t dga[P] = {}, dbe[P] = {};
    const int threads = static_cast<int>(blockDim.x);
    float4 *const my_gamma = params + threadIdx.x;
    {
        uint64_t ga[P];
        param_e<G, KIND, CH>(p.gamma, p.param_type, pl, 1.0f, ga);
        keep_params<CH>(my_gamma, threads, ga);
    }
    // turn n sends row n's sums, then finishes row n - 1
    const bool dx = p.dx != nullptr;
    bool sent = false;
    for (uint32_t n = 0; sent || row < p.R; ++n) {
        RawE<ES, G, CH> nx = lx;
        RawE<DES, G, CH> nd = ld;
        const float nmean = lmean, nrstd = lrstd;
        const bool more = row < p.R;
        if (more) {
            if (row + stride < p.R)
                load(row + stride);
            uint64_t h[P], w[P];
            float s[2];
            to_pairs<ES, G, CH>(nx, p.x_f16, h);
            to_pairs<DES, G, CH>(nd, p.dy_f16, w);
            grad_terms<G, KIND, CH>(h, w, ptx::f32x2(-nmean, -nmean), ptx::f32x2(nrstd, nrstd), my_gamma, threads, pl, dga,
                                    dbe, s);
            row += stride;
            if (dx) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
                    s[1] += __shfl_xor_sync(0xFFFFFFFFu, s[1], o);
                }
                cluster_send<2>(s, tm, red[n & 3], static_cast<int>(n & 3));
            }
        }
        if (sent) {
            RawE<ES, G, CH> rr;
            if (p.dres)
                load_e<ES, G, KIND, CH>(rr, pr, pl);
            else
                clear_e<ES, G, CH>(rr);
            const uint32_t k = (n - 1) & 3;
            if (!cluster_wait(tm, static_cast<int>(k), ((n - 1) >> 2) & 1u))
                break;                           // the results are void
            float s[2] = {0.0f, 0.0f};
            for (int e = static_cast<int>(threadIdx.x) & 31; e < static_cast<int>(tm.ctas) * tm.warps; e += 32) {
                s[0] += red[k][2 * e];
                s[1] += red[k][2 * e + 1];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
                s[1] += __shfl_xor_sync(0xFFFFFFFFu, s[1], o);
            }
            const float a = -s[0] * inv_c, b = -s[1] * inv_c;
            const uint64_t a2 = ptx::f32x2(a, a), b2 = ptx::f32x2(b, b), m2 = ptx::f32x2(-cmean, -cmean),
                           r2 = ptx::f32x2(crstd, crstd);
            uint64_t h[P], w[P], r[P];
            to_pairs<ES, G, CH>(cx, p.x_f16, h);
            to_pairs<DES, G, CH>(cd, p.dy_f16, w);
            to_pairs<ES, G, CH>(rr, p.x_f16, r);
#pragma unroll
            for (int j = 0; j < P / 2; ++j) {
                const float4 g4 = my_gamma[j * threads];
#pragma unroll
                for (int i = 2 * j; i < 2 * j + 2; ++i) {
                    h[i] = ptx::mul_f32x2(ptx::add_f32x2(h[i], m2), r2);
                    w[i] = ptx::fma_f32x2(w[i], i == 2 * j ? ptx::f32x2(g4.x, g4.y) : ptx::f32x2(g4.z, g4.w), a2);
                    w[i] = ptx::fma_f32x2(ptx::fma_f32x2(h[i], b2, w[i]), r2, r[i]);
                }
            }
            store_e<G, KIND, CH>(po, p.x_type, pl, w);
            pr += stride * p.lddres * ES;
            po += stride * p.lddx * ES;
        }
        cx = nx;
        cd = nd;
        cmean = nmean;
        crstd = nrstd;
        sent = more && dx;
    }
    if (p.partial != nullptr)
        store_column_sums<G, KIND, CH>(p, blockIdx.x / tm.ctas, t, pl, dga, dbe, nullptr);
    ptx::cluster_sync();                 // no CTA leaves while a peer's stores may reach it
}

// Rows of any length: dx by one CTA per row. The parameter sums come from
// norm_grad_cols_kernel.
template <int ES, int DES, int G>
__global__ void __launch_bounds__(kLongThreads) norm_grad_long_kernel(const NormGradParams p)
{
    __shared__ float red[2][64];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float inv_c = 1.0f / static_cast<float>(p.C);
    int flip = 0;
    for (long long row = blockIdx.x; row < p.R; row += gridDim.x) {
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float s[2] = {0.0f, 0.0f};
        for (long long g = threadIdx.x; g < p.groups; g += kLongThreads) {
            Raw<ES, G> rx;
            Raw<DES, G> rd;
            load_raw<ES, G>(rx, p.x, row * p.ldx + g * G);
            load_raw<DES, G>(rd, p.dy, row * p.lddy + g * G);
            float x[G], d[G], ga[G];
            to_float<ES, G>(rx, p.x_f16, x);
            to_float<DES, G>(rd, p.dy_f16, d);
            load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float w = d[i] * ga[i];
                s[0] += w;
                s[1] = fmaf(w, (x[i] - mean) * rstd, s[1]);
            }
        }
        team_sum<32, 32, 2>(s, red[flip]);
        flip ^= 1;
        const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
        for (long long g = threadIdx.x; g < p.groups; g += kLongThreads) {
            Raw<ES, G> rx;
            Raw<DES, G> rd;
            load_raw<ES, G>(rx, p.x, row * p.ldx + g * G);
            load_raw<DES, G>(rd, p.dy, row * p.lddy + g * G);
            float x[G], d[G], ga[G], o[G];
            to_float<ES, G>(rx, p.x_f16, x);
            to_float<DES, G>(rd, p.dy_f16, d);
            load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
#pragma unroll
            for (int i = 0; i < G; ++i)
                o[i] = rstd * (fmaf(-(x[i] - mean) * rstd, m2, d[i] * ga[i]) - m1);
            if (p.dres) {
                Raw<ES, G> rr;
                load_raw<ES, G>(rr, p.dres, row * p.lddres + g * G);
                float r[G];
                to_float<ES, G>(rr, p.x_f16, r);
#pragma unroll
                for (int i = 0; i < G; ++i)
                    o[i] += r[i];
            }
            store_group<G>(p.dx, p.x_type, row * p.lddx + g * G, o);
        }
    }
}

// The parameter sums of long rows: each CTA takes 256 G columns and the rows
// of its slab (blockIdx.y), thread t the columns G t .. G t + G - 1 of them.
template <int ES, int DES, int G>
__global__ void __launch_bounds__(256) norm_grad_cols_kernel(const NormGradParams p)
{
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const long long g = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (g >= p.groups)
        return;
    const long long slabs = gridDim.y, r0 = p.R * blockIdx.y / slabs, r1 = p.R * (blockIdx.y + 1) / slabs;
    float dga[G] = {}, dbe[G] = {};
#pragma unroll 4
    for (long long row = r0; row < r1; ++row) {
        Raw<ES, G> rx;
        Raw<DES, G> rd;
        load_raw<ES, G>(rx, p.x, row * p.ldx + g * G);
        load_raw<DES, G>(rd, p.dy, row * p.lddy + g * G);
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float x[G], d[G];
        to_float<ES, G>(rx, p.x_f16, x);
        to_float<DES, G>(rd, p.dy_f16, d);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            dga[i] = fmaf(d[i], (x[i] - mean) * rstd, dga[i]);
            dbe[i] += d[i];
        }
    }
    const long long at = static_cast<long long>(blockIdx.y) * p.partial_step + g * G;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        p.partial[at + i] = dga[i];
        p.partial1[at + i] = dbe[i];
    }
}

}  // namespace fp8norm
