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
// Both are bound by HBM. A team of LANES x WARPS threads holds a row: thread
// t the element groups t, t + T, ... (T threads), so that every element is
// read once. Rows whose starts are 16-byte aligned take groups of 8
// elements, others single elements. Rows too long for a team go through
// the long kernels, which read the row again from L2 for each pass.
#pragma once

#include "fp8mm_act.cuh"
#include "fp8mm_quant_convert.cuh"
#include "fp8mm_rows.cuh"

namespace fp8norm {

using namespace fp8rows;

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
    long long R, C, groups;
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

// Threads of a CTA of such teams.
template <int LANES, int WARPS>
constexpr int kCtaThreads = LANES * WARPS > 256 ? LANES * WARPS : 256;

template <int ES, int G, int LANES, int WARPS, int CH>
__global__ void __launch_bounds__(kCtaThreads<LANES, WARPS>) norm_rows_kernel(const NormParams p)
{
    constexpr int T = LANES * WARPS;
    constexpr int kTeams = kCtaThreads<LANES, WARPS> / T;
    __shared__ float red[3][32];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();

    const int team = static_cast<int>(threadIdx.x) / T;
    const int t = static_cast<int>(threadIdx.x) % T;
    const float c_f = static_cast<float>(p.C);
    for (long long base = static_cast<long long>(blockIdx.x) * kTeams; base < p.R;
         base += static_cast<long long>(gridDim.x) * kTeams) {
        const long long row = base + team;
        const bool valid = row < p.R;
        Raw<ES, G> raw[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const long long g = t + c * T;
            if (valid && g < p.groups)
                load_raw<ES, G>(raw[c], p.x, row * p.ldx + g * G);
            else
                clear_raw<ES, G>(raw[c]);
        }
        float v[CH][G];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            to_float<ES, G>(raw[c], p.x_f16, v[c]);
#pragma unroll
            for (int i = 0; i < G; ++i)
                s[0] += v[c][i];
        }
        team_sum<LANES, WARPS, 1>(s, red[0]);
        const float mean = s[0] / c_f;
        s[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool in = t + c * T < p.groups;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                v[c][i] = in ? v[c][i] - mean : 0.0f;
                s[0] = fmaf(v[c][i], v[c][i], s[0]);
            }
        }
        team_sum<LANES, WARPS, 1>(s, red[1]);
        const float rstd = 1.0f / sqrtf(s[0] / c_f + p.eps);
        if (valid && t == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const long long g = t + c * T;
            if (g < p.groups) {
                float ga[G], be[G];
                load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
                load_param<G>(p.beta, p.param_type, g * G, 0.0f, be);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    v[c][i] = fmaf(v[c][i] * rstd, ga[i], be[i]);
                    amax = fp8mm::max_nan(amax, fabsf(v[c][i]));
                }
                if (p.y && valid)
                    store_group<G>(p.y, p.y_type, row * p.ldy + g * G, v[c]);
            }
        }
        if (p.q) {
            amax = team_max<LANES, WARPS>(amax, red[2]);
            const float scale = __fdiv_rn(amax, fp8q::qmax_of(p.q_type));
            if (valid && t == 0)
                p.q_scale[row] = scale;
            const fp8q::Divider d = fp8q::make_divider(scale);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const long long g = t + c * T;
                if (valid && g < p.groups)
                    store_codes<G>(p.q + row * p.C + g * G, d, v[c], p.q_type);
            }
        }
    }
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
    float *partial;            // [grid][2][C]: dgamma and dbeta sums of each CTA's rows, or nullptr
    long long R, C, groups;
};

// Rows base + team, base + teams x grid + team, ... : each thread keeps the
// dgamma and dbeta sums of its columns in registers over all its rows; the
// CTA's teams then add theirs in order through shared memory.
template <int ES, int DES, int G, int LANES, int WARPS, int CH>
__global__ void __launch_bounds__(kCtaThreads<LANES, WARPS>) norm_grad_rows_kernel(const NormGradParams p)
{
    constexpr int T = LANES * WARPS;
    constexpr int kThreads = kCtaThreads<LANES, WARPS>;
    constexpr int kTeams = kThreads / T;
    __shared__ float red[2][64];
    __shared__ float cols[kTeams > 1 ? kThreads * CH * G : 1];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();

    const int team = static_cast<int>(threadIdx.x) / T;
    const int t = static_cast<int>(threadIdx.x) % T;
    const float inv_c = 1.0f / static_cast<float>(p.C);
    float dga[CH][G] = {}, dbe[CH][G] = {};
    int flip = 0;
    for (long long base = static_cast<long long>(blockIdx.x) * kTeams; base < p.R;
         base += static_cast<long long>(gridDim.x) * kTeams) {
        const long long row = base + team;
        const bool valid = row < p.R;
        Raw<ES, G> rx[CH];
        Raw<DES, G> rd[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const long long g = t + c * T;
            if (valid && g < p.groups) {
                load_raw<ES, G>(rx[c], p.x, row * p.ldx + g * G);
                load_raw<DES, G>(rd[c], p.dy, row * p.lddy + g * G);
            } else {
                clear_raw<ES, G>(rx[c]);
                clear_raw<DES, G>(rd[c]);
            }
        }
        const float mean = valid ? __ldg(p.mean + row) : 0.0f;
        const float rstd = valid ? __ldg(p.rstd + row) : 0.0f;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const long long g = t + c * T;
            if (g < p.groups) {
                float x[G], d[G], ga[G];
                to_float<ES, G>(rx[c], p.x_f16, x);
                to_float<DES, G>(rd[c], p.dy_f16, d);
                load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const float h = (x[i] - mean) * rstd;
                    const float w = d[i] * ga[i];
                    s[0] += w;
                    s[1] = fmaf(w, h, s[1]);
                    dga[c][i] = fmaf(d[i], h, dga[c][i]);
                    dbe[c][i] += d[i];
                }
            }
        }
        if (p.dx == nullptr)
            continue;                   // uniform: parameter sums only
        team_sum<LANES, WARPS, 2>(s, red[flip]);
        flip ^= 1;
        const float m1 = s[0] * inv_c, m2 = s[1] * inv_c;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const long long g = t + c * T;
            if (valid && g < p.groups) {
                float x[G], d[G], ga[G], o[G];
                to_float<ES, G>(rx[c], p.x_f16, x);
                to_float<DES, G>(rd[c], p.dy_f16, d);
                load_param<G>(p.gamma, p.param_type, g * G, 1.0f, ga);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const float h = (x[i] - mean) * rstd;
                    o[i] = rstd * (fmaf(-h, m2, d[i] * ga[i]) - m1);
                }
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
    if (p.partial == nullptr)
        return;
    // this CTA's column sums, the teams' in order
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float *dst = p.partial + (static_cast<long long>(blockIdx.x) * 2 + k) * p.C;
        float(*v)[G] = k == 0 ? dga : dbe;
        if constexpr (kTeams > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < G; ++i)
                    cols[team * (T * CH * G) + (t + c * T) * G + i] = v[c][i];
            __syncthreads();
            for (long long c = threadIdx.x; c < p.C; c += kThreads) {
                float a = cols[c];
                for (int m = 1; m < kTeams; ++m)
                    a += cols[m * (T * CH * G) + c];
                dst[c] = a;
            }
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const long long g = t + c * T;
                if (g < p.groups) {
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        dst[g * G + i] = v[c][i];
                }
            }
        }
    }
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
    float *dst = p.partial + static_cast<long long>(blockIdx.y) * 2 * p.C + g * G;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        dst[i] = dga[i];
        dst[p.C + i] = dbe[i];
    }
}

}  // namespace fp8norm
