// fp8mm_actgrad.cuh -- gradient of an activation and of the bias before it:
//
//   dz = dy * act'(z)            one rounding
//   dbias[n] = sum over m of dy act'(z), from the unrounded products
//
// Bound by HBM: two reads and one write per element. A CTA takes a strip of
// 32 G columns and the rows of its slab (blockIdx.y), warp w rows w, w + 8,
// ...; each lane keeps the sums of its columns in registers, the CTA's warps
// add theirs in order, and the slabs' partials are added by
// fp8rows::partial_sum_kernel.
#pragma once

#include "fp8mm_act.cuh"
#include "fp8mm_rows.cuh"

namespace fp8act {

using namespace fp8rows;

struct ActGradParams {
    const void *dy, *z;        // z: nullptr without activation
    long long ldy, ldz;
    int type, act;
    void *dz;                  // nullptr: not wanted
    long long ldd;
    float *partial;            // [slabs][N], or nullptr
    long long M, N;
};

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int ES, int G>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const ActGradParams p)
{
    // lane's columns: G neighbours (G = 8) or 8 columns 32 apart (G = 1)
    constexpr int K = G == 8 ? 1 : 8;
    constexpr int kCols = 256;
    __shared__ float cols[kWarps][kCols];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long n0 = static_cast<long long>(blockIdx.x) * kCols;
    const long long slabs = gridDim.y, r0 = p.M * blockIdx.y / slabs, r1 = p.M * (blockIdx.y + 1) / slabs;
    const bool f16 = p.type == kF16;
    float sum[K][G] = {};
    for (long long row = r0 + warp; row < r1; row += kWarps) {
        float v[K * G], z[K * G];
        Raw<ES, G> rd[K], rz[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long n = n0 + (k * 32 + lane) * G;
            if (n < p.N) {
                load_raw<ES, G>(rd[k], p.dy, row * p.ldy + n);
                if (p.z)
                    load_raw<ES, G>(rz[k], p.z, row * p.ldz + n);
                else
                    clear_raw<ES, G>(rz[k]);
            } else {
                clear_raw<ES, G>(rd[k]);
                clear_raw<ES, G>(rz[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float a[G], b[G];
            to_float<ES, G>(rd[k], f16, a);
            to_float<ES, G>(rz[k], f16, b);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                v[k * G + i] = a[i];
                z[k * G + i] = b[i];
            }
        }
        fp8mm::apply_slope<K * G>(p.act, v, z);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long n = n0 + (k * 32 + lane) * G;
            float o[G];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                o[i] = v[k * G + i];
                sum[k][i] += o[i];
            }
            if (p.dz && n < p.N)
                store_group<G>(p.dz, p.type, row * p.ldd + n, o);
        }
    }
    if (p.partial == nullptr)
        return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < G; ++i)
            cols[warp][(k * 32 + lane) * G + i] = sum[k][i];
    __syncthreads();
    const long long n = n0 + threadIdx.x;
    if (n < p.N) {
        float a = cols[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            a += cols[w][threadIdx.x];
        p.partial[static_cast<long long>(blockIdx.y) * p.N + n] = a;
    }
}

}  // namespace fp8act
