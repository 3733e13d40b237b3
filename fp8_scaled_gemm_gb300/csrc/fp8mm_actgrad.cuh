// fp8mm_actgrad.cuh -- gradient of an activation and of the bias before it:
//
//   dz = dy * act'(z)            one rounding
//   dbias[n] = sum over m of dy act'(z), from the unrounded products
//
// Bound by HBM: two reads and one write per element, and about 20
// instructions for the slope. A warp covers 8 LANES columns and 32 / LANES
// rows at a time (LANES < 32 for narrow matrices), NR times over, so that
// enough loads are in flight (16384 x 14336 bf16 gelu: one row of 256 columns
// per warp 296 us, two 279; with the slabs in whole waves of CTAs 240, 5.9 TB/s,
// 88 % of a copy; relu 219). 16-bit rows without 16-byte groups go in pairs where
// they start on 4 bytes (14334 columns 256 us, 82 %), else element by element
// (14335 columns 316 us, 67 %; two rows per warp 316). Each lane keeps
// the sums of its columns in registers over the rows of its slab (blockIdx.y).
// The CTA's warps add theirs in order, and the slabs' partials are added by
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
    float *partial;            // [slabs][N] (one slab: dbias itself), or nullptr
    long long M, N;
};

constexpr int kThreads = 256, kWarps = kThreads / 32;

// G = 8: a lane's columns are neighbours; G = 2 and 1: pairs and single columns,
// lane by lane (pairs: an even number of columns).
template <int ES, int G, int LANES, int NR>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const ActGradParams p)
{
    constexpr int K = 8 / G;                     // loads of a lane per row and operand
    constexpr int kCols = 8 * LANES, kRows = 32 / LANES;
    constexpr int kStep = G * LANES;             // columns between them
    __shared__ float cols[kWarps][kCols];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long n0 = static_cast<long long>(blockIdx.x) * kCols + (lane % LANES) * G;
    const int left = static_cast<int>(min(p.N - n0, 1ll << 20));   // columns from n0 on
    const long long slabs = gridDim.y, r0 = p.M * blockIdx.y / slabs, r1 = p.M * (blockIdx.y + 1) / slabs;
    const bool f16 = p.type == kF16;
    constexpr int kTurn = kWarps * kRows;        // rows of the CTA at a time
    float sum[8] = {};
    long long row = r0 + warp * kRows + lane / LANES;
    const uint8_t *dy = static_cast<const uint8_t *>(p.dy) + (row * p.ldy + n0) * ES;
    const uint8_t *z = static_cast<const uint8_t *>(p.z) + (row * p.ldz + n0) * ES;
    uint8_t *dz = static_cast<uint8_t *>(p.dz) + (row * p.ldd + n0) * ES;
    for (; row < r1; row += kTurn * NR) {
        Raw<ES, G> rd[NR][K], rz[NR][K];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const bool in_row = row + r * kTurn < r1;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool in = in_row && k * kStep < left;
                if (in)
                    load_raw<ES, G>(rd[r][k], dy + r * kTurn * p.ldy * ES, k * kStep);
                else
                    clear_raw<ES, G>(rd[r][k]);
                if (in && p.z)
                    load_raw<ES, G>(rz[r][k], z + r * kTurn * p.ldz * ES, k * kStep);
                else
                    clear_raw<ES, G>(rz[r][k]);
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float v[8], x[8];
            if constexpr (G == 8) {
                to_float<ES, 8>(rd[r][0], f16, v);
                to_float<ES, 8>(rz[r][0], f16, x);
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float a[G], b[G];
                    to_float<ES, G>(rd[r][k], f16, a);
                    to_float<ES, G>(rz[r][k], f16, b);
#pragma unroll
                    for (int e = 0; e < G; ++e) {
                        v[G * k + e] = a[e];
                        x[G * k + e] = b[e];
                    }
                }
            }
            fp8mm::apply_slope<8>(p.act, v, x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum[k] += v[k];
            if (p.dz && row + r * kTurn < r1) {
                uint8_t *o = dz + r * kTurn * p.ldd * ES;
                if constexpr (G == 8) {
                    if (left > 0)
                        store_group<8>(o, p.type, 0, v);
                } else if constexpr (G == 2) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (k * kStep < left)
                            *reinterpret_cast<uint32_t *>(o + k * kStep * 2) = pack2(v[2 * k], v[2 * k + 1], p.type);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k * kStep < left) {
                            const float one[1] = {v[k]};
                            store_group<1>(o, p.type, k * kStep, one);
                        }
                }
            }
        }
        dy += kTurn * NR * p.ldy * ES;
        z += kTurn * NR * p.ldz * ES;
        dz += kTurn * NR * p.ldd * ES;
    }
    if (p.partial == nullptr)
        return;
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
    if (lane < LANES) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            cols[warp][lane * G + k / G * kStep + k % G] = sum[k];
    }
    __syncthreads();
    const long long n = static_cast<long long>(blockIdx.x) * kCols + threadIdx.x;
    if (threadIdx.x < kCols && n < p.N) {
        float a = cols[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            a += cols[w][threadIdx.x];
        p.partial[static_cast<long long>(blockIdx.y) * p.N + n] = a;
    }
}

}  // namespace fp8act
