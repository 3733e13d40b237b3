// fp8mm_launch.cuh -- launches of the matmul kernels, with the plain epilogue
// (EPI = false) or the extended one.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8mm_host.h"
#include "fp8mm_kernel.cuh"
#include "fp8mm_kernel_ck.cuh"
#include "fp8mm_kernel_pair.cuh"

namespace fp8mm_host {

// The 256-wide 1-SM kernel runs 16 epilogue warps up to this K. Measured on
// GB300 (CUDA-graph replays, row-wise + bias) against 8 warps: 8191 x 8193 x
// 32 87.0 -> 71.3 us, 8192 x 8192 x 32 52.6 -> 44.8, 8192 x 8192 x 512
// 54.8 -> 46.1; at K = 1024 16 warps lost (16384 x 8192 x 1024 127.7 ->
// 141.1, 4096 x 4096 x 1024 21.3 -> 23.2).
constexpr int64_t kTileWideMaxK = 512;
// The same with the extended epilogue, whose 16 warps leave a ring of two
// stages. Measured at 8192 x 8192 with residual, gelu and z against 8 warps:
// K = 64 130 -> 105 us, 512 133 -> 108, 1024 144 -> 126 (without the residual
// and z, silu: 99 -> 89; no activation, residual only: 97 -> 102).
constexpr int64_t kTileWideMaxKExt = 1024;

// A kernel's argument of the extended epilogue's tensor maps.
template <bool EPI>
fp8mm::EpiMaps<EPI> maps_for(const fp8mm::EpiMaps<true> *em)
{
    if constexpr (EPI)
        return *em;
    else
        return {};
}

template <int BN, int CS, bool EPI>
int launch_swapk(const CUtensorMap &mp, const CUtensorMap &mq, const fp8mm::KernelParams &kp, int grid,
                 cudaStream_t stream)
{
    using C = fp8mm::ClusterKCfg<BN, CS>;
    auto kern = fp8mm::fp8mm_swap_ck_kernel<BN, CS, EPI>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    return launch_pdl(kern, grid, fp8mm::kThreads, C::kSmemBytes, stream, "cluster-K kernel launch", mp, mq, kp);
}

template <int BN, bool SWAP, bool WIDE, bool EPI>
int launch_kernel(const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
                  const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> *em, int grid, cudaStream_t stream)
{
    using C = fp8mm::TileCfg<BN, SWAP, WIDE, EPI>;
    auto kern = fp8mm::fp8mm_tc_kernel<BN, SWAP, WIDE, EPI>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    return launch_pdl(kern, grid, C::kThreads, C::kSmemBytes, stream, "kernel launch", mp, mq,
                      mo, kp, maps_for<EPI && !SWAP>(em));
}

template <int BN, bool SWAP, bool EPI>
int launch_pair(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo,
                const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> *em, int grid, cudaStream_t stream)
{
    using C = fp8mm::PairCfg<BN, SWAP, EPI>;
    auto kern = fp8mm::fp8mm_pair_kernel<BN, SWAP, EPI>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    return launch_pdl(kern, grid, fp8mm::EpiShape<SWAP>::kThreads, C::kSmemBytes, stream, "pair kernel launch",
                      ma, mb, mo, kp, maps_for<EPI && !SWAP>(em));
}

// Kernels a translation unit compiles: those whose tile rows run over M, and
// those with the operands swapped (skinny M).
constexpr int kRowKernels = 1, kSwapKernels = 2;

template <bool EPI, int KERNELS>
int dispatch(const Choice &c, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
             const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> *em, cudaStream_t stream)
{
    if constexpr ((KERNELS & kSwapKernels) != 0) {
        if (c.variant == FP8MM_VARIANT_SWAPK) {
            switch (c.tile_n * 10 + c.split) {
            case 162: return launch_swapk<16, 2, EPI>(mp, mq, kp, c.grid, stream);
            case 164: return launch_swapk<16, 4, EPI>(mp, mq, kp, c.grid, stream);
            case 168: return launch_swapk<16, 8, EPI>(mp, mq, kp, c.grid, stream);
            case 322: return launch_swapk<32, 2, EPI>(mp, mq, kp, c.grid, stream);
            case 324: return launch_swapk<32, 4, EPI>(mp, mq, kp, c.grid, stream);
            case 328: return launch_swapk<32, 8, EPI>(mp, mq, kp, c.grid, stream);
            case 642: return launch_swapk<64, 2, EPI>(mp, mq, kp, c.grid, stream);
            case 644: return launch_swapk<64, 4, EPI>(mp, mq, kp, c.grid, stream);
            case 648: return launch_swapk<64, 8, EPI>(mp, mq, kp, c.grid, stream);
            case 1282: return launch_swapk<128, 2, EPI>(mp, mq, kp, c.grid, stream);
            case 1284: return launch_swapk<128, 4, EPI>(mp, mq, kp, c.grid, stream);
            case 1288: return launch_swapk<128, 8, EPI>(mp, mq, kp, c.grid, stream);
            }
        } else if (c.variant == FP8MM_VARIANT_SWAPPAIR) {
            switch (c.tile_n) {
            case 16: return launch_pair<16, true, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 32: return launch_pair<32, true, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 64: return launch_pair<64, true, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 128: return launch_pair<128, true, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            }
        } else if (c.variant == FP8MM_VARIANT_SWAP) {
            switch (c.tile_n) {
            case 16: return launch_kernel<16, true, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 32: return launch_kernel<32, true, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 64: return launch_kernel<64, true, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 128: return launch_kernel<128, true, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            }
        }
    }
    if constexpr ((KERNELS & kRowKernels) != 0) {
        if (c.variant == FP8MM_VARIANT_PAIR) {
            switch (c.tile_n) {
            case 128: return launch_pair<128, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 256: return launch_pair<256, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            }
        } else if (c.variant == FP8MM_VARIANT_TILE) {
            switch (c.tile_n) {
            case 128: return launch_kernel<128, false, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            case 256:
                // shallow K: 16 epilogue warps (the epilogue sets the time per
                // tile); deeper K keeps 8 and a deeper ring
                if (kp.K <= (EPI ? kTileWideMaxKExt : kTileWideMaxK))
                    return launch_kernel<256, false, true, EPI>(mp, mq, mo, kp, em, c.grid, stream);
                return launch_kernel<256, false, false, EPI>(mp, mq, mo, kp, em, c.grid, stream);
            }
        }
    }
    return FP8MM_ERR_MODE;
}

}  // namespace fp8mm_host
