// fp8mm_host.h -- what the library's translation units share on the host side:
// error text, device checks, launch helper and kernel choice.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8mm.h"

namespace fp8mm {
struct KernelParams;
template <bool EPI>
struct EpiMaps;
}

namespace fp8mm_host {

constexpr int kMaxDevices = 64;

// The text fp8mm_last_error() returns on this thread.
void set_error(const char *text);

// Records a failed CUDA call's text; returns FP8MM_ERR_CUDA.
int cuda_fail(cudaError_t e, const char *what);

// Checks that the current device is one the library is built for (once per
// device) and returns its SM count.
int device_sms(int *sms);

// The current device's status word and the clocks a wait in a kernel may take.
int device_limit(int **status, unsigned long long *clocks);

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Choice {
    int variant;   // FP8MM_VARIANT_TILE, _SWAP, _PAIR, _SWAPK or _SWAPPAIR
    int tile_n;
    int split;
    int tiles_p, tiles_q, kblocks, units, grid;
    int sk_tiles;  // PAIR: tiles whose K blocks are spread over all pairs (stream-K), 0: none
};

// The launch of a chosen kernel with the extended epilogue
// (KernelParams::e), compiled in translation units of their own.
int dispatch_epilogue(const Choice &c, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
                      const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> &em, cudaStream_t stream);
int dispatch_epilogue_swap(const Choice &c, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
                           const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> &em, cudaStream_t stream);

// Launch with programmatic stream serialization: the kernel may start its
// set-up while the previous kernel in the stream finishes; it calls
// griddepcontrol.wait before touching global memory.
template <typename Kern, typename... Args>
int launch_pdl(Kern kern, int grid, int threads, int smem, cudaStream_t stream, const char *what, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess)
        return cuda_fail(e, what);
    return FP8MM_OK;
}

// The same with the grid in clusters of `cluster` CTAs.
template <typename Kern, typename... Args>
int launch_clusters(Kern kern, int grid, int cluster, int threads, int smem, cudaStream_t stream, const char *what,
                    Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess)
        return cuda_fail(e, what);
    return FP8MM_OK;
}

}  // namespace fp8mm_host
