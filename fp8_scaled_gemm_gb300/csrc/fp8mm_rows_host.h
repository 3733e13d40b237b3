// fp8mm_rows_host.h -- argument checks and small helpers of the row operators'
// C entries (layer norm, activation gradient).
#pragma once

#include <algorithm>

#include "fp8mm_host.h"

namespace fp8mm_host {

// Element types of the row operators: FP8MM_OUT_BF16, _F16 or _F32.
inline bool row_type_known(int t) { return t == FP8MM_OUT_BF16 || t == FP8MM_OUT_F16 || t == FP8MM_OUT_F32; }
inline int64_t row_type_bytes(int t) { return t == FP8MM_OUT_F32 ? 4 : 2; }

// A [R, C] matrix with row stride ld (0 = C): FP8MM_ERR_SHAPE for a stride
// under C, FP8MM_ERR_ALIGN for a base off its element.
inline int check_rows(const void *p, int64_t ld, int64_t C, int type)
{
    if (ld < 0 || (ld > 0 && ld < C) || ld >= (int64_t(1) << 36))
        return FP8MM_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(p) & (row_type_bytes(type) - 1))
        return FP8MM_ERR_ALIGN;
    return FP8MM_OK;
}

// Whether groups of 8 elements of every row start on 16 bytes.
inline bool rows_vec(const void *p, int64_t ld, int type)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * row_type_bytes(type)) % 16 == 0;
}

// Whether pairs of 16-bit elements of every row start on 4 bytes (fp32 rows do).
inline bool rows_pairs(const void *p, int64_t ld, int type)
{
    return type == FP8MM_OUT_F32 || ((reinterpret_cast<uintptr_t>(p) & 3) == 0 && ld % 2 == 0);
}

// Launch on a two-dimensional grid with programmatic stream serialization.
template <typename Kern, typename... Args>
int launch_grid2(Kern kern, int64_t gx, int64_t gy, int threads, cudaStream_t stream, const char *what, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? FP8MM_OK : cuda_fail(e, what);
}

}  // namespace fp8mm_host
