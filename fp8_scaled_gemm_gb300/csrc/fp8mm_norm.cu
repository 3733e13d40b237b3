// fp8mm_norm.cu -- C entry of layer norm's forward pass.
#include "fp8mm_norm.cuh"
#include "fp8mm_rows_host.h"

namespace {

using namespace fp8mm_host;
using fp8norm::NormParams;

template <int ES, int G, int KIND, int CH>
int launch_norm(const NormParams &p, int64_t grid, int threads, cudaStream_t stream)
{
    auto kern = fp8norm::norm_kernel<ES, G, KIND, CH>;
    const int smem = (KIND > 0 ? KIND : threads) * 4 * CH * 16;   // one team's gamma and beta
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (KIND <= 0 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * 4 * CH * 16);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    return launch_pdl(kern, static_cast<int>(grid), threads, smem, stream, "layer norm launch", p);
}

// Teams of LANES lanes of a warp, 256 threads to a CTA.
template <int ES, int G, int LANES, int CH>
int launch_lanes(const NormParams &p, int sms, cudaStream_t stream)
{
    return launch_norm<ES, G, LANES, CH>(
        p, std::min<int64_t>(cdiv(p.R, 256 / LANES), static_cast<int64_t>(sms) * (CH == 4 ? 3 : 4)), 256, stream);
}

// Longer rows go through the long kernel.
constexpr int64_t kMostColumns = 1024 * 16 * fp8norm::kMaxCluster;

// A CTA per row, as many of them on an SM as make 1024 threads.
template <int ES, int G, int CH>
int launch_cta(const NormParams &p, int sms, cudaStream_t stream)
{
    const int threads = static_cast<int>(cdiv(p.C, 32 * 8 * CH)) * 32;
    return launch_norm<ES, G, fp8norm::kCta, CH>(
        p, std::min<int64_t>(p.R, static_cast<int64_t>(sms) * (1024 / threads)), threads, stream);
}

// A cluster of CTAs per row, two as long as they suffice, else eight (32768
// bf16 columns with codes: two 194 us, four 298; 65536: four 386, eight 325).
// The long kernel, which reads the row once per quantity, took 428 and 455.
template <int ES, int G>
int launch_cluster(NormParams p, int sms, cudaStream_t stream)
{
    constexpr int warp_cols = 32 * 8 * 2;
    const int64_t warps = cdiv(p.C, warp_cols);
    const int ctas = warps <= 64 ? 2 : fp8norm::kMaxCluster;
    const int64_t each = cdiv(warps, ctas);
    p.slice_cols = each * warp_cols;
    int rc = device_limit(&p.limit.status, &p.limit.clocks);
    if (rc != FP8MM_OK)
        return rc;
    const int threads = static_cast<int>(each) * 32;
    const int64_t clusters =
        std::min<int64_t>(p.R, std::max<int64_t>(1, static_cast<int64_t>(sms) * (1024 / threads) / ctas));
    auto kern = fp8norm::norm_kernel<ES, G, fp8norm::kCluster, 2>;
    const int smem = threads * 4 * 2 * 16;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * 4 * 2 * 16);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    return launch_clusters(kern, static_cast<int>(clusters) * ctas, ctas, threads, smem, stream, "layer norm launch", p);
}

// Rows without 16-byte groups: pairs (G = 2) or single elements.
template <int ES, int G>
int launch_narrow(const NormParams &p, int sms, cudaStream_t stream)
{
    const int64_t C = p.C;
    if (C <= 256) return launch_lanes<ES, G, 32, 1>(p, sms, stream);
    if (C <= 512) return launch_lanes<ES, G, 32, 2>(p, sms, stream);
    if (C <= 1024) return launch_lanes<ES, G, 32, 4>(p, sms, stream);
    if (C <= 16384) return launch_cta<ES, G, 2>(p, sms, stream);
    return launch_cluster<ES, G>(p, sms, stream);
}

template <int ES>
int launch(const NormParams &p, bool vec, bool pairs, int sms, cudaStream_t stream)
{
    const int64_t C = p.C;
    if (vec) {
        if (C <= 32) return launch_lanes<ES, 8, 4, 1>(p, sms, stream);
        if (C <= 64) return launch_lanes<ES, 8, 8, 1>(p, sms, stream);
        if (C <= 128) return launch_lanes<ES, 8, 16, 1>(p, sms, stream);
        if (C <= 256) return launch_lanes<ES, 8, 32, 1>(p, sms, stream);
        if (C <= 512) return launch_lanes<ES, 8, 32, 2>(p, sms, stream);
        if (C <= 1024) return launch_lanes<ES, 8, 32, 4>(p, sms, stream);
        if (C <= 16384) return launch_cta<ES, 8, 2>(p, sms, stream);
        if (C <= kMostColumns) return launch_cluster<ES, 8>(p, sms, stream);
    } else if (C <= kMostColumns) {
        if constexpr (ES == 2)
            if (pairs)
                return launch_narrow<ES, 2>(p, sms, stream);
        return launch_narrow<ES, 1>(p, sms, stream);
    }
    const int grid = static_cast<int>(std::min<int64_t>(p.R, static_cast<int64_t>(sms) * 8));
    if (vec)
        return launch_pdl(fp8norm::norm_long_kernel<ES, 8>, grid, fp8norm::kLongThreads, 0, stream,
                          "layer norm launch", p);
    return launch_pdl(fp8norm::norm_long_kernel<ES, 1>, grid, fp8norm::kLongThreads, 0, stream, "layer norm launch", p);
}

}  // namespace

extern "C" int fp8_layer_norm(const void *x, int x_type, int64_t ldx, const void *gamma, const void *beta,
                              int param_type, float eps, void *y, int y_type, int64_t ldy, float *mean, float *rstd,
                              void *q, int q_type, float *q_scale, int64_t R, int64_t C, void *stream)
{
    if (!row_type_known(x_type) || !row_type_known(y_type) || !row_type_known(param_type) ||
        (q && q_type != FP8MM_TYPE_E4M3 && q_type != FP8MM_TYPE_E5M2))
        return FP8MM_ERR_MODE;
    if (R < 0 || C < 0 || R > (int64_t(1) << 40) / std::max<int64_t>(C, 1) || !(eps >= 0.0f) || eps > 3e38f)
        return FP8MM_ERR_SHAPE;
    int rc;
    if ((rc = check_rows(x, ldx, C, x_type)) != FP8MM_OK || (rc = check_rows(y, ldy, C, y_type)) != FP8MM_OK ||
        (rc = check_rows(gamma, 0, C, param_type)) != FP8MM_OK ||
        (rc = check_rows(beta, 0, C, param_type)) != FP8MM_OK ||
        (rc = check_rows(mean, 0, C, FP8MM_OUT_F32)) != FP8MM_OK ||
        (rc = check_rows(rstd, 0, C, FP8MM_OUT_F32)) != FP8MM_OK ||
        (rc = check_rows(q_scale, 0, C, FP8MM_OUT_F32)) != FP8MM_OK)
        return rc;
    if (R == 0 || C == 0)
        return FP8MM_OK;
    if (!x || (q && !q_scale))
        return FP8MM_ERR_NULL;
    if (y == x || q == x || (q && q == y))
        return FP8MM_ERR_MODE;   // a long row is read more than once
    int sms = 0;
    if ((rc = device_sms(&sms)) != FP8MM_OK)
        return rc;
    NormParams p{};
    p.x = x;
    p.ldx = ldx > 0 ? ldx : C;
    p.x_f16 = x_type == FP8MM_OUT_F16;
    p.gamma = gamma;
    p.beta = beta;
    p.param_type = param_type;
    p.eps = eps;
    p.y = y;
    p.y_type = y_type;
    p.ldy = ldy > 0 ? ldy : C;
    p.mean = mean;
    p.rstd = rstd;
    p.q = static_cast<uint8_t *>(q);
    p.q_type = q_type;
    p.q_scale = q_scale;
    p.R = R;
    p.C = C;
    const bool vec = C % 8 == 0 && rows_vec(x, p.ldx, x_type) && (!y || rows_vec(y, p.ldy, y_type)) &&
                     rows_vec(gamma, 0, param_type) && rows_vec(beta, 0, param_type) &&
                     (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    const bool pairs = C % 2 == 0 && rows_pairs(x, p.ldx, x_type) && (!y || rows_pairs(y, p.ldy, y_type)) &&
                       rows_pairs(gamma, 0, param_type) && rows_pairs(beta, 0, param_type) &&
                       (reinterpret_cast<uintptr_t>(q) & 1) == 0;
    p.groups = vec ? C / 8 : C;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return x_type == FP8MM_OUT_F32 ? launch<4>(p, vec, pairs, sms, s) : launch<2>(p, vec, pairs, sms, s);
}
