// fp8mm_norm_grad.cu -- C entry of layer norm's backward pass.
#include "fp8mm_norm.cuh"
#include "fp8mm_rows_host.h"

namespace {

using namespace fp8mm_host;
using fp8norm::NormGradParams;

// Threads of the row kernels on an SM (their registers allow 512), and so, at
// 64 threads for the smallest CTA with a row of its own, CTAs and partial sums.
constexpr int kMostPerSm = fp8norm::kGradThreads / 64;

// Rows each team takes at least, where there are enough: a team's column sums
// cost as much traffic as two to four rows.
constexpr int kRowsPerTeam = 4;

// Partial sums of dgamma and dbeta a call on R rows may write. Few rows go to
// one team, whose sums are the results: no workspace and no second launch
// (1 x 4096 bf16: 4.6 us with them, 2.9 without).
int64_t max_partials(int64_t R, int sms)
{
    return R <= kRowsPerTeam ? 1 : std::min<int64_t>(R, static_cast<int64_t>(sms) * kMostPerSm);
}

int64_t partials_bytes(int64_t R, int64_t C, int sms)
{
    const int64_t P = max_partials(R, sms);
    return P == 1 ? 0 : P * 2 * C * static_cast<int64_t>(sizeof(float));
}

int sum_partials(const NormGradParams &p, int P, float *dgamma, float *dbeta, cudaStream_t stream)
{
    fp8rows::PartialSumParams s{};
    s.partial = p.partial;
    s.out0 = dgamma;
    s.out1 = dbeta;
    s.C = p.C;
    s.P = P;
    s.K = 2;
    return launch_grid2(fp8rows::partial_sum_kernel, cdiv(p.C, 32), 2, fp8rows::kSumThreads, stream,
                        "parameter sum launch", s);
}

// Teams of LANES lanes of a warp.
template <int ES, int DES, int G, int LANES>
int launch_lanes(const NormGradParams &p, int sms, cudaStream_t stream, int *partials)
{
    constexpr int CH = fp8norm::kGradCh<ES, DES, G, LANES>, threads = fp8norm::kGradLaneThreads;
    const int64_t grid = std::min<int64_t>(cdiv(p.R, kRowsPerTeam * (threads / LANES)),
                                           static_cast<int64_t>(sms) * fp8norm::kGradLaneCtas<ES, DES>);
    *partials = static_cast<int>(grid);
    return launch_pdl(fp8norm::norm_grad_kernel<ES, DES, G, LANES, CH>, static_cast<int>(grid), threads,
                      threads * 2 * 16 * CH, stream, "layer norm gradient launch", p);
}

// A CTA per row, as many of them on an SM as make 512 threads.
template <int ES, int DES, int G>
int launch_cta(const NormGradParams &p, int threads, int sms, cudaStream_t stream, int *partials)
{
    constexpr int CH = fp8norm::kGradCh<ES, DES, G, fp8norm::kCta>;
    const int64_t grid = std::min<int64_t>(
        cdiv(p.R, kRowsPerTeam), static_cast<int64_t>(sms) * std::min(kMostPerSm, fp8norm::kGradThreads / threads));
    *partials = static_cast<int>(grid);
    return launch_pdl(fp8norm::norm_grad_kernel<ES, DES, G, fp8norm::kCta, CH>, static_cast<int>(grid), threads,
                      threads * 2 * 16 * CH, stream, "layer norm gradient launch", p);
}

// A cluster of `ctas` CTAs per row.
template <int ES, int DES, int G>
int launch_cluster(NormGradParams p, int ctas, int64_t slice_cols, int threads, int sms, cudaStream_t stream,
                   int *partials)
{
    p.slice_cols = slice_cols;
    const int64_t clusters =
        p.R <= kRowsPerTeam
            ? 1
            : std::min<int64_t>(p.R, std::max<int64_t>(1, static_cast<int64_t>(sms) *
                                                              std::min(kMostPerSm, fp8norm::kGradThreads / threads) / ctas));
    const int rc = device_limit(&p.limit.status, &p.limit.clocks);
    if (rc != FP8MM_OK)
        return rc;
    *partials = static_cast<int>(clusters);
    constexpr int CH = fp8norm::kGradCh<ES, DES, G, fp8norm::kCluster>;
    void (*kern)(NormGradParams);
    if constexpr (CH == 2)
        kern = fp8norm::norm_grad_cluster_kernel<ES, DES, G, CH>;
    else
        kern = fp8norm::norm_grad_kernel<ES, DES, G, fp8norm::kCluster, CH>;
    return launch_clusters(kern, static_cast<int>(clusters) * ctas, ctas, threads, threads * 2 * 16 * CH, stream,
                           "layer norm gradient launch", p);
}

template <int ES, int DES, int G>
int launch_long(const NormGradParams &p, int sms, cudaStream_t stream, int *partials)
{
    int rc = FP8MM_OK;
    if (p.dx)
        rc = launch_pdl(fp8norm::norm_grad_long_kernel<ES, DES, G>,
                        static_cast<int>(std::min<int64_t>(p.R, static_cast<int64_t>(sms) * 8)),
                        fp8norm::kLongThreads, 0, stream, "layer norm gradient launch", p);
    if (rc != FP8MM_OK || !p.partial)
        return rc;
    const int64_t strips = cdiv(p.groups, 256);
    const int64_t slabs = std::max<int64_t>(
        1, std::min<int64_t>(max_partials(p.R, sms), static_cast<int64_t>(sms) * 8 / strips));
    *partials = static_cast<int>(slabs);
    return launch_grid2(fp8norm::norm_grad_cols_kernel<ES, DES, G>, strips, slabs, 256, stream,
                        "layer norm parameter launch", p);
}

template <int ES, int DES, int G>
int launch_wide(const NormGradParams &p, int sms, cudaStream_t stream, int *P)
{
    constexpr int warp_cols = 32 * 8 * fp8norm::kGradCh<ES, DES, G, fp8norm::kCta>;
    constexpr int most = fp8norm::kGradThreads / 32;
    const int64_t warps = cdiv(p.C, warp_cols);
    if (warps <= most)
        return launch_cta<ES, DES, G>(p, static_cast<int>(warps) * 32, sms, stream, P);
    // two CTAs as long as they suffice, else eight (4096 x 20000 bf16: four 422
    // us, eight 292)
    for (int ctas : {2, fp8norm::kMaxCluster})
        if (warps <= most * ctas) {
            const int64_t each = cdiv(warps, ctas);
            return launch_cluster<ES, DES, G>(p, ctas, each * warp_cols, static_cast<int>(each) * 32, sms, stream, P);
        }
    return launch_long<ES, DES, G == 8 ? 8 : 1>(p, sms, stream, P);
}

template <int ES, int DES>
int launch(const NormGradParams &p, bool vec, bool pairs, int sms, cudaStream_t stream, int *P)
{
    const int64_t C = p.C;
    if (vec) {
        if (C <= 32) return launch_lanes<ES, DES, 8, 4>(p, sms, stream, P);
        if (C <= 64) return launch_lanes<ES, DES, 8, 8>(p, sms, stream, P);
        if (C <= 128) return launch_lanes<ES, DES, 8, 16>(p, sms, stream, P);
        if (C <= 256) return launch_lanes<ES, DES, 8, 32>(p, sms, stream, P);
        return launch_wide<ES, DES, 8>(p, sms, stream, P);
    }
    if constexpr (ES == 2 && DES == 2)
        if (pairs)
            return C <= 256 ? launch_lanes<ES, DES, 2, 32>(p, sms, stream, P) : launch_wide<ES, DES, 2>(p, sms, stream, P);
    if (C <= 256)
        return launch_lanes<ES, DES, 1, 32>(p, sms, stream, P);
    return launch_wide<ES, DES, 1>(p, sms, stream, P);
}

}  // namespace

extern "C" {

int64_t fp8_layer_norm_grad_workspace(int64_t R, int64_t C)
{
    if (R < 0 || C < 0 || R > (int64_t(1) << 40) / std::max<int64_t>(C, 1))
        return FP8MM_ERR_SHAPE;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc != FP8MM_OK)
        return rc;
    return partials_bytes(R, C, sms);
}

int fp8_layer_norm_grad(const void *dy, int dy_type, int64_t lddy, const void *x, int x_type, int64_t ldx,
                        const void *gamma, int param_type, const float *mean, const float *rstd, const void *dres,
                        int64_t lddres, void *dx, int64_t lddx, float *dgamma, float *dbeta, int64_t R, int64_t C,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!row_type_known(x_type) || !row_type_known(dy_type) || !row_type_known(param_type))
        return FP8MM_ERR_MODE;
    if (R < 0 || C < 0 || R > (int64_t(1) << 40) / std::max<int64_t>(C, 1))
        return FP8MM_ERR_SHAPE;
    int rc;
    if ((rc = check_rows(x, ldx, C, x_type)) != FP8MM_OK || (rc = check_rows(dy, lddy, C, dy_type)) != FP8MM_OK ||
        (rc = check_rows(dres, lddres, C, x_type)) != FP8MM_OK || (rc = check_rows(dx, lddx, C, x_type)) != FP8MM_OK ||
        (rc = check_rows(gamma, 0, C, param_type)) != FP8MM_OK)
        return rc;
    for (const void *f : {static_cast<const void *>(mean), static_cast<const void *>(rstd),
                          static_cast<const void *>(dgamma), static_cast<const void *>(dbeta),
                          static_cast<const void *>(workspace)})
        if ((rc = check_rows(f, 0, C, FP8MM_OUT_F32)) != FP8MM_OK)
            return rc;
    if (reinterpret_cast<uintptr_t>(workspace) & 15)
        return FP8MM_ERR_ALIGN;
    if (!dgamma != !dbeta)
        return FP8MM_ERR_NULL;
    if (C == 0 || (R == 0 && !dgamma))
        return FP8MM_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (R == 0) {
        // sums over no rows
        if ((rc = device_sms(&sms)) != FP8MM_OK)
            return rc;
        cudaError_t e = cudaMemsetAsync(dgamma, 0, static_cast<size_t>(C) * 4, s);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(dbeta, 0, static_cast<size_t>(C) * 4, s);
        return e == cudaSuccess ? FP8MM_OK : cuda_fail(e, "cudaMemsetAsync(parameter gradients)");
    }
    if (!dy || !x || !mean || !rstd)
        return FP8MM_ERR_NULL;
    const int64_t ldr = lddres > 0 ? lddres : C, ldd = lddx > 0 ? lddx : C;
    if (dx && (dx == dy || dx == x || (dx == dres && ldr != ldd)))
        return FP8MM_ERR_MODE;   // dx may replace dres only, every element over itself
    if ((rc = device_sms(&sms)) != FP8MM_OK)
        return rc;
    if (dgamma) {
        const int64_t need = partials_bytes(R, C, sms);
        if (need > 0 && !workspace)
            return FP8MM_ERR_NULL;
        if (workspace_bytes < need)
            return FP8MM_ERR_SHAPE;
    }
    NormGradParams p{};
    p.dy = dy;
    p.x = x;
    p.lddy = lddy > 0 ? lddy : C;
    p.ldx = ldx > 0 ? ldx : C;
    p.dy_f16 = dy_type == FP8MM_OUT_F16;
    p.x_f16 = x_type == FP8MM_OUT_F16;
    p.gamma = gamma;
    p.param_type = param_type;
    p.mean = mean;
    p.rstd = rstd;
    p.dres = dx ? dres : nullptr;
    p.lddres = ldr;
    p.dx = dx;
    p.lddx = ldd;
    p.x_type = x_type;
    const bool direct = dgamma && max_partials(R, sms) == 1;
    p.partial = direct ? dgamma : dgamma ? static_cast<float *>(workspace) : nullptr;
    p.partial1 = direct ? dbeta : p.partial + C;
    p.partial_step = 2 * C;
    p.R = R;
    p.C = C;
    const bool vec = C % 8 == 0 && rows_vec(x, p.ldx, x_type) && rows_vec(dy, p.lddy, dy_type) &&
                     (!p.dres || rows_vec(dres, ldr, x_type)) && (!dx || rows_vec(dx, ldd, x_type)) &&
                     rows_vec(gamma, 0, param_type) &&
                     (!direct || (rows_vec(dgamma, 0, FP8MM_OUT_F32) && rows_vec(dbeta, 0, FP8MM_OUT_F32)));
    const bool pairs = C % 2 == 0 && rows_pairs(x, p.ldx, x_type) && rows_pairs(dy, p.lddy, dy_type) &&
                       (!p.dres || rows_pairs(dres, ldr, x_type)) && (!dx || rows_pairs(dx, ldd, x_type)) &&
                       rows_pairs(gamma, 0, param_type);
    p.groups = vec ? C / 8 : C;
    int P = 0;
    const bool x4 = x_type == FP8MM_OUT_F32, d4 = dy_type == FP8MM_OUT_F32;
    rc = x4 ? (d4 ? launch<4, 4>(p, vec, pairs, sms, s, &P) : launch<4, 2>(p, vec, pairs, sms, s, &P))
            : (d4 ? launch<2, 4>(p, vec, pairs, sms, s, &P) : launch<2, 2>(p, vec, pairs, sms, s, &P));
    if (rc != FP8MM_OK || !dgamma || direct)
        return rc;
    return sum_partials(p, P, dgamma, dbeta, s);
}

}  // extern "C"
