// fp8mm_actgrad.cu -- C entry of the activation and bias gradient.
#include "fp8mm_actgrad.cuh"
#include "fp8mm_rows_host.h"

namespace {

using namespace fp8mm_host;
using fp8act::ActGradParams;

// Lanes of a warp across the columns, 8 columns each.
int lanes_for(int64_t N) { return N <= 64 ? 8 : N <= 128 ? 16 : 32; }

// Row slabs of a call on [M, N]: enough CTAs to fill the SMs, each with at
// least a few turns of its warps. Up to six turns go to one slab, whose sums
// need no second launch (32 x 4096 bf16: kernels 5.1 us in slabs, 3.2 in one, a
// call 7.3 and 4.3; 64 x 16384: kernels 6.6 and 8.6).
int64_t slabs_for(int64_t M, int64_t N, int sms)
{
    const int lanes = lanes_for(N);
    const int64_t strips = cdiv(N, 8 * lanes), turn = fp8act::kWarps * (32 / lanes);
    if (M <= 6 * turn)
        return 1;
    // four CTAs fit an SM: up to four whole waves of them
    return std::max<int64_t>(1, std::min<int64_t>({cdiv(M, 2 * turn), static_cast<int64_t>(sms) * 16 / strips, 65535}));
}

// A single slab's sums go straight to dbias (one token of 4096: 1.9 us, through
// a workspace and a second launch 3.5).
int64_t partial_bytes(int64_t slabs, int64_t N)
{
    return slabs == 1 ? 0 : slabs * N * static_cast<int64_t>(sizeof(float));
}

template <int ES, int G, int LANES>
int launch_lanes(const ActGradParams &p, int64_t slabs, cudaStream_t stream)
{
    return launch_grid2(fp8act::act_grad_kernel<ES, G, LANES, (ES == 2 && G > 1) ? 2 : 1>, cdiv(p.N, 8 * LANES), slabs,
                        fp8act::kThreads, stream, "activation gradient launch", p);
}

template <int ES, int G>
int launch(const ActGradParams &p, int64_t slabs, cudaStream_t stream)
{
    switch (lanes_for(p.N)) {
    case 8: return launch_lanes<ES, G, 8>(p, slabs, stream);
    case 16: return launch_lanes<ES, G, 16>(p, slabs, stream);
    default: return launch_lanes<ES, G, 32>(p, slabs, stream);
    }
}

bool shape_ok(int64_t M, int64_t N)
{
    return M >= 0 && N >= 0 && N <= INT32_MAX && M <= (int64_t(1) << 40) / std::max<int64_t>(N, 1);
}

}  // namespace

extern "C" {

int64_t fp8_act_grad_workspace(int64_t M, int64_t N)
{
    if (!shape_ok(M, N))
        return FP8MM_ERR_SHAPE;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc != FP8MM_OK)
        return rc;
    return M == 0 || N == 0 ? 0 : partial_bytes(slabs_for(M, N, sms), N);
}

int fp8_act_grad(const void *dy, int64_t lddy, const void *z, int64_t ldz, int type, int activation, void *dz,
                 int64_t lddz, float *dbias, int64_t M, int64_t N, void *workspace, int64_t workspace_bytes,
                 void *stream)
{
    if (!row_type_known(type) || activation < FP8MM_ACT_NONE || activation > FP8MM_ACT_SILU)
        return FP8MM_ERR_MODE;
    if (!shape_ok(M, N))
        return FP8MM_ERR_SHAPE;
    int rc;
    if ((rc = check_rows(dy, lddy, N, type)) != FP8MM_OK || (rc = check_rows(z, ldz, N, type)) != FP8MM_OK ||
        (rc = check_rows(dz, lddz, N, type)) != FP8MM_OK ||
        (rc = check_rows(dbias, 0, N, FP8MM_OUT_F32)) != FP8MM_OK ||
        (rc = check_rows(workspace, 0, N, FP8MM_OUT_F32)) != FP8MM_OK)
        return rc;
    if (N == 0 || (M == 0 && !dbias) || (!dz && !dbias))
        return FP8MM_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (M == 0) {
        // a sum over no rows
        if ((rc = device_sms(&sms)) != FP8MM_OK)
            return rc;
        const cudaError_t e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s);
        return e == cudaSuccess ? FP8MM_OK : cuda_fail(e, "cudaMemsetAsync(bias gradient)");
    }
    if (!dy || (activation != FP8MM_ACT_NONE && !z))
        return FP8MM_ERR_NULL;
    ActGradParams p{};
    p.dy = dy;
    p.z = activation == FP8MM_ACT_NONE ? nullptr : z;
    p.ldy = lddy > 0 ? lddy : N;
    p.ldz = ldz > 0 ? ldz : N;
    p.type = type;
    p.act = activation;
    p.dz = dz;
    p.ldd = lddz > 0 ? lddz : N;
    p.M = M;
    p.N = N;
    if (dz && ((dz == dy && p.ldd != p.ldy) || (dz == p.z && p.ldd != p.ldz)))
        return FP8MM_ERR_MODE;   // in place: every element over itself
    if ((rc = device_sms(&sms)) != FP8MM_OK)
        return rc;
    const int64_t slabs = slabs_for(M, N, sms);
    if (dbias) {
        const int64_t need = partial_bytes(slabs, N);
        if (need > 0 && !workspace)
            return FP8MM_ERR_NULL;
        if (workspace_bytes < need)
            return FP8MM_ERR_SHAPE;
        p.partial = need > 0 ? static_cast<float *>(workspace) : dbias;
    }
    const bool vec = N % 8 == 0 && rows_vec(dy, p.ldy, type) && (!p.z || rows_vec(z, p.ldz, type)) &&
                     (!dz || rows_vec(dz, p.ldd, type));
    const bool pairs = N % 2 == 0 && rows_pairs(dy, p.ldy, type) && (!p.z || rows_pairs(z, p.ldz, type)) &&
                       (!dz || rows_pairs(dz, p.ldd, type));
    if (type == FP8MM_OUT_F32)
        rc = vec ? launch<4, 8>(p, slabs, s) : launch<4, 1>(p, slabs, s);
    else
        rc = vec ? launch<2, 8>(p, slabs, s) : pairs ? launch<2, 2>(p, slabs, s) : launch<2, 1>(p, slabs, s);
    if (rc != FP8MM_OK || !dbias || slabs == 1)
        return rc;
    fp8rows::PartialSumParams sum{};
    sum.partial = p.partial;
    sum.out0 = dbias;
    sum.C = N;
    sum.P = static_cast<int>(slabs);
    sum.K = 1;
    return launch_grid2(fp8rows::partial_sum_kernel, cdiv(N, 32), 1, fp8rows::kSumThreads, s, "bias sum launch", sum);
}

}  // extern "C"
