// fp8mm_epilogue.cu -- the matmul kernels with the extended epilogue
// (activation, residual, stored pre-activation; activation gradient), tile
// rows over M. The swapped kernels are in fp8mm_epilogue_swap.cu.
#include "fp8mm_launch.cuh"

namespace fp8mm_host {

int dispatch_epilogue(const Choice &c, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
                      const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> &em, cudaStream_t stream)
{
    if (c.variant == FP8MM_VARIANT_TILE || c.variant == FP8MM_VARIANT_PAIR)
        return dispatch<true, kRowKernels>(c, mp, mq, mo, kp, &em, stream);
    return dispatch_epilogue_swap(c, mp, mq, mo, kp, em, stream);
}

}  // namespace fp8mm_host
