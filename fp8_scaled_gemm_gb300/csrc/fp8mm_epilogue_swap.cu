// fp8mm_epilogue_swap.cu -- the matmul kernels with the extended epilogue and
// swapped operands (skinny M).
#include "fp8mm_launch.cuh"

namespace fp8mm_host {

int dispatch_epilogue_swap(const Choice &c, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mo,
                           const fp8mm::KernelParams &kp, const fp8mm::EpiMaps<true> &em, cudaStream_t stream)
{
    return dispatch<true, kSwapKernels>(c, mp, mq, mo, kp, &em, stream);
}

}  // namespace fp8mm_host
