// Instances of the block-scaled product whose operands both carry one scale
// for each row and block (the weight gradient).
#include "fp8_gemm.cuh"

namespace deto {

cudaError_t launch_fp8_wgrad(const Fp8Params &p, int sms, cudaStream_t s)
{
    return p.out_fp32 ? run_plain<kFp8Wgrad, true, 192>(p, sms, s) : run_plain<kFp8Wgrad, false, 192>(p, sms, s);
}

}  // namespace deto
