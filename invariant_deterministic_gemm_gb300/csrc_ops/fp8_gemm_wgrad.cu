// Instances of the block-scaled product whose operands both carry one scale
// for each row and block (the weight gradient).
#include "fp8_gemm.cuh"

namespace deto {

cudaError_t launch_fp8_wgrad(const Fp8Params &p, const Fp8Plan &plan, int sms, cudaStream_t s)
{
    const bool f = p.out_fp32 != 0;
    if (plan.tile_n == 128) return f ? run_plain<kFp8Wgrad, true, 128>(p, sms, s) : run_plain<kFp8Wgrad, false, 128>(p, sms, s);
    return f ? run_plain<kFp8Wgrad, true, 192>(p, sms, s) : run_plain<kFp8Wgrad, false, 192>(p, sms, s);
}

}  // namespace deto
