// Instances of the block-scaled product whose B operand is a weight (one
// scale for each 128 x 128 tile of it).
#include "fp8_gemm.cuh"

namespace deto {

cudaError_t launch_fp8_wgrad(const Fp8Params &p, int sms, cudaStream_t s);

cudaError_t launch_fp8(const Fp8Params &p, const Fp8Plan &plan, int sms, cudaStream_t s)
{
    if (plan.kind == kFp8Wgrad) return launch_fp8_wgrad(p, sms, s);
    const bool f = p.out_fp32 != 0;
    if (plan.swap) {
        if (plan.tile_m == 16) return f ? run_swap<true, 16>(p, plan.tile_n, sms, s) : run_swap<false, 16>(p, plan.tile_n, sms, s);
        if (plan.tile_m == 32) return f ? run_swap<true, 32>(p, plan.tile_n, sms, s) : run_swap<false, 32>(p, plan.tile_n, sms, s);
        return f ? run_swap<true, 64>(p, plan.tile_n, sms, s) : run_swap<false, 64>(p, plan.tile_n, sms, s);
    }
    if (plan.tile_n == 128) return f ? run_plain<kFp8Rows, true, 128>(p, sms, s) : run_plain<kFp8Rows, false, 128>(p, sms, s);
    return f ? run_plain<kFp8Rows, true, 192>(p, sms, s) : run_plain<kFp8Rows, false, 192>(p, sms, s);
}

}  // namespace deto
