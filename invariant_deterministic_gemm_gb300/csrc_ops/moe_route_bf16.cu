// Routing of BF16 logits.
#include "moe_route.cuh"

namespace deto {

cudaError_t launch_route_bf16(const RouteParams &p, cudaStream_t s) { return pick<false>(p, false, s); }
cudaError_t launch_route_bwd_bf16(const RouteParams &p, cudaStream_t s) { return pick<false>(p, true, s); }

}  // namespace deto
