// Routing of FP32 logits.
#include "moe_route.cuh"

namespace deto {

cudaError_t launch_route_f32(const RouteParams &p, cudaStream_t s) { return pick<true>(p, false, s); }
cudaError_t launch_route_bwd_f32(const RouteParams &p, cudaStream_t s) { return pick<true>(p, true, s); }

}  // namespace deto
