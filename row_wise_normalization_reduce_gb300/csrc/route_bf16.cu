// route_bf16.cu -- routing to experts from bfloat16 logits.
#include "route.cuh"

namespace nrm {

cudaError_t launch_route_bf16(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    return launch_route_t<__nv_bfloat16>(a, back, sms, s, p);
}

}  // namespace nrm
