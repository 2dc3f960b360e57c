// route_f32.cu -- routing to experts from binary32 logits.
#include "route.cuh"

namespace nrm {

cudaError_t launch_route_f32(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    return launch_route_t<float>(a, back, sms, s, p);
}

}  // namespace nrm
