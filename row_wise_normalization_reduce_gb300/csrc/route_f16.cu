// route_f16.cu -- routing to experts from binary16 logits.
#include "route.cuh"

namespace nrm {

cudaError_t launch_route_f16(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    return launch_route_t<__half>(a, back, sms, s, p);
}

}  // namespace nrm
