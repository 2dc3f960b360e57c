// qk_f16.cu -- head norms with the position rotation for binary16 data.
#include "qk.cuh"

namespace nrm {

cudaError_t launch_qk_f16(const QkArgs &a, int ve, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    return launch_qk_t<__half>(a, ve, back, sms, s, p, parts);
}

}  // namespace nrm
