// qk_f32.cu -- head norms with the position rotation for binary32 data.
#include "qk.cuh"

namespace nrm {

cudaError_t launch_qk_f32(const QkArgs &a, int ve, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    return launch_qk_t<float>(a, ve, back, sms, s, p, parts);
}

}  // namespace nrm
