// qk_bf16.cu -- head norms with the position rotation for bfloat16 data.
#include "qk.cuh"

namespace nrm {

cudaError_t launch_qk_bf16(const QkArgs &a, int ve, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    return launch_qk_t<__nv_bfloat16>(a, ve, back, sms, s, p, parts);
}

}  // namespace nrm
