// logits_f32.cu -- the kernels over rows of logits for binary32 data.
#include "logits.cuh"

namespace nrm {

cudaError_t launch_logit_rows_f32(const LogitArgs &a, bool policy, bool stream, int sms, cudaStream_t s, Plan *p) {
    return policy ? launch_logit_rows_t<float, true>(a, stream, sms, s, p) : launch_logit_rows_t<float, false>(a, stream, sms, s, p);
}
cudaError_t launch_logit_grad_f32(const LogitArgs &a, cudaStream_t s) {
    return launch_logit_grad_t<float>(a, s);
}

}  // namespace nrm
