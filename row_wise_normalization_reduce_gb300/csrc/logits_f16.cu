// logits_f16.cu -- the kernels over rows of logits for binary16 data.
#include "logits.cuh"

namespace nrm {

cudaError_t launch_logit_rows_f16(const LogitArgs &a, bool policy, bool stream, int sms, cudaStream_t s, Plan *p) {
    return policy ? launch_logit_rows_t<__half, true>(a, stream, sms, s, p) : launch_logit_rows_t<__half, false>(a, stream, sms, s, p);
}
cudaError_t launch_logit_grad_f16(const LogitArgs &a, cudaStream_t s) {
    return launch_logit_grad_t<__half>(a, s);
}

}  // namespace nrm
