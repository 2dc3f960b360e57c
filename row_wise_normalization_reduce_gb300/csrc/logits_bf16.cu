// logits_bf16.cu -- the kernels over rows of logits for bfloat16 data.
#include "logits.cuh"

namespace nrm {

cudaError_t launch_logit_rows_bf16(const LogitArgs &a, bool policy, bool stream, int sms, cudaStream_t s, Plan *p) {
    return policy ? launch_logit_rows_t<__nv_bfloat16, true>(a, stream, sms, s, p) : launch_logit_rows_t<__nv_bfloat16, false>(a, stream, sms, s, p);
}
cudaError_t launch_logit_grad_bf16(const LogitArgs &a, cudaStream_t s) {
    return launch_logit_grad_t<__nv_bfloat16>(a, s);
}

}  // namespace nrm
