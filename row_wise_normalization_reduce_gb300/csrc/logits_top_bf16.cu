// logits_top_bf16.cu -- rows of logits with entropy and alternatives for bfloat16 data.
#include "logits_top.cuh"

namespace nrm {

cudaError_t launch_logit_top_bf16(const TopArgs &a, int sms, cudaStream_t s, Plan *p) {
    return launch_logit_top_t<__nv_bfloat16>(a, sms, s, p);
}
cudaError_t launch_logit_top_grad_bf16(const TopArgs &a, cudaStream_t s) { return launch_logit_top_grad_t<__nv_bfloat16>(a, s); }

}  // namespace nrm
