// logits_top_f16.cu -- rows of logits with entropy and alternatives for binary16 data.
#include "logits_top.cuh"

namespace nrm {

cudaError_t launch_logit_top_f16(const TopArgs &a, int sms, cudaStream_t s, Plan *p) {
    return launch_logit_top_t<__half>(a, sms, s, p);
}
cudaError_t launch_logit_top_grad_f16(const TopArgs &a, cudaStream_t s) { return launch_logit_top_grad_t<__half>(a, s); }

}  // namespace nrm
