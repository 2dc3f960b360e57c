// logits_top_f32.cu -- rows of logits with entropy and alternatives for binary32 data.
#include "logits_top.cuh"

namespace nrm {

cudaError_t launch_logit_top_f32(const TopArgs &a, int sms, cudaStream_t s, Plan *p) {
    return launch_logit_top_t<float>(a, sms, s, p);
}
cudaError_t launch_logit_top_grad_f32(const TopArgs &a, cudaStream_t s) { return launch_logit_top_grad_t<float>(a, s); }

}  // namespace nrm
