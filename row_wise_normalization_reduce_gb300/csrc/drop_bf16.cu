// drop_bf16.cu -- the dropout kernels for bfloat16 data.
#include "drop.cuh"

namespace nrm {

cudaError_t launch_dropout_bf16(const DropoutArgs &a, int map, int sms, cudaStream_t s) {
    return launch_dropout_t<__nv_bfloat16>(a, map, sms, s);
}
cudaError_t launch_drop_fwd_bf16(const DropRmsArgs &a, int map, bool longrow, int sms, cudaStream_t s,
                                Plan *p) {
    return launch_drop_fwd_t<__nv_bfloat16>(a, map, longrow, sms, s, p);
}
cudaError_t launch_drop_bwd_bf16(const DropRmsBwdArgs &a, int map, bool longrow, int sms, cudaStream_t s,
                                Plan *p, int64_t *parts) {
    return launch_drop_bwd_t<__nv_bfloat16>(a, map, longrow, sms, s, p, parts);
}

}  // namespace nrm
