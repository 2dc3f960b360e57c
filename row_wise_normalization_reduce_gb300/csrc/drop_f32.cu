// drop_f32.cu -- the dropout kernels for binary32 data.
#include "drop.cuh"

namespace nrm {

cudaError_t launch_dropout_f32(const DropoutArgs &a, int map, int sms, cudaStream_t s) {
    return launch_dropout_t<float>(a, map, sms, s);
}
cudaError_t launch_drop_fwd_f32(const DropRmsArgs &a, int map, bool longrow, int sms, cudaStream_t s,
                                Plan *p) {
    return launch_drop_fwd_t<float>(a, map, longrow, sms, s, p);
}
cudaError_t launch_drop_bwd_f32(const DropRmsBwdArgs &a, int map, bool longrow, int sms, cudaStream_t s,
                                Plan *p, int64_t *parts) {
    return launch_drop_bwd_t<float>(a, map, longrow, sms, s, p, parts);
}

}  // namespace nrm
