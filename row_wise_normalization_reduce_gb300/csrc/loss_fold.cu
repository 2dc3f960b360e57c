// loss_fold.cu -- the policy loss' last step: the rows' terms added in
// binary64, in an order that depends on their number alone (the same bits
// every time).  One CTA: the terms are 4 bytes a row and just written.
#include "logits.cuh"

namespace nrm {

namespace {

__global__ void __launch_bounds__(1024) loss_fold_kernel(const float *row_loss, float *loss, const int64_t rows) {
    __shared__ double sh[32];
    pdl_wait();
    pdl_launch_dependents();
    double s = 0.0;
    for (int64_t r = threadIdx.x; r < rows; r += 4096) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = r + u * 1024 < rows ? row_loss[r + u * 1024] : 0.f;
        s += (double)v[0] + (double)v[1] + ((double)v[2] + (double)v[3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = sh[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) *loss = (float)s;
    }
}

}  // namespace

cudaError_t launch_loss_fold(const float *row_loss, float *loss, int64_t rows, cudaStream_t s) {
    return launch_row(loss_fold_kernel, 1u, 1024u, 0, s, row_loss, loss, rows);
}

}  // namespace nrm
