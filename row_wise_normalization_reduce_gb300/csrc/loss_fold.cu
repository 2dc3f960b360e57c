// loss_fold.cu -- the policy loss' last step: the rows' terms added up, in an
// order that depends on their number alone (the same bits every time).  One
// CTA: the terms are 4 bytes a row and just written.  The sum is the
// unevaluated sum of two binary32 numbers, 46 bits: in binary64, of which an SM
// adds two a cycle, the loss of 8192 x 1000 bf16 took 16.6 us instead of 11.2.
#include "logits.cuh"

namespace nrm {

namespace {

__global__ void __launch_bounds__(1024) loss_fold_kernel(const float *row_loss, float *loss, const int64_t rows) {
    __shared__ float2 sh[32];
    pdl_wait();
    pdl_launch_dependents();
    Two s{0.f, 0.f};
    auto add = [&s](float hi, float lo) {
        const Two t = two_sum(s.hi, hi);
        s = Two{t.hi, s.lo + (lo + t.lo)};
    };
    auto add_lanes = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add(__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o));
    };
    for (int64_t r = threadIdx.x; r < rows; r += 4096) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = r + u * 1024 < rows ? row_loss[r + u * 1024] : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) add(v[u], 0.f);
    }
    add_lanes();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(s.hi, s.lo);
    __syncthreads();
    if (threadIdx.x < 32) {
        s = Two{sh[threadIdx.x].x, sh[threadIdx.x].y};
        add_lanes();
        // an infinite or NaN sum has no remainder
        if (threadIdx.x == 0) *loss = fabsf(s.hi) < INFINITY ? s.hi + s.lo : s.hi;
    }
}

}  // namespace

cudaError_t launch_loss_fold(const float *row_loss, float *loss, int64_t rows, cudaStream_t s) {
    return launch_row(loss_fold_kernel, 1u, 1024u, 0, s, row_loss, loss, rows);
}

}  // namespace nrm
