// drop_fold.cu -- the weight gradient's last step: dw[c] = the sum over the
// row partials of column c (one per CTA of the backward, or one per row
// split), added in a fixed order.  16 rows of warps a CTA, 32 columns wide:
// the partials come from L2 where the backward just wrote them, so what
// counts is the number of loads in flight, not bandwidth.
#include "drop.cuh"

namespace nrm {

namespace {

// 16 warps x 20 loads at once cover the 304 partial rows of two CTAs per SM in
// one round trip (2.8 us behind the backward; 16 a time 3.1, 64-bit indices 4.3).
constexpr int kFoldWarps = 16, kFoldLoads = 20;

__global__ void __launch_bounds__(32 * kFoldWarps) dw_fold_kernel(const float *part, float *dw,
                                                                 const int64_t parts, const int64_t N) {
    __shared__ float sh[kFoldWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < N; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + lane;
        float s = 0.f;
        const float *q = part + warp * N + c;
        const int64_t step = N * kFoldWarps;
        for (int left = (int)parts - warp; left > 0; left -= kFoldWarps * kFoldLoads) {
            float v[kFoldLoads];
#pragma unroll
            for (int u = 0; u < kFoldLoads; ++u) {
                v[u] = c < N && u * kFoldWarps < left ? *q : 0.f;
                q += step;
            }
#pragma unroll
            for (int u = 0; u < kFoldLoads; ++u) s += v[u];
        }
        sh[warp][lane] = s;
        __syncthreads();
        if (warp == 0) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kFoldWarps; ++w) t += sh[w][lane];
            if (c < N) dw[c] = t;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_dw_fold(const float *part, float *dw, int64_t parts, int64_t N, cudaStream_t s) {
    const int64_t ctas = (N + 31) / 32;
    return launch_row(dw_fold_kernel, (unsigned)(ctas < 65536 ? ctas : 65536), 32u * kFoldWarps, 0, s, part,
                      dw, parts, N);
}

}  // namespace nrm
