// qk_fold.cu -- the last step of the head norms' weight gradients: the CTAs'
// partial rows [parts][2][D] added up in a fixed order, the first D columns into
// dwq and the others into dwk.  As in drop_fold.cu the partials come from L2,
// and the loads in flight are what counts: 16 warps over the rows, 32 columns.
#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

namespace {

constexpr int kFoldWarps = 16, kFoldLoads = 20;

__global__ void __launch_bounds__(32 * kFoldWarps) qk_fold_kernel(const float *part, float *dwq, float *dwk,
                                                                 const int parts, const int D) {
    __shared__ float sh[kFoldWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float *const dw = c < D ? dwq : dwk;
    const bool on = c < 2 * D && dw;
    float s = 0.f;
    for (int r0 = warp; r0 < parts; r0 += kFoldWarps * kFoldLoads) {
        float v[kFoldLoads];
#pragma unroll
        for (int u = 0; u < kFoldLoads; ++u) {
            const int r = r0 + u * kFoldWarps;
            v[u] = on && r < parts ? part[(int64_t)r * 2 * D + c] : 0.f;
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
        if (on) dw[c < D ? c : c - D] = t;
    }
}

}  // namespace

cudaError_t launch_qk_fold(const float *part, float *dwq, float *dwk, int64_t parts, int D, cudaStream_t s) {
    return launch_row(qk_fold_kernel, (unsigned)((2 * D + 31) / 32), 32u * kFoldWarps, 0, s, part, dwq, dwk,
                      (int)parts, D);
}

}  // namespace nrm
