// logits.cuh -- the rows of logits [rows, V] at the end of a model: the
// log-probability of one target per row, its gradient, and the clipped policy
// loss.  The reduction is the row softmax's (softmax.cu): one pass with a
// running (max, sum), two pairs merged by rescaling both sums to the larger
// max.  With s the inverse temperature and c = s log2(e):
//
//   m = max_j z_j,  d = sum_j 2^((z_j - m) c),  lse = s m + log d
//   logp = s z_a - lse
//   dz_j = g s (delta_ja - 2^((z_j - m) c) / d)       g: the gradient of logp
//
// The row's policy term needs g before any dz_j, so a row is passed over
// twice.  A row of logits is 64 KB to 600 KB; the second pass of a CTA finds
// in L2 what its first pass read from HBM.
//
// A row takes part ("is live") when its target lies in [0, V) (and, for the
// loss, its weight is not 0); of the others nothing is read and their gradient
// is 0.  A live row without a finite logit (every entry -inf) has no
// distribution: lse = logp = -inf, its gradient is 0 and the loss skips it.
#pragma once

#include <cmath>
#include <cstdint>

#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

constexpr float kLog2e = 1.44269504088896341f;

// 2^x: an error of 2 binary32 ulp; inputs below -126 give 0 (their terms are
// below 2^-126 of the row's largest).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct RowMax {
    float m, d;
};
// A side without elements is (-inf, 0); one whose elements are all NaN is
// (-inf, NaN) and has to stay visible.
__device__ __forceinline__ RowMax rm_merge(RowMax a, RowMax b, float c) {
    if (b.m == -INFINITY && b.d == 0.f) return a;
    if (a.m == -INFINITY && a.d == 0.f) return b;
    const float M = fmaxf(a.m, b.m);
    return RowMax{M, a.d * exp2_fast((a.m - M) * c) + b.d * exp2_fast((b.m - M) * c)};
}
template <int NW>
__device__ __forceinline__ RowMax cta_row_max(RowMax v, float c, float2 *slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = rm_merge(v, RowMax{__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.d, o)}, c);
    if (lane == 0) slot[warp] = make_float2(v.m, v.d);
    __syncthreads();
    const float2 w = slot[lane & (NW - 1)];
    v = RowMax{w.x, w.y};
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1)
        v = rm_merge(v, RowMax{__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.d, o)}, c);
    return v;
}

// log d as a sum of a part in binary64 and a binary32 part below 0.41: d =
// 2^e f with f in [0.75, 1.5), log d = e log 2 + log1p(f - 1).  A binary32
// log would cost the log-probability half an ulp of log d (2.4e-7 at 10).
__device__ __forceinline__ double log_sum(float d) {
    if (!(d < INFINITY)) return (double)d;  // NaN stays NaN
    const int e = ((__float_as_int(d) - 0x3f400000) >> 23);
    const float f = __int_as_float(__float_as_int(d) - (e << 23));
    return fma((double)e, 0.693147180559945309, (double)log1pf(f - 1.f));
}

// exp(q) - q - 1 without the cancellation at small q: its Taylor series to
// q^8 below 1/2 (the next term is under 4e-8 of the sum).
__device__ __forceinline__ float kl_term(float q) {
    if (fabsf(q) < 0.5f) {
        float t = fmaf(q, 1.f / 40320, 1.f / 5040);
        t = fmaf(q, t, 1.f / 720);
        t = fmaf(q, t, 1.f / 120);
        t = fmaf(q, t, 1.f / 24);
        t = fmaf(q, t, 1.f / 6);
        t = fmaf(q, t, 0.5f);
        return q * q * t;
    }
    return expf(q) - q - 1.f;
}

// One row's policy term and its slope in logp.  The clip is decided on the
// logarithm of the ratio, against the logarithms of the bounds in binary64:
// the ratio itself carries expf's rounding.
__device__ __forceinline__ void policy_row(const LogitArgs &a, int64_t row, double logp, float *loss,
                                           float *slope) {
    const float A = a.adv[row], w = a.weight ? a.weight[row] : 1.f;
    const double q = logp - (double)a.old[row];
    const bool held = A > 0.f ? q > a.log_hi : A < 0.f && q < a.log_lo;
    const float free_ = -A * expf((float)q);
    float l = held ? -A * (A > 0.f ? a.ratio_hi : a.ratio_lo) : free_;
    float g = held ? 0.f : free_;
    if (a.ref) {
        const float k = (float)((double)a.ref[row] - logp);
        l = fmaf(a.kl, kl_term(k), l);
        g = fmaf(a.kl, -expm1f(k), g);
    }
    *loss = w * l;
    *slope = w * g;
}

// Elements of a row before its first 16-byte boundary, whole packs after it,
// and what is left: any N and any element alignment.
template <typename T> struct RowCut {
    int head;   // elements before the first pack
    int packs;
    int tail;   // elements after the last
};
template <typename T> __device__ __forceinline__ RowCut<T> cut_row(const T *p, int64_t n) {
    constexpr int V = IO<T>::V;
    RowCut<T> c;
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    c.head = off ? V - off : 0;
    if (c.head > n) c.head = (int)n;
    c.packs = (int)((n - c.head) / V);
    c.tail = (int)(n - c.head) - c.packs * V;
    return c;
}

// 16-byte load of data that may be overwritten in place later.
__device__ __forceinline__ uint4 ld_pack(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
template <typename T> __device__ __forceinline__ void st_pack(T *p, const uint4 &v, bool wide) {
    if (wide) {
        st_stream(p, v);
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                reinterpret_cast<unsigned short *>(p)[i] = (unsigned short)(w[i >> 1] >> 16 * (i & 1));
        }
    }
}

// dz of one element and of a pack: k * 2^((a z + b) c); a, b, c and k are the
// row's.
__device__ __forceinline__ float grad_one(float z, float a, float b, float c, float k) {
    return k * exp2_fast(fmaf(z, a, b) * c);
}
template <typename T>
__device__ __forceinline__ uint4 grad_pack(const uint4 &z, float a, float b, float c, float k) {
    float2 v[IO2<T>::H];
    IO2<T>::unpack(z, v);
#pragma unroll
    for (int i = 0; i < IO2<T>::H; ++i) {
        v[i] = __fmul2_rn(__ffma2_rn(v[i], f2(a), f2(b)), f2(c));
        v[i].x = exp2_fast(v[i].x);
        v[i].y = exp2_fast(v[i].y);
        v[i] = __fmul2_rn(v[i], f2(k));
    }
    return IO2<T>::pack(v);
}

// ---------------------------------------------------------------------------
// One row per cluster of CTAs (1 where rows are many; up to 8 where they are
// few, each CTA a slice of the row's packs, the pairs joined over distributed
// shared memory in rank order).
// ---------------------------------------------------------------------------
constexpr int kLogitThreads = 512;

template <typename T, bool POLICY>
__global__ void __launch_bounds__(kLogitThreads) logit_rows_kernel(const LogitArgs a, const int cs) {
    constexpr int TH = kLogitThreads, NW = TH / 32, V = IO<T>::V, H = IO2<T>::H, U = 8;
    __shared__ float2 slot[2][NW];
    __shared__ float2 pub[2];
    __shared__ float sh[2][2];  // the row's gradient factor; whether it has a gradient
    const int t = threadIdx.x;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    pdl_wait();
    pdl_launch_dependents();
    const float c = a.scale * kLog2e;
    const float gs = POLICY && a.grad_scale ? *a.grad_scale : 1.f;
    // the exchange slots alternate between live rows (each has a barrier; the
    // others have none)
    int parity = 1;
    for (int64_t row = blockIdx.x / cs; row < a.rows; row += gridDim.x / cs) {
        const T *Z = static_cast<const T *>(a.z) + row * a.ldz;
        T *D = POLICY && a.dz ? static_cast<T *>(a.dz) + row * a.lddz : nullptr;
        const int64_t tgt = a.target[row];
        const bool live = tgt >= 0 && tgt < a.V && !(POLICY && a.weight && a.weight[row] == 0.f);
        const RowCut<T> cut = cut_row(Z, a.V);
        const int p0 = (int)((int64_t)cut.packs * rank / cs), p1 = (int)((int64_t)cut.packs * (rank + 1) / cs);
        const T *body = Z + cut.head;
        // the scalar elements of the row, one per thread of the first rank:
        // the head, then the tail
        const int ns = rank == 0 ? cut.head + cut.tail : 0;
        const int64_t sc = t < cut.head ? t : a.V - cut.tail + (t - cut.head);
        float k = 0.f;  // -g s / d
        RowMax r{-INFINITY, 0.f};
        if (live) {
            parity ^= 1;
            const float za = IO<T>::to_f(Z[tgt]);
            if (t < ns) {
                const float z = IO<T>::to_f(Z[sc]);
                r.m = z != z ? -INFINITY : z;
                r.d = exp2_fast((z - (r.m == -INFINITY ? 0.f : r.m)) * c);
            }
            for (int p = p0 + t; p < p1; p += TH * U) {
                uint4 raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * TH < p1) raw[u] = ld_pack(body + (int64_t)(p + u * TH) * V);
                float bm = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (p + u * TH < p1) {
                        float2 v[H];
                        IO2<T>::unpack(raw[u], v);
#pragma unroll
                        for (int h = 0; h < H; ++h) bm = fmaxf(bm, fmaxf(v[h].x, v[h].y));
                    }
                }
                if (bm > r.m) {
                    r.d *= exp2_fast((r.m - bm) * c);
                    r.m = bm;
                }
                const float2 ref = f2(r.m == -INFINITY ? 0.f : -r.m);
                float2 acc = f2(0.f);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (p + u * TH < p1) {
                        float2 v[H];
                        IO2<T>::unpack(raw[u], v);
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            float2 e = __fmul2_rn(__fadd2_rn(v[h], ref), f2(c));
                            e.x = exp2_fast(e.x);
                            e.y = exp2_fast(e.y);
                            acc = __fadd2_rn(acc, e);
                        }
                    }
                }
                r.d += acc.x + acc.y;
            }
            r = cta_row_max<NW>(r, c, slot[parity]);
            if (cs > 1) {
                if (t == 0) pub[parity] = make_float2(r.m, r.d);
                cluster_arrive();
                cluster_wait();
                const int lane = t & 31;
                const float2 mine = lane < cs ? ld_dsmem(&pub[parity], (uint32_t)lane) : make_float2(-INFINITY, 0.f);
                r = RowMax{__shfl_sync(0xffffffffu, mine.x, 0), __shfl_sync(0xffffffffu, mine.y, 0)};
                for (int q = 1; q < cs; ++q)
                    r = rm_merge(r, RowMax{__shfl_sync(0xffffffffu, mine.x, q), __shfl_sync(0xffffffffu, mine.y, q)}, c);
            }
            if (t == 0) {
                const bool empty = r.m == -INFINITY && r.d == 0.f;
                const double ls = empty ? 0.0 : log_sum(r.d);
                const double sm = (double)a.scale * (double)r.m;
                const double logp = empty ? -INFINITY : (double)a.scale * (double)za - sm - ls;
                float l = 0.f, g = 0.f;
                if (POLICY && !empty) policy_row(a, row, logp, &l, &g);
                if (rank == 0) {
                    if (a.logp) a.logp[row] = (float)logp;
                    if (a.lse) a.lse[row] = empty ? -INFINITY : (float)(sm + ls);
                    if (POLICY) a.row_loss[row] = l;
                }
                if (POLICY) {
                    sh[parity][0] = g * gs * a.scale;
                    sh[parity][1] = za;
                }
            }
            if (POLICY && D) {
                __syncthreads();
                const float g = sh[parity][0];
                k = -g / r.d;
                if (g != 0.f) {
                    const bool wide = (reinterpret_cast<uintptr_t>(D + cut.head) & 15) == 0;
                    T *out = D + cut.head;
                    const float m = r.m;
                    // this thread's last pack (before p0 + t: it has none)
                    const int last = p0 + t < p1 ? p1 - 1 - (p1 - 1 - p0 - t) % TH : p0 + t - 1;
                    // newest first: what the first pass read last is still near
                    for (int p = last; p >= p0 + t; p -= TH * 4) {
                        uint4 raw[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (p - u * TH >= p0) raw[u] = ld_pack(body + (int64_t)(p - u * TH) * V);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (p - u * TH >= p0)
                                st_pack(out + (int64_t)(p - u * TH) * V, grad_pack<T>(raw[u], 1.f, -m, c, k), wide);
                    }
                    if (t < ns) D[sc] = IO<T>::from_f(grad_one(IO<T>::to_f(Z[sc]), 1.f, -m, c, k));
                    // the target's own element, by the thread that wrote it just now
                    const int ip = (int)(tgt - cut.head) / V;
                    const bool scalar = tgt < cut.head || tgt >= a.V - cut.tail;
                    const bool owner = scalar ? (t < ns && sc == tgt) : (ip >= p0 && ip < p1 && (ip - p0) % TH == t);
                    if (owner) D[tgt] = IO<T>::from_f(g + grad_one(sh[parity][1], 1.f, -m, c, k));
                }
                if (g != 0.f) continue;
            }
        } else if (t == 0 && rank == 0) {
            if (a.logp) a.logp[row] = 0.f;
            if (a.lse) a.lse[row] = 0.f;
            if (POLICY) a.row_loss[row] = 0.f;
        }
        if (POLICY && D) {  // no gradient: zeros
            const bool wide = (reinterpret_cast<uintptr_t>(D + cut.head) & 15) == 0;
            T *out = D + cut.head;
            for (int p = p0 + t; p < p1; p += TH) st_pack(out + (int64_t)p * V, make_uint4(0, 0, 0, 0), wide);
            if (t < ns) D[sc] = IO<T>::from_f(0.f);
        }
    }
    if (cs > 1) {
        // stay resident until every peer has read this CTA's pairs
        cluster_arrive();
        cluster_wait();
    }
}

// ---------------------------------------------------------------------------
// The gradient for a given slope dlogp and the forward's lse: element-wise.
// A CTA takes one tile of a row.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) logit_grad_kernel(const LogitArgs a, const int tiles) {
    constexpr int TH = 256, V = IO<T>::V, U = 4;
    const int t = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t id = blockIdx.x; id < a.rows * tiles; id += gridDim.x) {
        const int64_t row = id / tiles;
        const int tile = (int)(id - row * tiles);
        const T *Z = static_cast<const T *>(a.z) + row * a.ldz;
        T *D = static_cast<T *>(a.dz) + row * a.lddz;
        const int64_t tgt = a.target[row];
        const float lse = a.lse_in[row];
        const bool in = tgt >= 0 && tgt < a.V;
        const float g = in && lse != -INFINITY ? a.dlogp[row] * a.scale : 0.f;
        const RowCut<T> cut = cut_row(Z, a.V);
        const T *body = Z + cut.head;
        T *out = D + cut.head;
        const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const int base = tile * (TH * U), p0 = base + t;
        const int ns = tile == 0 ? cut.head + cut.tail : 0;
        const int64_t sc = t < cut.head ? t : a.V - cut.tail + (t - cut.head);
        if (g != 0.f) {
            // the target's own element belongs to the thread that owns its pack
            // (or its scalar place)
            const bool scalar = tgt < cut.head || tgt >= a.V - cut.tail;
            const int ip = (int)(tgt - cut.head) / V;
            const bool owner = scalar ? (t < ns && sc == tgt) : (ip >= base && ip < base + TH * U && ip % TH == t);
            const float za = owner ? IO<T>::to_f(Z[tgt]) : 0.f;
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * TH < cut.packs) raw[u] = ld_pack(body + (int64_t)(p0 + u * TH) * V);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * TH < cut.packs)
                    st_pack(out + (int64_t)(p0 + u * TH) * V, grad_pack<T>(raw[u], a.scale, -lse, kLog2e, -g), wide);
            if (t < ns) D[sc] = IO<T>::from_f(grad_one(IO<T>::to_f(Z[sc]), a.scale, -lse, kLog2e, -g));
            if (owner) D[tgt] = IO<T>::from_f(g + grad_one(za, a.scale, -lse, kLog2e, -g));
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * TH < cut.packs)
                    st_pack(out + (int64_t)(p0 + u * TH) * V, make_uint4(0, 0, 0, 0), wide);
            if (t < ns) D[sc] = IO<T>::from_f(0.f);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (logits_<type>.cu).
// ---------------------------------------------------------------------------
template <typename T, bool POLICY>
cudaError_t launch_logit_rows_t(const LogitArgs &a, int sms, cudaStream_t s, Plan *p) {
    // a row over more CTAs while the SMs are not twice covered and each CTA
    // keeps a pack per thread
    int cs = 1;
    while (cs < 8 && a.rows * cs < 2 * (int64_t)sms && a.V / IO<T>::V >= 2 * cs * (int64_t)kLogitThreads) cs *= 2;
    const int64_t most = 0x7fffffff / cs;
    p->kind = cs > 1 ? PLAN_CLUSTER : PLAN_CTA;
    p->threads = kLogitThreads;
    p->packs = 1;
    p->groups = cs > 1 ? cs : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows < most ? a.rows : most) * cs));
    cfg.blockDim = dim3(kLogitThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, logit_rows_kernel<T, POLICY>, a, cs);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename T> cudaError_t launch_logit_grad_t(const LogitArgs &a, cudaStream_t s) {
    const int64_t packs = a.V / IO<T>::V + 1;
    const int64_t tiles = (packs + 1023) / 1024;
    const int64_t n = a.rows * tiles;
    return launch_row(logit_grad_kernel<T>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff), 256u, 0, s, a,
                      (int)tiles);
}

}  // namespace nrm
