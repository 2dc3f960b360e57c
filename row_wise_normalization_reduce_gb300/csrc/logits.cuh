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
// The policy loss' slope g needs the whole row's (m, d), so dz_j can only be
// written once the row has been seen to its end; a row of logits is 2 KB to
// 640 KB.  All of it is bound by HBM (the log-probability reads a row, its
// gradient and the loss read and write one), and which kernel comes nearest
// depends on where the row can wait:
//
//   logit_reg_kernel   in the registers of a warp, a CTA or a cluster of CTAs
//   logit_seg_kernel   nowhere: the log-probability alone needs no second look
//   logit_grad_kernel  the gradient for a slope and lse that are there already
//   logit_rows_kernel  in L2, passed over twice: rows longer than a cluster's
//                      registers
//
// A row takes part ("is live") when its target lies in [0, V) (and, for the
// loss, its weight is not 0); of the others nothing is read and their gradient
// is 0.  A live row without a finite logit (every entry -inf) has no
// distribution: lse = logp = -inf, its gradient is 0 and the loss skips it.
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>

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

// Send a pair to `rank`'s copy of a shared variable and count its 8 bytes on
// that CTA's copy of an mbarrier.
__device__ __forceinline__ void send_pair(float2 *p, float2 v, uint64_t *bar, uint32_t rank) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
                 ::"r"(dsmem_addr(p, rank)), "f"(v.x), "f"(v.y), "r"(dsmem_addr(bar, rank))
                 : "memory");
}

// What a row's factors are computed in: a value as the unevaluated sum of two
// binary32 numbers.  One rounding to binary32 of a log-probability of -12 is
// 5e-7, as much as everything else together, and the clip has a border; the
// binary64 units would take 64 cycles for each operation of this one thread.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// s (z - m) - log d.  The logarithm's range reduction is that of W. J. Cody and
// W. Waite, "Software Manual for the Elementary Functions" (1980), ALOG:
// d = 2^e f with f in [sqrt(1/2), sqrt 2), log d = e log 2 + log f, and log 2 =
// C1 + C2 with C1 = 355/512.  C1 has nine bits and e is below 2^15, so e C1 is
// exact; C2 = log 2 - 355/512 = -2.12194440054690583e-4, rounded to binary32,
// leaves an error of e 2^-37.  f - 1 is exact.  What is not exact is log f and
// two sums of its size: 2^-24 in all, an eighth of the last place of a
// log-probability of -8, and most of it stays in the low part.
__device__ __forceinline__ Two log_prob(float z, float m, float d, float s) {
    const Two x = two_sum(z, -m);
    const float p = __fmul_rn(s, x.hi);
    // no remainder where the product is not finite (z at the type's lowest value
    // and s > 1 suffice)
    if (!(d < INFINITY) || !(fabsf(p) < INFINITY)) return Two{p - logf(d), 0.f};
    const int bits = __float_as_int(d);
    float f = __int_as_float((bits & 0x007fffff) | 0x3f800000), fe = (float)((bits >> 23) - 127);  // d is normal
    if (f >= 1.41421356f) {
        f *= 0.5f;
        fe += 1.f;
    }
    const float pl = fmaf(s, x.lo, fmaf(s, x.hi, -p));
    const Two y = two_sum(p, -fe * (355.f / 512.f));
    const float l = y.lo + (pl - fmaf(fe, -2.12194440e-4f, log1pf(f - 1.f)));
    const float hi = __fadd_rn(y.hi, l);
    return Two{hi, __fadd_rn(__fsub_rn(y.hi, hi), l)};
}

// exp(q) - q - 1 without the cancellation at small q: its Taylor series to
// q^8 below 1/2 (the rest is at most 5.1e-8 of the sum, at q = -1/2).
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
// logarithm of the ratio, against the logarithms of the bounds: the ratio
// itself carries expf's rounding.
struct RowTerms {
    float adv, weight, old, ref;
};
__device__ __forceinline__ RowTerms row_terms(const LogitArgs &a, int64_t row) {
    return RowTerms{a.adv[row], a.weight ? a.weight[row] : 1.f, a.old[row], a.ref ? a.ref[row] : 0.f};
}
__device__ __forceinline__ void policy_row(const LogitArgs &a, const RowTerms &r, Two logp, float *loss,
                                           float *slope) {
    const float q = (logp.hi - r.old) + logp.lo;
    const bool held = r.adv > 0.f ? q > a.log_hi : r.adv < 0.f && q < a.log_lo;
    const float free_ = -r.adv * expf(q);
    float l = held ? -r.adv * (r.adv > 0.f ? a.ratio_hi : a.ratio_lo) : free_;
    float g = held ? 0.f : free_;
    if (a.ref) {
        const float k = (r.ref - logp.hi) - logp.lo;
        l = fmaf(a.kl, kl_term(k), l);
        g = fmaf(a.kl, -expm1f(k), g);
    }
    *loss = r.weight * l;
    *slope = r.weight * g;
}

// Elements of a row before its first 16-byte boundary, whole packs after it,
// and what is left: any N and any element alignment.
template <typename T> struct RowCut {
    int head;   // elements before the first pack
    int packs;
    int tail;   // elements after the last
};
template <typename T> __device__ __forceinline__ RowCut<T> cut_row(const T *p, int64_t n) {
    constexpr uint32_t V = IO<T>::V;
    RowCut<T> c;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (V - 1);
    const uint32_t head = (V - off) & (V - 1), m = (uint32_t)n;  // n < 2^31
    c.head = (int)(head < m ? head : m);
    c.packs = (int)((m - c.head) / V);
    c.tail = (int)((m - c.head) & (V - 1));
    return c;
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
// row's.  BASE: (z - base) in the place of z.
__device__ __forceinline__ float grad_one(float z, float a, float b, float c, float k) {
    return k * exp2_fast(fmaf(z, a, b) * c);
}
template <typename T, bool BASE = false>
__device__ __forceinline__ uint4 grad_pack(const uint4 &z, float a, float b, float c, float k, float base = 0.f) {
    float2 v[IO2<T>::H];
    IO2<T>::unpack(z, v);
#pragma unroll
    for (int i = 0; i < IO2<T>::H; ++i) {
        if (BASE) v[i] = __fadd2_rn(v[i], f2(-base));
        v[i] = __fmul2_rn(__ffma2_rn(v[i], f2(a), f2(b)), f2(c));
        v[i].x = exp2_fast(v[i].x);
        v[i].y = exp2_fast(v[i].y);
        v[i] = __fmul2_rn(v[i], f2(k));
    }
    return IO2<T>::pack(v);
}

// The same as k * 2^(a z + b).
template <typename T> __device__ __forceinline__ uint4 grad_pack1(const uint4 &z, float a, float b, float k) {
    float2 v[IO2<T>::H];
    IO2<T>::unpack(z, v);
#pragma unroll
    for (int i = 0; i < IO2<T>::H; ++i) {
        v[i] = __ffma2_rn(v[i], f2(a), f2(b));
        v[i].x = exp2_fast(v[i].x);
        v[i].y = exp2_fast(v[i].y);
        v[i] = __fmul2_rn(v[i], f2(k));
    }
    return IO2<T>::pack(v);
}

// A live row's scalar outputs and its slope (by one thread; `write`: this is
// the rank that stores them).
template <bool POLICY>
__device__ __forceinline__ void finish_row(const LogitArgs &a, int64_t row, const RowMax &r, float za, bool write,
                                           const RowTerms &terms, float *loss, float *slope) {
    const bool empty = r.m == -INFINITY && r.d == 0.f;
    const Two logp = empty ? Two{-INFINITY, 0.f} : log_prob(za, r.m, r.d, a.scale);
    if (POLICY && !empty) policy_row(a, terms, logp, loss, slope);
    if (write) {
        if (a.logp) a.logp[row] = logp.hi;
        // the log-sum as that of the row's own maximum
        if (!POLICY) {
            const float logd = empty ? -INFINITY : -log_prob(r.m, r.m, r.d, a.scale).hi;
            if (a.lse) a.lse[row] = fmaf(a.scale, r.m, logd);
            if (a.stats) {
                a.stats[2 * row] = r.m;
                a.stats[2 * row + 1] = logd;
            }
        }
        if (POLICY) a.row_loss[row] = *loss;
    }
}

// The scalar outputs of a row that takes no part.
template <bool POLICY> __device__ __forceinline__ void no_row(const LogitArgs &a, int64_t row) {
    if (a.logp) a.logp[row] = 0.f;
    if (!POLICY && a.lse) a.lse[row] = 0.f;
    if (!POLICY && a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.f;
    if (POLICY) a.row_loss[row] = 0.f;
}

// ---------------------------------------------------------------------------
// Streaming plan, any length.  One row per cluster of CTAs (1 where rows are
// many; up to 8 where they are few, each CTA a slice of the row's packs, the
// pairs joined over distributed shared memory in rank order).  The loss reads
// the row again for its gradient, newest packs first; 152 x 4 resident CTAs
// hold more rows than the L2 does, so much of that comes from HBM again: 516 us
// for the loss of 4096 x 131072 bf16 (10 % of the rows out) where the register
// plan takes 303; the log-probability alone 162, in segments 137.
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
                    if (p + u * TH < p1) raw[u] = ld_once(body + (int64_t)(p + u * TH) * V);
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
                float l = 0.f, g = 0.f;
                finish_row<POLICY>(a, row, r, za, rank == 0, POLICY ? row_terms(a, row) : RowTerms{}, &l, &g);
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
                            if (p - u * TH >= p0) raw[u] = ld_once(body + (int64_t)(p - u * TH) * V);
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
            no_row<POLICY>(a, row);
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
// Register plan.  A group of TH threads (a warp, a CTA, or the CTAs of a
// cluster with a slice each) takes a batch of rows.  The row at hand is in
// registers, at most PK packs a thread, so it is read once; the packs of the
// batch's next live row are on their way into shared memory meanwhile (each
// thread copies and reads back its own, so nothing but its own copies has to
// be waited for).
//
// What a cluster has to exchange is one (max, sum) a warp: the sum is taken
// around the warp's own maximum and rescaled, so there is a single exchange a
// row.  The pairs travel as st.async counted on the receiver's mbarrier; with
// barrier.cluster, whose arrival waits for the previous row's stores, 4096 x
// 131072 bf16 took 417 us.
//
// 4096 x 131072 bf16, 30 % of the rows out, loss and gradient: 290 us, 6.3
// TB/s, 93 % of the measured copy rate.
// 152 x 32 warps issue 56 % of the cycles, 26 % of them exponentials.  Rows
// of a few thousand logits are bound by the latency of a row's scalar part
// instead (log, exp, one thread): 8192 x 4096 bf16 31.0 us, 61 %.
// ---------------------------------------------------------------------------
// (max, sum) over a set of pairs, two butterflies: the maximum, then the sums
// rescaled to it.  Every lane gets the same bits.
__device__ __forceinline__ RowMax lanes_row_max(float m, float d, float c) {
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // nothing finite: the pairs are (-inf, 0) or (-inf, NaN), rescaled from 0
    d *= exp2_fast((m - (M == -INFINITY ? 0.f : M)) * c);
    return RowMax{M, warp_sum_all(d)};
}

// Arrival at the cluster barrier that orders nothing: a releasing one would
// wait for the CTA's stores of dlogits to reach L2.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// Accesses under a predicate without a branch: a pack is one instruction, and
// the branches around eight of them cost more than the packs' arithmetic.
__device__ __forceinline__ void cp_async16_if(bool on, void *dst, const void *src) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}"
                 ::"r"(smem_u32(dst)), "l"(src), "r"((uint32_t)on)
                 : "memory");
}
__device__ __forceinline__ void st_stream_if(bool on, void *p, const uint4 &v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};\n\t}"
                 ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((uint32_t)on)
                 : "memory");
}

// A pack of -inf: what a place without a logit holds, it adds nothing.
template <typename T> __device__ __forceinline__ uint4 no_pack() {
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}
// The largest value of a set of packs (NaN are passed over; none: -inf).
// 16-bit types compare in their own type, two at a time.
template <int PK> __device__ __forceinline__ float packs_max(const uint4 (&raw)[PK], float) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < PK; ++k) {
        m = fmaxf(fmaxf(m, __uint_as_float(raw[k].x)), __uint_as_float(raw[k].y));
        m = fmaxf(fmaxf(m, __uint_as_float(raw[k].z)), __uint_as_float(raw[k].w));
    }
    return m;
}
template <int PK, typename T> __device__ __forceinline__ float packs_max(const uint4 (&raw)[PK], T) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    auto as2 = [](const uint32_t &w) { return *reinterpret_cast<const T2 *>(&w); };
    T2 m = __hmax2(__hmax2(as2(raw[0].x), as2(raw[0].y)), __hmax2(as2(raw[0].z), as2(raw[0].w)));
#pragma unroll
    for (int k = 1; k < PK; ++k)
        m = __hmax2(m, __hmax2(__hmax2(as2(raw[k].x), as2(raw[k].y)), __hmax2(as2(raw[k].z), as2(raw[k].w))));
    const float a = IO<T>::to_f(m.x), b = IO<T>::to_f(m.y);
    const float r = fmaxf(a, b);
    return r != r ? -INFINITY : r;
}

// 2^((z - m) c) takes one fused multiply-add an element as 2^(z c - b), b = m c
// rounded; what b's rounding leaves, 2^(b - m c), is one factor for all of
// them.  That factor has to stay near 1: below |m c| = 2^24 the rounding leaves
// at most 1/2, at 1e10 it leaves hundreds (2^-440 times a sum of terms 2^440).
// Beyond that (masked logits of -1e10, -1e30 or the type's lowest value) the
// difference comes first instead.
struct Shift {
    float b, left;
    bool direct;
    __device__ __forceinline__ Shift(float m, float c) {
        const float p = m * c;
        direct = !(fabsf(p) < 16777216.f) && fabsf(m) < INFINITY;
        b = m == -INFINITY || direct ? 0.f : p;
        // (an infinite or NaN m reaches the sum through b)
        left = m == -INFINITY || direct ? 1.f : exp2_fast(-fmaf(m, c, -b));
    }
};
// Sum of 2^((z - m) c) over a set of packs.
template <typename T, int PK>
__device__ __forceinline__ float packs_sum(const uint4 (&raw)[PK], float m, float c) {
    constexpr int H = IO2<T>::H;
    const Shift s(m, c);
    float2 acc = f2(0.f);
    if (!s.direct) {
#pragma unroll
        for (int k = 0; k < PK; ++k) {
            float2 v[H];
            IO2<T>::unpack(raw[k], v);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float2 e = __ffma2_rn(v[h], f2(c), f2(-s.b));
                e.x = exp2_fast(e.x);
                e.y = exp2_fast(e.y);
                acc = __fadd2_rn(acc, e);
            }
        }
        return (acc.x + acc.y) * s.left;
    }
#pragma unroll 1
    for (int k = 0; k < PK; ++k) {
        uint4 q = raw[0];
#pragma unroll
        for (int j = 1; j < PK; ++j)
            if (j == k) q = raw[j];
        float2 v[H];
        IO2<T>::unpack(q, v);
#pragma unroll
        for (int h = 0; h < H; ++h)
            acc = __fadd2_rn(acc, make_float2(exp2_fast((v[h].x - m) * c), exp2_fast((v[h].y - m) * c)));
    }
    return acc.x + acc.y;
}

__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Tries of the wait for pairs still on their way after a wait gave up.
constexpr uint32_t kDrainTries = 1u << 16;

// A row as a thread sees it: its packs (k * TH apart, `mine` of them in all
// counting from its first), and its scalar element of the row's ends, if any.
template <typename T> struct RowView {
    const T *z, *body;
    T *d, *out;
    int p0, p1, mine, ns, head, tail;
    int64_t sc;
    bool wide;
    __device__ __forceinline__ RowView(const LogitArgs &a, int64_t row, int rank, int log_cs, int t) {
        constexpr int V = IO<T>::V;
        z = static_cast<const T *>(a.z) + row * a.ldz;
        d = a.dz ? static_cast<T *>(a.dz) + row * a.lddz : nullptr;
        const RowCut<T> cut = cut_row(z, a.V);
        head = cut.head;
        tail = cut.tail;
        // fits 32 bits: a cluster's rows have at most 8 x 256 x 20 packs, any
        // others are all rank 0's
        p0 = cut.packs * rank >> log_cs;
        p1 = cut.packs * (rank + 1) >> log_cs;
        body = z + head + (int64_t)(p0 + t) * V;
        out = d + head + (int64_t)(p0 + t) * V;
        mine = p1 - p0 - t;
        ns = rank == 0 ? head + tail : 0;
        sc = t < head ? t : a.V - tail + (t - head);
        wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    }
};

template <typename T, bool POLICY, int TH, int PK, int MINB>
__global__ void __launch_bounds__(TH < 128 ? 128 : TH, MINB)
    logit_reg_kernel(const LogitArgs a, const int log_cs, const int batch) {
    constexpr int CTA = TH < 128 ? 128 : TH, G = CTA / TH, NW = TH / 32, V = IO<T>::V, H = IO2<T>::H;
    constexpr int CSMAX = 8, PAIRS = (CSMAX * NW + 31) / 32;
    extern __shared__ __align__(16) uint4 next_row[];  // [PK][CTA]
    // every warp of the cluster sends its pair to every CTA of it, counted on
    // that CTA's barrier
    __shared__ float2 pairs[2][CSMAX * NW];
    __shared__ uint64_t arrived[2];
    __shared__ float sh[2][2];  // the row's gradient factor; the target's logit
    const int t = G > 1 ? threadIdx.x % TH : threadIdx.x, lane = threadIdx.x & 31, warp = t >> 5;
    const int cs = 1 << log_cs, rank = log_cs ? (int)cluster_rank() : 0;
    // the first pair may go to a peer only once its barriers stand: the other
    // half of this cluster barrier is before that
    bool joined = log_cs == 0;
    uint32_t phases = 0;  // bit p: the parity of arrived[p]'s next phase
    bool broken = false;  // a pair never came: no further waits
    if (!joined) {
        if (threadIdx.x == 0) {
            mbar_init(&arrived[0], 1);
            mbar_init(&arrived[1], 1);
            fence_mbar_init();
        }
        __syncwarp();
        cluster_arrive_relaxed();  // the fence has released the barriers' state
    }
    pdl_wait();
    pdl_launch_dependents();
    const float c = a.scale * kLog2e;
    const float gs = POLICY && a.grad_scale ? *a.grad_scale : 1.f;
    int parity = 1;  // the exchange slots alternate between live rows
    const int64_t group = (int64_t)(blockIdx.x >> log_cs) * G + (G > 1 ? threadIdx.x / TH : 0),
                  step = (int64_t)(gridDim.x >> log_cs) * G;
    for (int64_t r0 = group * batch; r0 < a.rows; r0 += step * batch) {
        // lane i keeps the target of row r0 + i
        const bool have = lane < batch && r0 + lane < a.rows;
        const int64_t my_target = have ? a.target[r0 + lane] : -1;
        const bool takes_part = my_target >= 0 && my_target < a.V && !(POLICY && a.weight && a.weight[r0 + lane] == 0.f);
        uint32_t live = __ballot_sync(0xffffffffu, takes_part);
        uint32_t dead = __ballot_sync(0xffffffffu, have && !takes_part);
        float zn = 0.f;  // the next row's scalar element
        auto fetch = [&](int64_t row) {
            const RowView<T> w(a, row, rank, log_cs, t);
            if (t < w.ns) zn = IO<T>::to_f(w.z[w.sc]);
#pragma unroll
            for (int k = 0; k < PK; ++k)
                cp_async16_if(k * TH < w.mine, &next_row[k * CTA + threadIdx.x], w.body + k * TH * V);
        };
        auto zero_fill = [&](const RowView<T> &w) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            if (w.wide) {
#pragma unroll
                for (int k = 0; k < PK; ++k) st_stream_if(k * TH < w.mine, w.out + k * TH * V, z);
            } else {
                for (int k = 0; k * TH < w.mine; ++k) st_pack(w.out + k * TH * V, z, false);
            }
            if (t < w.ns) w.d[w.sc] = IO<T>::from_f(0.f);
        };
        if (live) fetch(r0 + __ffs(live) - 1);
        for (; dead; dead &= dead - 1) {
            const int64_t row = r0 + __ffs(dead) - 1;
            if (t == 0 && rank == 0) no_row<POLICY>(a, row);
            if (POLICY && a.dz) zero_fill(RowView<T>(a, row, rank, log_cs, t));
        }
        while (live) {
            const int at = __ffs(live) - 1;
            const int64_t row = r0 + at, tgt = __shfl_sync(0xffffffffu, my_target, at);
            live &= live - 1;
            parity ^= 1;
            const RowView<T> w(a, row, rank, log_cs, t);
            const float zs = zn;
            float za = 0.f;
            RowTerms terms = {};
            if (t == 0) {
                za = IO<T>::to_f(w.z[tgt]);
                if (POLICY) terms = row_terms(a, row);
            }
            cp_async_wait();
            uint4 raw[PK];
#pragma unroll
            for (int k = 0; k < PK; ++k) {
                raw[k] = no_pack<T>();
                if (k * TH < w.mine) raw[k] = next_row[k * CTA + threadIdx.x];
            }
            float m = packs_max<PK>(raw, T());
            // the maximum is there, so the packs have left shared memory
            asm volatile("" : "+f"(m)::"memory");
            if (live) fetch(r0 + __ffs(live) - 1);
            if (t < w.ns) m = fmaxf(m, zs);
            float d = packs_sum<T, PK>(raw, m, c);
            if (t < w.ns) d += exp2_fast((zs - (m == -INFINITY ? 0.f : m)) * c);
            // Where dlogits replaces the logits, the CTA of a cluster that holds
            // the target overwrites its logit once it has every warp's pair, and
            // every CTA's thread 0 reads that logit from global memory for itself.
            // That read has to be done before its warp sends: the sum takes the
            // logit in as an operand (masked to no bits; log_cs <= 3, which the
            // compiler does not know), every lane's pair is made from that sum,
            // so nothing can be sent before the value is in a register.  The CTA
            // sending the logit with its pair instead took registers that the
            // packs need: 4096 x 131072 bf16 390 us, this 290
            if constexpr (POLICY && TH > 32)
                d = __uint_as_float(__float_as_uint(d) | (__float_as_uint(za) & (uint32_t)(log_cs >> 4)));
            RowMax r = lanes_row_max(m, d, c);
            if constexpr (TH > 32) {
                if (log_cs) {
                    if (!joined) {
                        cluster_wait();
                        joined = true;
                    }
                    uint64_t *bar = &arrived[parity];
                    if (threadIdx.x == 0 && !broken) mbar_arrive_expect_tx(bar, (uint32_t)(cs * NW * sizeof(float2)));
                    // lane q sends the warp's pair to CTA q.  A peer sends the
                    // pair of the next row but one, into the same place, only
                    // after it has this warp's pair of the next row, which
                    // this warp sends after it has read the place
                    if (lane < cs) send_pair(&pairs[parity][rank * NW + warp], make_float2(r.m, r.d), bar, (uint32_t)lane);
                    const uint32_t ph = phases >> parity & 1u;
                    phases ^= 1u << parity;
                    if (!broken && !mbar_wait_bounded(bar, ph, a.wait_limit)) {
                        // the wait gave up: say so, and stay for what is still
                        // on its way here
                        if (a.fault && lane == 0) atomicOr(a.fault, (unsigned)FAULT_WAIT);
                        broken = !mbar_wait_bounded(bar, ph, kDrainTries);
                        if (broken && a.fault && lane == 0) atomicOr(a.fault, (unsigned)FAULT_DRAIN);
                    }
                } else {
                    if (lane == 0) pairs[parity][warp] = make_float2(r.m, r.d);
                    __syncthreads();
                }
                float pm[PAIRS], pd[PAIRS], M = -INFINITY;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const int q = i * 32 + lane;
                    const float2 v = q < cs * NW ? pairs[parity][q] : make_float2(-INFINITY, 0.f);
                    pm[i] = v.x;
                    pd[i] = v.y;
                    M = fmaxf(M, v.x);
                }
                const float mr = M == -INFINITY ? 0.f : M;
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) s += pd[i] * exp2_fast((pm[i] - mr) * c);
                r = lanes_row_max(M, s, c);
            }
            float g = 0.f;
            if (t == 0) {
                float l = 0.f;
                finish_row<POLICY>(a, row, r, za, rank == 0, terms, &l, &g);
                g *= gs * a.scale;
                if (POLICY && TH > 32) {
                    sh[parity][0] = g;
                    sh[parity][1] = za;
                }
            }
            if (POLICY && a.dz) {
                if constexpr (TH > 32) {
                    __syncthreads();
                    g = sh[parity][0];
                    za = sh[parity][1];
                } else {
                    g = __shfl_sync(0xffffffffu, g, 0);
                    za = __shfl_sync(0xffffffffu, za, 0);
                }
                if (g == 0.f) {
                    zero_fill(w);
                    continue;
                }
                const float f = -g / r.d;
                const Shift sf(r.m, c);
                if (w.wide && !sf.direct) {
#pragma unroll
                    for (int k = 0; k < PK; ++k)
                        st_stream_if(k * TH < w.mine, w.out + k * TH * V, grad_pack1<T>(raw[k], c, -sf.b, f * sf.left));
                } else {
#pragma unroll
                    for (int k = 0; k < PK; ++k)
                        if (k * TH < w.mine)
                            st_pack(w.out + k * TH * V,
                                    sf.direct ? grad_pack<T>(raw[k], 1.f, -r.m, c, f)
                                              : grad_pack1<T>(raw[k], c, -sf.b, f * sf.left),
                                    w.wide);
                }
                if (t < w.ns) w.d[w.sc] = IO<T>::from_f(grad_one(zs, 1.f, -r.m, c, f));
                // the target's own element, by the thread that wrote it just now
                const int ip = (int)(tgt - w.head) / V;
                const bool scalar = tgt < w.head || tgt >= a.V - w.tail;
                const bool owner = scalar ? (t < w.ns && w.sc == tgt) : (ip >= w.p0 && ip < w.p1 && (ip - w.p0) % TH == t);
                if (owner) w.d[tgt] = IO<T>::from_f(g + grad_one(za, 1.f, -r.m, c, f));
            }
        }
    }
    if (log_cs) {
        // no CTA leaves before its peers have sent all they send
        if (!joined) cluster_wait();
        cluster_arrive_relaxed();
        cluster_wait();
    }
}

// ---------------------------------------------------------------------------
// Log-probabilities alone, rows longer than a CTA's registers: nothing of the
// row is needed again, so a CTA passes over it in segments of TH x PK packs
// with a running (max, sum) per thread, the next segment (of this row or of
// the batch's next live one) on its way meanwhile; one exchange a row.  Held
// in a cluster's registers instead, a row waits for eight CTAs' exchange:
// 4096 x 131072 bf16 (10 % of the rows out) 136 us against 170, 4096 x 32000
// 37.9 against 46.3, f32 2048 x 50001 60.7 against 70.4.  Reads alone run at
// 7.0 TB/s, a little above the copy rate.
// ---------------------------------------------------------------------------
template <typename T, int TH, int PK, int MINB>
__global__ void __launch_bounds__(TH, MINB) logit_seg_kernel(const LogitArgs a, const int batch) {
    constexpr int NW = TH / 32, V = IO<T>::V;
    extern __shared__ __align__(16) uint4 next_row[];  // [PK][TH]
    __shared__ float2 slot[2][NW];
    const int t = threadIdx.x, lane = t & 31;
    pdl_wait();
    pdl_launch_dependents();
    const float c = a.scale * kLog2e;
    int parity = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * batch; r0 < a.rows; r0 += (int64_t)gridDim.x * batch) {
        const bool have = lane < batch && r0 + lane < a.rows;
        const int64_t my_target = have ? a.target[r0 + lane] : -1;
        const bool takes_part = my_target >= 0 && my_target < a.V;
        uint32_t live = __ballot_sync(0xffffffffu, takes_part);
        if (t < 32 && have && !takes_part) no_row<false>(a, r0 + lane);
        float zn = 0.f;  // the next row's scalar element
        auto fetch = [&](int64_t row, int seg) {
            const RowView<T> w(a, row, 0, 0, t);
            if (seg == 0 && t < w.ns) zn = IO<T>::to_f(w.z[w.sc]);
#pragma unroll
            for (int k = 0; k < PK; ++k) {
                const int at = (seg * PK + k) * TH;
                cp_async16_if(at < w.mine, &next_row[k * TH + t], w.body + (int64_t)at * V);
            }
        };
        if (live) fetch(r0 + __ffs(live) - 1, 0);
        while (live) {
            const int at = __ffs(live) - 1;
            const int64_t row = r0 + at, tgt = __shfl_sync(0xffffffffu, my_target, at);
            live &= live - 1;
            const RowView<T> w(a, row, 0, 0, t);
            float za = 0.f;
            RowMax r{-INFINITY, 0.f};
            if (t < w.ns) {
                const float z = zn;
                r.m = z != z ? -INFINITY : z;
                r.d = exp2_fast((z - (r.m == -INFINITY ? 0.f : r.m)) * c);
            }
            if (t == 0) za = IO<T>::to_f(w.z[tgt]);
            const int segs = w.p1 > 0 ? (w.p1 + TH * PK - 1) / (TH * PK) : 1;
            for (int seg = 0; seg < segs; ++seg) {
                cp_async_wait();
                uint4 raw[PK];
#pragma unroll
                for (int k = 0; k < PK; ++k) {
                    raw[k] = no_pack<T>();
                    if ((seg * PK + k) * TH < w.mine) raw[k] = next_row[k * TH + t];
                }
                float m = packs_max<PK>(raw, T());
                // the maximum is there, so the packs have left shared memory
                asm volatile("" : "+f"(m)::"memory");
                if (seg + 1 < segs)
                    fetch(row, seg + 1);
                else if (live)
                    fetch(r0 + __ffs(live) - 1, 0);
                // a segment below the running maximum is summed from that
                m = fmaxf(m, r.m);
                if (m > r.m) {
                    r.d *= exp2_fast((r.m - m) * c);
                    r.m = m;
                }
                r.d += packs_sum<T, PK>(raw, m, c);
            }
            r = lanes_row_max(r.m, r.d, c);
            if (lane == 0) slot[parity][t >> 5] = make_float2(r.m, r.d);
            __syncthreads();
            const float2 v = lane < NW ? slot[parity][lane] : make_float2(-INFINITY, 0.f);
            r = lanes_row_max(v.x, v.y, c);
            parity ^= 1;
            float l, g;
            if (t == 0) finish_row<false>(a, row, r, za, true, RowTerms{}, &l, &g);
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient for a given slope dlogp and the forward's lse, or (STATS) the
// row's maximum m and log d, lse = s m + log d: element-wise.  With lse the
// rounding of that one number is a factor on the whole row, |lse| 2^-24 of it;
// s (z - m) - log d costs one more subtraction an element, which HBM hides.
// A group of TH threads (the CTA, or a warp where rows are short) takes one
// tile of 4 x TH packs of a row, so there is nothing to wait for but the loads
// of one tile: 2048 x 131072 bf16 137 us, 6.9 TB/s.  An element at its row's
// lse takes exp(s z - lse), no max: lse is the maximum's own upper bound.
// ---------------------------------------------------------------------------
template <typename T, int TH, bool STATS>
__global__ void __launch_bounds__(256) logit_grad_kernel(const LogitArgs a, const int tiles) {
    constexpr int G = 256 / TH, V = IO<T>::V, U = 4;
    const int t = threadIdx.x % TH;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = a.rows * tiles;
    for (int64_t id = (int64_t)blockIdx.x * G + threadIdx.x / TH; id < total; id += (int64_t)gridDim.x * G) {
        const int64_t row = total <= 0xffffffffll ? (int64_t)((uint32_t)id / (uint32_t)tiles) : id / tiles;
        const int tile = (int)(id - row * tiles);
        const T *Z = static_cast<const T *>(a.z) + row * a.ldz;
        T *D = static_cast<T *>(a.dz) + row * a.lddz;
        const int64_t tgt = a.target[row];
        const float lse = STATS ? a.stats_in[2 * row + 1] : a.lse_in[row];  // STATS: log d
        const float top = STATS ? a.stats_in[2 * row] : 0.f;
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
                if (p0 + u * TH < cut.packs) raw[u] = ld_once(body + (int64_t)(p0 + u * TH) * V);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * TH < cut.packs)
                    st_pack(out + (int64_t)(p0 + u * TH) * V,
                            grad_pack<T, STATS>(raw[u], a.scale, -lse, kLog2e, -g, top), wide);
            if (t < ns) D[sc] = IO<T>::from_f(grad_one(IO<T>::to_f(Z[sc]) - top, a.scale, -lse, kLog2e, -g));
            if (owner) D[tgt] = IO<T>::from_f(g + grad_one(za - top, a.scale, -lse, kLog2e, -g));
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
template <typename K, typename... Args>
cudaError_t launch_clusters(K kernel, int64_t rows, int cs, int threads, size_t smem, cudaStream_t s, Args... args) {
    const int64_t most = 0x7fffffff / cs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows < most ? rows : most) * cs));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Rows per batch.  A batch starts with nothing on its way, but few batches
// leave the SMs unevenly loaded where rows take no part: six per resident
// group, and where that leaves less than three rows each, down to two.  Loss and
// gradient, inputs beyond L2, at one row a batch, at three and at four: 1335 x
// 50257 bf16 64.8, 58.2 and 60.8 us, 8192 x 6000 44.8, 42.3 and 42.3; with rows
// enough for six batches, at four, six and twelve of them (10 % of the rows out):
// 4096 x 131072 bf16 308.8, 303.2 and 303.2, 8192 x 32000 170.8, 166.8 and 171.5.
inline int64_t rows_per_batch(int64_t rows, int64_t groups, int64_t least) {
    if (groups < 1) groups = 1;
    const int64_t even = rows / (groups * 6), ahead = rows / (groups * 2);
    const int64_t batch = even >= least ? even : ahead < least ? ahead : least;
    return batch < 1 ? 1 : batch > 32 ? 32 : batch;
}

template <typename T, bool POLICY, int TH, int PK, int MINB>
cudaError_t launch_logit_reg(const LogitArgs &a, int cs, int sms, cudaStream_t s, Plan *p) {
    constexpr int CTA = TH < 128 ? 128 : TH, G = CTA / TH;
    constexpr size_t smem = (size_t)PK * CTA * 16;
    auto kernel = logit_reg_kernel<T, POLICY, TH, PK, MINB>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), CTA, smem, &per_sm);
    if (e != cudaSuccess) return e;
    p->kind = cs > 1 ? PLAN_CLUSTER : TH == 32 ? PLAN_WARP : PLAN_CTA;
    p->threads = CTA;
    p->packs = PK;
    p->groups = cs > 1 ? cs : 0;
    const int64_t groups = (int64_t)sms * per_sm / cs * G;
    const int64_t batch = rows_per_batch(a.rows, groups, 3);
    int log_cs = 0;
    while (1 << log_cs < cs) ++log_cs;
    return launch_clusters(kernel, (a.rows + batch * G - 1) / (batch * G), cs, CTA, smem, s, a, log_cs, (int)batch);
}

template <typename T, int TH, int PK, int MINB>
cudaError_t launch_logit_seg(const LogitArgs &a, int sms, cudaStream_t s, Plan *p) {
    constexpr size_t smem = (size_t)PK * TH * 16;
    auto kernel = logit_seg_kernel<T, TH, PK, MINB>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), TH, smem, &per_sm);
    if (e != cudaSuccess) return e;
    p->kind = PLAN_CTA;
    p->threads = TH;
    p->packs = PK;
    // (a row's own segments follow one another: batches of one row will do, 4096
    // x 32000 bf16 with 10 % of the rows out 37.9 us, of three 41.0)
    const int64_t batch = rows_per_batch(a.rows, (int64_t)sms * per_sm, 1);
    const int64_t n = (a.rows + batch - 1) / batch;
    return launch_row(kernel, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff), (unsigned)TH, smem, s, a, (int)batch);
}

template <typename T, bool POLICY>
cudaError_t launch_logit_rows_t(const LogitArgs &a, bool stream, int sms, cudaStream_t s, Plan *p) {
    const int64_t packs = a.V / IO<T>::V;
    // The fewest threads that hold the row, while rows are enough for every SM:
    // what a row costs beside its packs (the exchange, the scalar part) costs a
    // warp least.  Loss and gradient of 8192 rows bf16, by a warp and by a CTA
    // of 128: 1000 logits 10.7 and 35.4 us, 2501 21.0 and 37.5; by a CTA of 128
    // and the next larger: 4096 x 8192 bf16 26.1 and 29.9, f32 4096 x 4096 24.7
    // and 26.1.  With 304 rows of 2501 a warp is still ahead (5.0 us, a CTA of
    // 256 6.1); with 64 rows of 4000 the CTA is (log-probability 2.4, a warp
    // 2.7).  The CTAs per SM are those that the registers of the packs leave:
    // without that bound the compiler took 172 for sixteen packs (8192 x 4096
    // 37.6 us, 31.0 with 128).  More CTAs a row than its packs need do not help:
    // 200 x 16000 bf16 takes 0.7 us more by two.
    if (!stream) {
        if (packs <= 32 * 4) return launch_logit_reg<T, POLICY, 32, 4, 8>(a, 1, sms, s, p);
        if (a.rows >= 2 * (int64_t)sms) {
            if (packs <= 32 * 8) return launch_logit_reg<T, POLICY, 32, 8, 6>(a, 1, sms, s, p);
            if (packs <= 32 * 12) return launch_logit_reg<T, POLICY, 32, 12, 5>(a, 1, sms, s, p);
            if (packs <= 32 * 16) return launch_logit_reg<T, POLICY, 32, 16, (POLICY ? 4 : 5)>(a, 1, sms, s, p);
            if (packs <= 128 * 8) return launch_logit_reg<T, POLICY, 128, 8, 8>(a, 1, sms, s, p);
            if (!POLICY && packs > 256 * 8) return launch_logit_seg<T, 256, 8, 4>(a, sms, s, p);
        }
        int cs = 1;
        while (cs < 8 && packs > 256 * 8 * cs) cs *= 2;
        // packs that a CTA has room for and the row does not fill cost their
        // instructions all the same, so a CTA is no larger than the slice needs:
        // 6710 x 10001 bf16 by 160 threads 52.7 us, by 256 65.6; 1365 x 49152
        // by 192 52.2 and 59.1; 1335 x 50257 by 224 58.2 and 60.9.  With less
        // than four rows or slices for each resident CTA the larger one is
        // ahead (333 x 50001 f16 16.9 us, by 224 17.9).  The strides stay
        // constants: with the CTA's size read at run time 4096 x 131072 took
        // 344 us, not 289
        if (a.rows * cs >= 16 * (int64_t)sms) {
            if (packs <= 160 * 8 * cs) return launch_logit_reg<T, POLICY, 160, 8, 6>(a, cs, sms, s, p);
            if (packs <= 192 * 8 * cs) return launch_logit_reg<T, POLICY, 192, 8, 5>(a, cs, sms, s, p);
            if (packs <= 224 * 8 * cs) return launch_logit_reg<T, POLICY, 224, 8, 4>(a, cs, sms, s, p);
        }
        if (packs <= 256 * 8 * cs) return launch_logit_reg<T, POLICY, 256, 8, 4>(a, cs, sms, s, p);
        // longer rows: more packs a thread, fewer CTAs per SM.  1024 x 150001
        // bf16 at ten packs 125 us, twelve 132, by 512 threads at eight 168;
        // f32 1024 x 120000 at sixteen 160 and 182; 700 x 151936 at twenty 141,
        // in the streaming plan 197
        if (packs <= 8 * 256 * 10) return launch_logit_reg<T, POLICY, 256, 10, 3>(a, 8, sms, s, p);
        if (packs <= 8 * 256 * 12) return launch_logit_reg<T, POLICY, 256, 12, 3>(a, 8, sms, s, p);
        if (packs <= 8 * 256 * 16) return launch_logit_reg<T, POLICY, 256, 16, 2>(a, 8, sms, s, p);
        if (packs <= 8 * 256 * 20) return launch_logit_reg<T, POLICY, 256, 20, 2>(a, 8, sms, s, p);
    }
    // a row over more CTAs while the SMs are not twice covered and each CTA
    // keeps a pack per thread
    int cs = 1;
    while (cs < 8 && a.rows * cs < 2 * (int64_t)sms && packs >= 2 * cs * (int64_t)kLogitThreads) cs *= 2;
    p->kind = PLAN_GENERIC;
    p->threads = kLogitThreads;
    p->packs = 1;
    p->groups = cs > 1 ? cs : 0;
    return launch_clusters(logit_rows_kernel<T, POLICY>, a.rows, cs, kLogitThreads, 0, s, a, cs);
}

template <typename T, int TH, bool STATS> cudaError_t launch_logit_grad_g(const LogitArgs &a, cudaStream_t s) {
    constexpr int G = 256 / TH;
    const int64_t packs = a.V / IO<T>::V + 1;
    const int64_t tiles = (packs + 4 * TH - 1) / (4 * TH);
    const int64_t n = (a.rows * tiles + G - 1) / G;
    return launch_row(logit_grad_kernel<T, TH, STATS>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff), 256u, 0, s, a,
                      (int)tiles);
}
// Rows of up to 512 packs by warps: 8192 x 1000 bf16 5.8 us, by CTAs 17.4; 8192
// x 4096 23.3 and 23.9; at 750 packs (8192 x 6000) 32.7 and 30.9.
template <typename T> cudaError_t launch_logit_grad_t(const LogitArgs &a, cudaStream_t s) {
    const bool warps = a.V / IO<T>::V <= 512;
    if (a.stats_in) return warps ? launch_logit_grad_g<T, 32, true>(a, s) : launch_logit_grad_g<T, 256, true>(a, s);
    return warps ? launch_logit_grad_g<T, 32, false>(a, s) : launch_logit_grad_g<T, 256, false>(a, s);
}

}  // namespace nrm
