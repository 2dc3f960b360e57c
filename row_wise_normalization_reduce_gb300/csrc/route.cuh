// route.cuh -- routing of tokens to experts.  A token's logits x become scores
// s = softmax(x) or sigmoid(x); what is chosen by is c = s + bias.  Of G groups of
// neighbouring experts the top_groups with the largest sums of their group_top
// best c stay, in those the k largest c are taken, ties going to the lowest
// index; the weights are scale s, divided by the sum of the chosen s if wanted.
//
// One warp a token; a lane holds up to PL neighbouring experts, and the lanes of
// a group lie together, so that lane order is expert order.  A router's rows are
// short (64 to 1024 logits) and the kernel is bound by the instructions of the
// selection, not by HBM, so the selection works on one 32-bit key an expert:
//
//   key = (c in 22-bit fixed point below the row's largest) 2^10 + 1023 - expert
//
// A lane sorts its keys (two instructions an exchange), and each place takes one
// redux.max over the lanes' heads.  The fixed point and binary32's own error can
// put two experts in the wrong order only where their keys are a few steps
// apart.  Such tokens are found afterwards by the gaps between neighbouring
// places: the few experts in question are then compared in 64 bits, one a lane,
// and where a border between groups is that near the whole token is done again
// in 64 bits.  Equal logits with equal biases are equal, not near.
//
// Without a bias and without sums over two experts the order of c is that of x;
// 16-bit logits then fit the key as they are and nothing is in question.
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

constexpr int kRouteThreads = 256;
constexpr int kIdxBits = 10, kIdxMask = (1 << kIdxBits) - 1;  // experts: at most 1024
constexpr float kRouteLog2e = 1.44269504088896341f;
static_assert(kRouteMaxExperts == 1 << kIdxBits, "an expert's index fits the key");

__device__ __forceinline__ uint32_t ordered32(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 counts as 0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered32(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t ordered64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// Descending order of N keys: K. E. Batcher's odd-even merge network.
template <int N> __device__ __forceinline__ void sort_desc(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int j = i - q % p;
                if (j >= 0 && i + q < N && (j / q) % 2 == 0 && i / (2 * p) == (i + q) / (2 * p)) {
                    const uint32_t hi = max(k[i], k[i + q]), lo = min(k[i], k[i + q]);
                    k[i] = hi;
                    k[i + q] = lo;
                }
            }
}

// Where a lane's experts lie: `n` of them from `first`.
struct RouteLane {
    int first, n;
    __device__ __forceinline__ RouteLane(const RouteArgs &a, int lane) {
        const int g = lane >> a.log_lanes, at = (lane & ((1 << a.log_lanes) - 1)) * a.per_lane;
        first = g * a.group_size + at;
        n = g < a.groups ? min(a.per_lane, a.group_size - at) : 0;
        if (n < 0) n = 0;
    }
};

template <typename T, int PL>
__device__ __forceinline__ void route_load(const RouteArgs &a, const T *row, const RouteLane &r, float (&x)[PL]) {
    constexpr int V = PL < IO<T>::V ? PL : IO<T>::V;
    if (a.wide) {  // whole packs, PL experts a lane
        using Raw = typename std::conditional<V * sizeof(T) == 16, uint4,
                                              typename std::conditional<V * sizeof(T) == 8, uint2, uint32_t>::type>::type;
        union Words {
            Raw r;
            T t[V];
            __device__ __forceinline__ Words() {}
        } w[PL / V];
        if (r.n > 0) {
#pragma unroll
            for (int i = 0; i < PL / V; ++i) w[i].r = *reinterpret_cast<const Raw *>(row + r.first + i * V);
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) x[i] = r.n > 0 ? IO<T>::to_f(w[i / V].t[i % V]) : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) x[i] = i < r.n ? IO<T>::to_f(row[r.first + i]) : -INFINITY;
    }
}

__device__ __forceinline__ float route_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float route_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ double warp_max64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A token's largest logit and the sum of exp(x - it), in 64 bits.
template <typename T> __device__ __forceinline__ void route_softmax64(const RouteArgs &a, const T *row, int lane, double *m,
                                                                      double *d) {
    double top = -INFINITY, sum = 0.0;
    for (int e = lane; e < a.experts; e += 32) top = fmax(top, (double)IO<T>::to_f(row[e]));
    top = warp_max64(top);
    for (int e = lane; e < a.experts; e += 32) sum += exp((double)IO<T>::to_f(row[e]) - top);
    *m = top;
    *d = warp_sum64(sum);
}
// What one expert is chosen by.
__device__ __forceinline__ double route_choice64(const RouteArgs &a, float x, int e, double m, double d) {
    const double s = a.softmax ? exp((double)x - m) / d : 1.0 / (1.0 + exp(-(double)x));
    return x == -INFINITY ? -INFINITY : a.bias ? s + (double)a.bias[e] : s;
}

// The whole selection in 64 bits.  Lane r returns the expert at place r, or -1.
template <typename T, int PL>
__device__ __noinline__ int route_exact(const RouteArgs &a, const T *row, int lane) {
    const RouteLane r(a, lane);
    const uint64_t none = ordered64(-INFINITY);
    double m = 0.0, d = 1.0;
    if (a.softmax && a.by_score) route_softmax64(a, row, lane, &m, &d);
    uint64_t key[PL];
    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        double c = -INFINITY;
        if (i < r.n) {
            const float x = IO<T>::to_f(row[r.first + i]);
            c = a.by_score ? route_choice64(a, x, r.first + i, m, d) : (double)x;
            if (c != c) c = -INFINITY;
        }
        key[i] = ordered64(c);
        if (c > b1) {
            b2 = b1;
            b1 = c;
        } else if (c > b2) {
            b2 = c;
        }
    }
    if (a.top_groups < a.groups) {
        const int lanes = 1 << a.log_lanes;
        for (int o = 1; o < lanes; o <<= 1) {
            const double c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = c1 > b1 ? fmax(b1, c2) : fmax(b2, c1);
            b1 = fmax(b1, c1);
        }
        const double worth = a.group_top > 1 && b2 > -INFINITY ? b1 + b2 : b1;
        int rank = 0;
        const int g = lane >> a.log_lanes;
        for (int h = 0; h < a.groups; ++h) {
            const double w = __shfl_sync(0xffffffffu, worth, h << a.log_lanes);
            if (w > worth || (w == worth && h < g)) ++rank;
        }
        if (rank >= a.top_groups) {
#pragma unroll
            for (int i = 0; i < PL; ++i) key[i] = none;
        }
    }
    int mine = -1;
    for (int p = 0; p < a.k; ++p) {
        uint64_t best = none;
        int at = -1;
#pragma unroll
        for (int i = PL - 1; i >= 0; --i)
            if (key[i] > none && key[i] >= best) {
                best = key[i];
                at = i;
            }
        uint64_t top = best;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t v = __shfl_xor_sync(0xffffffffu, top, o);
            top = v > top ? v : top;
        }
        const uint32_t who = __ballot_sync(0xffffffffu, best == top && at >= 0);
        if (!who) break;
        const int src = __ffs(who) - 1, id = __shfl_sync(0xffffffffu, r.first + at, src);
        if (lane == p) mine = id;
        if (lane == src) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (i == at) key[i] = none;
        }
    }
    return mine;
}

template <typename T, int PL>
__global__ void __launch_bounds__(kRouteThreads) route_fwd_kernel(const RouteArgs a) {
    constexpr int LIST = PL < 8 ? PL : 8;
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const RouteLane r(a, lane);
    const bool limited = a.top_groups < a.groups;
    // 16-bit logits that order by themselves go into the key whole
    const bool whole = sizeof(T) == 2 && !a.by_score;
    float bias[PL];
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int i = 0; i < PL; ++i) bias[i] = a.bias && i < r.n ? a.bias[r.first + i] : 0.f;
    const int64_t step = (int64_t)gridDim.x * (kRouteThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5); t < a.tokens; t += step) {
        const T *row = static_cast<const T *>(a.x) + t * a.ldx;
        float x[PL];
        route_load<T, PL>(a, row, r, x);
        // the softmax' maximum and sum, where they are needed
        float m = 0.f, d = 1.f;
        if (a.softmax && a.need_sum) {
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < PL; ++i) m = fmaxf(m, x[i]);
            m = from_ordered32(__reduce_max_sync(ALL, ordered32(m)));
            const float mr = m == -INFINITY ? 0.f : m;
            d = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) d += route_exp2((x[i] - mr) * kRouteLog2e);
            d = warp_sum_all(d);
            m = mr;
        }
        if (a.scores) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (i < r.n)
                    a.scores[t * a.experts + r.first + i] =
                        x[i] == -INFINITY ? 0.f : a.softmax ? expf(x[i] - m) / d : 1.f / (1.f + expf(-x[i]));
        }
        // keys, largest first
        uint32_t key[PL];
        float near_ = 0.f;  // keys no further apart than this are in question
        bool again = false; // the whole token is
        if (whole) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                key[i] = x[i] > -INFINITY ? (ordered32(x[i]) >> 16 << kIdxBits) + (uint32_t)(kIdxMask - (r.first + i)) : 0u;
            if (std::is_same<T, __half>::value) {  // binary16 keeps more bits than a binary32's upper half
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const uint32_t b = __half_as_ushort(__float2half_rn(x[i] + 0.f));
                    key[i] = x[i] > -INFINITY ? ((b & 0x8000u ? ~b & 0xffffu : b | 0x8000u) << kIdxBits) +
                                                    (uint32_t)(kIdxMask - (r.first + i))
                                              : 0u;
                }
            }
        } else {
            float top = -INFINITY;
            if (a.by_score) {
                const float inv = 1.f / d;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const float s = a.softmax ? route_exp2((x[i] - m) * kRouteLog2e) * inv
                                              : route_rcp(1.f + route_exp2(x[i] * -kRouteLog2e));
                    x[i] = x[i] == -INFINITY ? -INFINITY : s + bias[i];
                }
            }
#pragma unroll
            for (int i = 0; i < PL; ++i) top = fmaxf(top, x[i]);
            top = from_ordered32(__reduce_max_sync(ALL, ordered32(top)));
            // scores lie within 1 of each other; logits are taken 16 below the largest
            const float S = a.by_score ? 4194300.f : 262143.f;
            again = top == INFINITY;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const float q = fmaxf(fmaf(x[i] - top, S, 8388608.f + 4194303.f), 8388609.f);
                key[i] = x[i] > -INFINITY
                             ? (__float_as_uint(q) << kIdxBits) + (uint32_t)(kIdxMask - (r.first + i))
                             : 0u;
            }
            // A sigmoid is good to 3e-7 (the exponent's argument, ex2, rcp), a
            // softmax to 6e-7 of the largest and half a step for each addition
            // of its sum; adding the bias and taking the difference to the
            // largest cost half a step of their results each, the fixed point one
            // step of its own.
            const float score = a.softmax ? (6e-7f + 6e-8f * (PL + 6)) / d : 3e-7f;
            near_ = a.by_score ? 2.f * S * (score + 1.2e-7f * (fabsf(top) + 1.f)) + 2.f : 2.f;
        }
        sort_desc<PL>(key);
        if (limited) {
            uint32_t b1 = key[0] >> kIdxBits, b2 = PL > 1 ? key[PL > 1 ? 1 : 0] >> kIdxBits : 0u;
            for (int o = 1; o < 1 << a.log_lanes; o <<= 1) {
                const uint32_t c1 = __shfl_xor_sync(ALL, b1, o), c2 = __shfl_xor_sync(ALL, b2, o);
                b2 = max(min(b1, c1), max(b2, c2));
                b1 = max(b1, c1);
            }
            const bool two = a.group_top > 1;
            const uint32_t worth = two ? b1 + b2 : b1;
            int rank = 0;
            const int g = lane >> a.log_lanes;
            for (int h = 0; h < a.groups; ++h) {
                const uint32_t w = __shfl_sync(ALL, worth, h << a.log_lanes);
                rank += w > worth || (w == worth && h < g);
            }
            const bool keep = g < a.groups && rank < a.top_groups;
            if (!whole) {
                const uint32_t least = __reduce_min_sync(ALL, keep ? worth : ALL);
                const uint32_t most = __reduce_max_sync(ALL, keep || g >= a.groups ? 0u : worth);
                // too near; or a kept group owes its place to a value below the fixed point's range
                const bool low = keep && (b1 == 1u || (two && b2 == 1u));
                again = again || (most > 0u && (float)(least - most) <= (two ? 2.f : 1.f) * near_) ||
                        __any_sync(ALL, low);
            }
            if (!keep) {
#pragma unroll
                for (int i = 0; i < PL; ++i) key[i] = 0u;
            }
        }
        // places: the k largest, and those that may belong among them
        uint32_t list[LIST + 1], mine = 0u;
#pragma unroll
        for (int i = 0; i < LIST; ++i) list[i] = key[i];
        list[LIST] = 0u;
        // a lane whose list ran out may hold more
        int left = PL > LIST && key[PL > LIST ? LIST : 0] ? LIST : PL + 1;
        uint32_t last = 0u;  // the k-th place
        int places = 0;
        while (!again) {
            const uint32_t w = __reduce_max_sync(ALL, list[0]);
            if (w == 0u) break;
            if (places >= a.k && (whole || (float)((last >> kIdxBits) - (w >> kIdxBits)) > near_)) break;
            if (places == 32) {  // more in question than lanes
                again = true;
                break;
            }
            if (places == a.k - 1) last = w;
            if (lane == places) mine = w;
            ++places;
            if (list[0] == w) {
#pragma unroll
                for (int i = 0; i < LIST; ++i) list[i] = list[i + 1];
                --left;
            }
            if (PL > LIST && !(whole && places == a.k)) again = __any_sync(ALL, left == 0);
        }
        int id = mine ? kIdxMask - (int)(mine & kIdxMask) : -1;
        float xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
        if (!whole && !again) {
            const float bs = a.bias && id >= 0 ? a.bias[id] : 0.f;
            const uint32_t up = __shfl_up_sync(ALL, mine, 1);
            const float xu = __shfl_up_sync(ALL, xs, 1), bu = __shfl_up_sync(ALL, bs, 1);
            const bool close = lane > 0 && id >= 0 && (float)((up >> kIdxBits) - (mine >> kIdxBits)) <= near_ &&
                               !(xs == xu && bs == bu);
            if (__any_sync(ALL, close)) {
                // one expert a lane in 64 bits, and its rank among them
                double ms = 0.0, ds = 1.0;
                if (a.softmax && a.by_score) route_softmax64(a, row, lane, &ms, &ds);
                double c = -INFINITY;
                if (id >= 0) c = a.by_score ? route_choice64(a, xs, id, ms, ds) : (double)xs;
                const uint64_t ck = id >= 0 ? ordered64(c) : 0ull;
                int rank = 0;
                for (int p = 0; p < places; ++p) {
                    const uint64_t o = __shfl_sync(ALL, ck, p);
                    const int oid = __shfl_sync(ALL, id, p);
                    rank += o > ck || (o == ck && oid < id);
                }
                // lane `rank` takes the expert: who has the rank of this lane?
                int src = lane;
                for (int p = 0; p < places; ++p)
                    if (__shfl_sync(ALL, rank, p) == lane) src = p;
                id = __shfl_sync(ALL, id, src);
                xs = __shfl_sync(ALL, xs, src);
            }
        }
        if (again) {
            id = route_exact<T, PL>(a, row, lane);
            xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
        }
        const bool have = lane < a.k && id >= 0;
        // The chosen scores.  Renormalised softmax scores need no sum over all, and
        // are taken from the largest of the chosen: none of it underflows.
        float w;
        if (a.softmax) {
            if (a.renorm) m = from_ordered32(__reduce_max_sync(ALL, ordered32(have ? xs : -INFINITY)));
            w = !have ? 0.f : a.renorm ? expf(xs - m) : expf(xs - m) / d;
        } else {
            w = have ? 1.f / (1.f + expf(-xs)) : 0.f;
        }
        if (a.renorm) {
            const float sum = warp_sum_all(w);
            w = sum == 0.f ? 0.f : w / sum;
        }
        if (lane < a.k) {
            a.weights[t * a.k + lane] = w * a.scale;
            a.ids[t * a.k + lane] = have ? id : -1;
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient of the logits.  With d_i the gradient of chosen weight i times
// scale, s_i its score and S the chosen scores' sum, the scores' gradients are
//   ds_i = d_i,  or renormalised  (d_i - sum_j d_j s_j / S) / S,
// plus dscores on every expert, and
//   softmax  dx = s (ds - sum ds s),   sigmoid  dx = ds s (1 - s).
// One warp a token; the row is written without the chosen experts' part first,
// then lane i writes the entry of chosen expert i whole.
// ---------------------------------------------------------------------------
template <typename T, int PL>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(const RouteArgs a) {
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = (int64_t)gridDim.x * (kRouteThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5); t < a.tokens; t += step) {
        const T *row = static_cast<const T *>(a.x) + t * a.ldx;
        T *out = static_cast<T *>(a.dx) + t * a.lddx;
        const float *dsc = a.dscores ? a.dscores + t * a.experts : nullptr;
        float x[PL], g[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = i * 32 + lane;
            x[i] = e < a.experts ? IO<T>::to_f(row[e]) : -INFINITY;
            g[i] = dsc && e < a.experts ? dsc[e] : 0.f;
        }
        int64_t id = lane < a.k ? a.ids_in[t * a.k + lane] : -1;
        if (id < 0 || id >= a.experts) id = -1;
        float dw = id >= 0 ? a.dweights[t * a.k + lane] * a.scale : 0.f;
        const float xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
        const float gs = id >= 0 && dsc ? dsc[id] : 0.f;
        float m = 0.f, inv = 1.f;
        if (a.softmax) {
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < PL; ++i) m = fmaxf(m, x[i]);
            m = from_ordered32(__reduce_max_sync(ALL, ordered32(m)));
            if (m == -INFINITY) m = 0.f;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                x[i] = expf(x[i] - m);
                d += x[i];
            }
            d = warp_sum_all(d);
            inv = d > 0.f ? 1.f / d : d == 0.f ? 0.f : d;
#pragma unroll
            for (int i = 0; i < PL; ++i) x[i] *= inv;
        }
        // the chosen score and its slope in the logit
        float s, slope;
        if (a.softmax) {
            s = slope = id >= 0 ? expf(xs - m) * inv : 0.f;
        } else {
            const float e = expf(-fabsf(xs)), q = 1.f / (1.f + e);
            s = id >= 0 ? (xs < 0.f ? e * q : q) : 0.f;
            slope = id >= 0 ? e * q * q : 0.f;
        }
        if (a.renorm) {
            const float sum = warp_sum_all(s), mean = warp_sum_all(dw * s) / sum;
            dw = sum == 0.f ? 0.f : (dw - mean) / sum;
        }
        float dot = 0.f;
        if (a.softmax) {
#pragma unroll
            for (int i = 0; i < PL; ++i) dot = fmaf(g[i], x[i], dot);
            dot = warp_sum_all(fmaf(dw, s, dot));
        }
        __syncwarp();  // dx may replace the logits: every lane has read its own
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = i * 32 + lane;
            float v;
            if (a.softmax) {
                v = x[i] * (g[i] - dot);
            } else {
                const float z = expf(-fabsf(x[i])), q = 1.f / (1.f + z);
                v = g[i] * z * q * q;
            }
            if (e < a.experts) out[e] = IO<T>::from_f(v);
        }
        // an expert listed twice: its gradients add up, and its first lane writes
        const uint32_t same = __match_any_sync(ALL, (int)id);
        if (__any_sync(ALL, id >= 0 && (same & (same - 1)) != 0)) {
            float all = 0.f;
            for (int p = 0; p < a.k; ++p) {
                const float v = __shfl_sync(ALL, dw, p);
                if (same >> p & 1u) all += v;
            }
            dw = all;
        }
        __syncwarp();
        if (id >= 0 && lane == __ffs(same) - 1) out[id] = IO<T>::from_f(slope * (gs + dw - dot));
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (route_<type>.cu).
// ---------------------------------------------------------------------------
template <typename T, int PL> cudaError_t launch_route_n(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    auto kernel = back ? route_bwd_kernel<T, PL> : route_fwd_kernel<T, PL>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), kRouteThreads, 0, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t need = (a.tokens + kRouteThreads / 32 - 1) / (kRouteThreads / 32), most = (int64_t)sms * per_sm;
    p->kind = PLAN_WARP;
    p->threads = kRouteThreads;
    p->packs = PL;
    return launch_row(kernel, (unsigned)(need < most ? need : most), (unsigned)kRouteThreads, 0, s, a);
}

template <typename T> cudaError_t launch_route_t(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    const int n = back ? (a.experts + 31) / 32 : a.per_lane;
    if (n <= 2) return launch_route_n<T, 2>(a, back, sms, s, p);
    if (n <= 4) return launch_route_n<T, 4>(a, back, sms, s, p);
    if (n <= 8) return launch_route_n<T, 8>(a, back, sms, s, p);
    if (n <= 16) return launch_route_n<T, 16>(a, back, sms, s, p);
    return launch_route_n<T, 32>(a, back, sms, s, p);
}

}  // namespace nrm
