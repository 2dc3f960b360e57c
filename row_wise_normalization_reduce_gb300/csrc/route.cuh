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
// places: the few experts in question are then compared to 42 bits, one a lane,
// and where a border between groups is that near, or experts equal to the last place
// were passed over, the whole token is done again so.  Equal logits with equal biases are equal, not near.
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
// What a group's sum of two is in fixed point where it has one available expert
// alone, whose key counts the least bias once, not twice: that key and the one of c =
// 0, `zero`.  With a `zero` beyond kZeroMost (biases far from 0 for their range) sums
// would not fit, and the token is done again.  Groups without an expert come last.
constexpr float kZeroMost = 33554432.f;
constexpr int kWorthNone = 1, kWorthBase = 33554432 + 2;  // so that any sum is above kWorthNone
__device__ __forceinline__ uint32_t pair_worth(uint32_t b1, uint32_t b2, int zero) {
    return (uint32_t)(b1 ? (int)b1 + (b2 ? (int)b2 : zero) + kWorthBase : kWorthNone);
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

// 1 / (1 + exp(-x)), to a few steps of 2^-24.
__device__ __forceinline__ float route_sigmoid(float x) {
    const float e = expf(-fabsf(x)), q = __fdividef(1.f, 1.f + e);
    return x < 0.f ? e * q : q;
}

// ---------------------------------------------------------------------------
// What an expert is chosen by to some 42 bits, for choices that binary32 cannot
// tell apart: as the unevaluated sum of two binary32 numbers.  (In binary64, of
// which an SM adds two a cycle, the exponentials and divisions of 256 experts, some
// 60 operations each, are 8000 cycles of an SM's.)  The products and sums are T. J. Dekker's and
// D. E. Knuth's.
// ---------------------------------------------------------------------------
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair pair_norm(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair pair_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    const Pair s = pair_sum(a.hi, b.hi), t = pair_sum(a.lo, b.lo);
    const Pair u = pair_norm(s.hi, __fadd_rn(s.lo, t.hi));
    return pair_norm(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    const float e = fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, __fmul_rn(a.lo, b.hi));
    return pair_norm(p, e);
}
// 1 / a: a first quotient and one step of the remainder.
__device__ __forceinline__ Pair pair_inv(Pair a) {
    const float q = 1.f / a.hi, p = __fmul_rn(a.hi, q);
    const float rest = __fsub_rn(__fsub_rn(__fsub_rn(1.f, p), fmaf(a.hi, q, -p)), __fmul_rn(a.lo, q));
    return pair_norm(q, __fmul_rn(rest, q));
}
// exp(x) for x <= 0.  The reduction is W. J. Cody and W. Waite's ("Software Manual
// for the Elementary Functions", 1980, EXP): x - n log 2 with log 2 = 355/512 + C,
// the first product exact, C = -2.12194440054690583e-4 in two numbers.  Then the
// Taylor series at an eighth of the rest, at most 0.044 (what comes after x^7 is
// below 2^-47), in pairs up to x^4 and binary32 beyond (x^5 / 120 < 2^-29 and its
// rounding 2^-53), and three squarings.
__device__ __forceinline__ Pair pair_exp(Pair x) {
    if (!(x.hi > -104.f)) return Pair{x.hi != x.hi ? x.hi : 0.f, 0.f};
    const float n = rintf(x.hi * kRouteLog2e);
    const float c = -2.12194440e-4f, c_rest = (float)(-2.12194440054690583e-4 - (double)-2.12194440e-4f);
    const Pair nc{__fmul_rn(n, -c), fmaf(n, -c, -__fmul_rn(n, -c)) - n * c_rest};
    Pair r = pair_add(pair_sum(fmaf(n, -355.f / 512.f, x.hi), x.lo), nc);
    r.hi *= 0.125f;
    r.lo *= 0.125f;
    const float q = fmaf(r.hi, fmaf(r.hi, 1.f / 5040, 1.f / 720), 1.f / 120);
    auto over = [](double v) { return Pair{(float)v, (float)(v - (double)(float)v)}; };
    Pair s = pair_add(pair_mul(r, Pair{q, 0.f}), over(1.0 / 24));
    s = pair_add(pair_mul(r, s), over(1.0 / 6));
    s = pair_add(pair_mul(r, s), Pair{0.5f, 0.f});
    s = pair_add(pair_mul(r, s), Pair{1.f, 0.f});
    s = pair_add(pair_mul(r, s), Pair{1.f, 0.f});
    s = pair_mul(s, s);
    s = pair_mul(s, s);
    s = pair_mul(s, s);
    const float f = __int_as_float(((int)n / 2 + 127) << 23), h = __int_as_float(((int)n - (int)n / 2 + 127) << 23);
    return Pair{s.hi * f * h, s.lo * f * h};  // 2^n, n >= -151, in two steps
}
// Order of pairs as that of integers: values first, then what they leave.
__device__ __forceinline__ uint64_t ordered_pair(Pair v) {
    if (!(fabsf(v.hi) < INFINITY)) v.lo = 0.f;
    return (uint64_t)ordered32(v.hi) << 32 | ordered32(v.lo);
}
// A token's largest logit and 1 / the sum of exp(x - it).
template <typename T>
__device__ __forceinline__ void route_softmax_pair(const RouteArgs &a, const T *row, int lane, float *m, Pair *inv) {
    float top = -INFINITY;
    for (int e = lane; e < a.experts; e += 32) top = fmaxf(top, IO<T>::to_f(row[e]));
    top = from_ordered32(__reduce_max_sync(0xffffffffu, ordered32(top)));
    Pair sum{0.f, 0.f};
    for (int e = lane; e < a.experts; e += 32) {
        const float x = IO<T>::to_f(row[e]);
        if (x > -INFINITY || x != x) sum = pair_add(sum, pair_exp(pair_sum(x, -top)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = pair_add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    *m = top;
    *inv = pair_inv(sum);
}
// What one expert is chosen by; -inf where it is not available.
__device__ __forceinline__ Pair route_choice(const RouteArgs &a, float x, int e, float m, Pair inv) {
    const float b = a.bias ? a.bias[e] : 0.f;
    if (x == -INFINITY || !(fabsf(b) < INFINITY)) return Pair{x == -INFINITY || b != b ? -INFINITY : b, 0.f};
    Pair s;
    if (a.softmax) {
        s = pair_mul(pair_exp(pair_sum(x, -m)), inv);
    } else {
        const Pair z = pair_exp(Pair{-fabsf(x), 0.f});
        s = pair_inv(pair_add(Pair{1.f, 0.f}, z));
        if (x < 0.f) s = pair_mul(z, s);
    }
    s = pair_add(s, Pair{b, 0.f});
    return s.hi != s.hi ? Pair{-INFINITY, 0.f} : s;
}

// The whole selection by those.  Lane r returns the expert at place r, or -1.
// (Taking only the experts in question as pairs, in two steps, changed nothing.)
template <typename T, int PL>
__device__ __noinline__ int route_exact(const RouteArgs &a, const T *row, int lane) {
    constexpr uint32_t ALL = 0xffffffffu;
    const RouteLane r(a, lane);
    const Pair no{-INFINITY, 0.f};
    const uint64_t none = ordered_pair(no);
    float m = 0.f;
    Pair inv{1.f, 0.f};
    if (a.softmax && a.by_score) route_softmax_pair(a, row, lane, &m, &inv);
    // (loops, not unrolled: this code is cold when it runs, and eight copies of a
    // choice have to be fetched; unrolled, 65536 tokens of 256 took 41 us, so 37)
    uint64_t key[PL], k1 = none, k2 = none;
    Pair b1 = no, b2 = no;  // the lane's two largest
#pragma unroll 1
    for (int i = 0; i < PL; ++i) {
        Pair c = no;
        if (i < r.n) {
            const float x = IO<T>::to_f(row[r.first + i]);
            if (a.by_score) c = route_choice(a, x, r.first + i, m, inv);
            else if (x > -INFINITY) c = Pair{x, 0.f};
        }
        const uint64_t k = ordered_pair(c);
        key[i] = k;
        if (k > k1) {
            b2 = b1;
            k2 = k1;
            b1 = c;
            k1 = k;
        } else if (k > k2) {
            b2 = c;
            k2 = k;
        }
    }
    if (a.top_groups < a.groups) {
        const int lanes = 1 << a.log_lanes;
        auto other = [&](Pair v, int o) { return Pair{__shfl_xor_sync(ALL, v.hi, o), __shfl_xor_sync(ALL, v.lo, o)}; };
        for (int o = 1; o < lanes; o <<= 1) {
            const Pair c1 = other(b1, o), c2 = other(b2, o);
            const uint64_t j1 = __shfl_xor_sync(ALL, k1, o), j2 = __shfl_xor_sync(ALL, k2, o);
            if (j1 > k1) {
                b2 = j2 > k1 ? c2 : b1;
                k2 = j2 > k1 ? j2 : k1;
                b1 = c1;
                k1 = j1;
            } else if (j1 > k2) {
                b2 = c1;
                k2 = j1;
            }
        }
        const bool two = a.group_top > 1 && k2 > none && fabsf(b1.hi) < INFINITY && fabsf(b2.hi) < INFINITY;
        // (halves: the sum of two large biases is beyond binary32)
        auto half = [](Pair v) { return Pair{0.5f * v.hi, 0.5f * v.lo}; };
        const uint64_t worth = ordered_pair(two ? pair_add(half(b1), half(b2)) : half(b1));
        int rank = 0;
        const int g = lane >> a.log_lanes;
        for (int h = 0; h < a.groups; ++h) {
            const uint64_t w = __shfl_sync(ALL, worth, h << a.log_lanes);
            if (w > worth || (w == worth && h < g)) ++rank;
        }
        if (rank >= a.top_groups) {
#pragma unroll 1
            for (int i = 0; i < PL; ++i) key[i] = none;
        }
    }
    int mine = -1;
    for (int p = 0; p < a.k; ++p) {
        uint64_t best = none;
        int at = -1;
#pragma unroll 1
        for (int i = PL - 1; i >= 0; --i)
            if (key[i] > none && key[i] >= best) {
                best = key[i];
                at = i;
            }
        const uint32_t hi = __reduce_max_sync(ALL, (uint32_t)(best >> 32));
        const uint32_t lo = __reduce_max_sync(ALL, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const uint32_t who = __ballot_sync(ALL, at >= 0 && best == ((uint64_t)hi << 32 | lo));
        if (!who) break;
        const int src = __ffs(who) - 1, id = __shfl_sync(ALL, r.first + at, src);
        if (lane == p) mine = id;
        if (lane == src) key[at] = none;
    }
    return mine;
}

// What the forward's keys are made of.
//   WHOLE   16-bit logits as they are: nothing is in question
//   LOGIT   binary32 logits in fixed point, up to 16 below the row's largest
//   SCORE   score + bias in fixed point over the range that they can have, [least
//           bias, 1 + largest bias]: one multiply-add from the score
enum RouteKey { KEY_WHOLE, KEY_LOGIT, KEY_SCORE };

// Places that may be in the wrong order: the experts around and on the border of
// the k-th place, one a lane, compared as pairs.  `mine` is the key at this
// lane's place, `list` the lane's remaining keys; returns false where there are
// more of them than lanes.  Called by few tokens, so kept out of line.
template <typename T, int PL, int LIST>
__device__ __noinline__ bool route_resolve(const RouteArgs &a, const T *row, int lane, uint32_t mine, uint32_t last,
                                           uint32_t (&list)[LIST + 1], int left, float near_, int *id, float *xs) {
    constexpr uint32_t ALL = 0xffffffffu;
    int places = a.k;
    while (true) {
        const uint32_t w = __reduce_max_sync(ALL, list[0]);
        if (w == 0u || (float)((last >> kIdxBits) - (w >> kIdxBits)) > near_) break;
        if (places == 32) return false;
        if (lane == places) mine = w;
        ++places;
        if (list[0] == w) {
#pragma unroll
            for (int i = 0; i < LIST; ++i) list[i] = list[i + 1];
            --left;
        }
        if (PL > LIST && __any_sync(ALL, left == 0)) return false;
    }
    const int e = mine ? kIdxMask - (int)(mine & kIdxMask) : -1;
    const float x = e >= 0 ? IO<T>::to_f(row[e]) : -INFINITY;
    float m = 0.f;
    Pair inv{1.f, 0.f};
    if (a.softmax && a.by_score) route_softmax_pair(a, row, lane, &m, &inv);
    uint64_t key = 0;
    if (e >= 0) key = ordered_pair(a.by_score ? route_choice(a, x, e, m, inv) : Pair{x, 0.f});
    int rank = 0;
    for (int p = 0; p < places; ++p) {
        const uint64_t o = __shfl_sync(ALL, key, p);
        const int oe = __shfl_sync(ALL, e, p);
        rank += o > key || (o == key && oe < e);
    }
    // who has the rank of this lane?
    int src = lane;
    for (int p = 0; p < places; ++p)
        if (__shfl_sync(ALL, rank, p) == lane) src = p;
    *id = __shfl_sync(ALL, e, src);
    *xs = __shfl_sync(ALL, x, src);
    return true;
}

template <typename T, int PL, int MODE>
__global__ void __launch_bounds__(kRouteThreads) route_fwd_kernel(const RouteArgs a) {
    constexpr int LIST = PL < 8 ? PL : 8;
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const RouteLane r(a, lane);
    const bool limited = a.top_groups < a.groups;
    const int g = lane >> a.log_lanes;
    // (expert's part of the key of slot i: first - i)
    const uint32_t index = (uint32_t)(kIdxMask - r.first);
    pdl_wait();
    pdl_launch_dependents();
    // SCORE: the fixed point's step is 1 / S, and bias i's part base[i]
    float base[MODE == KEY_SCORE ? PL : 1], S = 262143.f, near_bias = 0.f;
    int zero = 0;           // what a missing second of a group counts
    bool zero_far = false;  // beyond what sums hold
    bool odd_bias = false;  // infinite or NaN ones
    bool wild = false;      // their range is beyond binary32: every token is done again
    if constexpr (MODE == KEY_SCORE) {
        float lo = INFINITY, hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            base[i] = i < r.n ? (a.bias ? a.bias[r.first + i] : 0.f) : -INFINITY;
            if (fabsf(base[i]) < INFINITY) {
                lo = fminf(lo, base[i]);
                hi = fmaxf(hi, base[i]);
            } else if (i < r.n) {
                odd_bias = true;
            }
        }
        odd_bias = __any_sync(ALL, odd_bias);
        lo = from_ordered32(__reduce_min_sync(ALL, ordered32(lo)));
        hi = from_ordered32(__reduce_max_sync(ALL, ordered32(hi)));
        if (!(hi >= lo)) lo = hi = 0.f;  // no expert has a finite bias
        S = 4194300.f / (1.f + (hi - lo));
        wild = !(hi - lo < INFINITY);
        // the rounding of base: half a step of its size, relative to 2^23
        near_bias = 1.2e-7f * (fabsf(lo) + fabsf(hi)) * S + 1.f;
        const float z = rintf(fmaf(-lo, S, 2.f));
        zero_far = !(fabsf(z) < kZeroMost);
        zero = zero_far ? 0 : (int)z;
#pragma unroll
        for (int i = 0; i < PL; ++i) base[i] = fmaf(base[i] - lo, S, 8388610.f);
    }
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
            m = m == -INFINITY ? 0.f : m;
            d = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) d += route_exp2((x[i] - m) * kRouteLog2e);
            d = warp_sum_all(d);
        }
        if (a.scores) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (i < r.n)
                    a.scores[t * a.experts + r.first + i] =
                        x[i] == -INFINITY ? 0.f : a.softmax ? expf(x[i] - m) / d : 1.f / (1.f + expf(-x[i]));
        }
        // keys, largest first; 0: not available
        uint32_t key[PL];
        float near_ = 0.f;   // keys no further apart than this are in question
        bool again = false;  // the whole token is
        if constexpr (MODE == KEY_WHOLE) {
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                uint32_t b = ordered32(x[i]) >> 16;
                if (std::is_same<T, __half>::value) {  // binary16 keeps more bits than a binary32's upper half
                    b = __half_as_ushort(__float2half_rn(x[i] + 0.f));
                    b = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
                }
                key[i] = x[i] > -INFINITY ? (b << kIdxBits) + (index - i) : 0u;
            }
        } else if constexpr (MODE == KEY_LOGIT) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < PL; ++i) top = fmaxf(top, x[i]);
            top = from_ordered32(__reduce_max_sync(ALL, ordered32(top)));
            again = top == INFINITY;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const float q = fmaxf(fmaf(x[i] - top, S, 8388608.f + 4194303.f), 8388609.f);
                key[i] = x[i] > -INFINITY ? (__float_as_uint(q) << kIdxBits) + (index - i) : 0u;
            }
            near_ = 2.f;  // the difference and the fixed point: half a step each, of either
        } else {
            // A sigmoid is good to 3e-7 (the exponent's argument, ex2, rcp), a
            // softmax to 6e-7 of the largest and half a step for each addition
            // of its sum; the multiply-add rounds to half a step.
            const float inv = a.softmax ? 1.f / d : 1.f;
            near_ = 2.f * (S * (a.softmax ? (6e-7f + 6e-8f * (PL + 6)) * inv : 3e-7f) + near_bias);
            float odd = 0.f;  // NaN or inf where a logit is
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                odd += x[i];
                const float s = a.softmax ? route_exp2((x[i] - m) * kRouteLog2e) * inv
                                          : route_rcp(1.f + route_exp2(x[i] * -kRouteLog2e));
                key[i] = (__float_as_uint(fmaf(s, S, base[i])) << kIdxBits) + (index - i);
            }
            // experts that a lane has not, and those that are not available
            if (__any_sync(ALL, !(fabsf(odd) < INFINITY)) || odd_bias) {
                bool far = false;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    if (!(x[i] > -INFINITY) || !(base[i] > 0.f) || !(d < INFINITY)) key[i] = 0u;
                    far = far || x[i] == INFINITY || base[i] == INFINITY;
                }
                again = __any_sync(ALL, far);
            }
            again = again || wild;
        }
        sort_desc<PL>(key);
        if (limited) {
            uint32_t b1 = key[0] >> kIdxBits, b2 = key[PL > 1 ? 1 : 0] >> kIdxBits;
            for (int o = 1; o < 1 << a.log_lanes; o <<= 1) {
                const uint32_t c1 = __shfl_xor_sync(ALL, b1, o), c2 = __shfl_xor_sync(ALL, b2, o);
                b2 = max(min(b1, c1), max(b2, c2));
                b1 = max(b1, c1);
            }
            // sum and then the lower group first; + 1: groups without an expert are
            // still groups
            const bool two = MODE == KEY_SCORE && a.group_top > 1, real = g < a.groups;
            if (two) again = again || (zero_far && __any_sync(ALL, b1 && !b2));
            const uint32_t sum = two ? pair_worth(b1, b2, zero) : b1 + 1u;
            const uint32_t worth = real ? sum * 32u + (uint32_t)(31 - g) : 0u;
            uint32_t rest = worth, least = 0u;
            for (int i = 0; i < a.top_groups; ++i) {
                least = __reduce_max_sync(ALL, rest);
                rest = rest == least ? 0u : rest;
            }
            const bool keep = real && rest == 0u;
            if constexpr (MODE != KEY_WHOLE) {
                const uint32_t most = __reduce_max_sync(ALL, rest);
                // too near; or a kept group owes its place to a logit below the range
                const bool low = MODE == KEY_LOGIT && keep && b1 == 1u;
                again = again || (float)(least / 32u - most / 32u) <= (two ? 2.f : 1.f) * near_ || __any_sync(ALL, low);
            }
            // all that the list below may take, for an emptied place would move up
            // what lies behind it
            if (!keep) {
#pragma unroll
                for (int i = 0; i < (PL > LIST ? LIST + 1 : PL); ++i) key[i] = 0u;
            }
        }
        // a softmax of a NaN or of infinity is NaN for every expert (keys of scores
        // show that themselves)
        if (MODE != KEY_SCORE && a.softmax) {
            float odd = 0.f;  // finite or -inf where none is, but for overflow
#pragma unroll
            for (int i = 0; i < PL; ++i) odd += x[i];
            if (__any_sync(ALL, !(odd < INFINITY))) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i < PL; ++i) bad = bad || !(x[i] < INFINITY);
                if (__any_sync(ALL, bad)) {
                    again = false;
#pragma unroll
                    for (int i = 0; i < PL; ++i) key[i] = 0u;
                }
            }
        }
        // places: the k largest
        uint32_t list[LIST + 1], mine = 0u, last = 0u;
#pragma unroll
        for (int i = 0; i < LIST; ++i) list[i] = key[i];
        list[LIST] = 0u;
        // a lane whose list runs out may hold more
        int left = PL > LIST && key[PL > LIST ? LIST : 0] ? LIST : kRouteMaxK + 1;
        for (int p = 0; p < a.k; ++p) {
            last = __reduce_max_sync(ALL, list[0]);
            if (lane == p) mine = last;
            if (list[0] == last) {
#pragma unroll
                for (int i = 0; i < LIST; ++i) list[i] = list[i + 1];
                if (PL > LIST) --left;
            }
            if (PL > LIST && __any_sync(ALL, left == 0)) {
                again = again || MODE != KEY_WHOLE || p + 1 < a.k;
                left = kRouteMaxK + 1;
            }
        }
        int id = mine ? kIdxMask - (int)(mine & kIdxMask) : -1;
        float xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
        if constexpr (MODE != KEY_WHOLE) {
            // gaps between neighbouring places, and to the first one left out
            const uint32_t after = __reduce_max_sync(ALL, list[0]);
            const uint32_t up = __shfl_up_sync(ALL, mine, 1);
            const float xu = __shfl_up_sync(ALL, xs, 1);
            bool close = false;
            if (lane == 0) close = after && (float)((last >> kIdxBits) - (after >> kIdxBits)) <= near_;
            else if (mine) close = (float)((up >> kIdxBits) - (mine >> kIdxBits)) <= near_;
            if (__any_sync(ALL, close)) {
                // equal logits with equal biases are equal, not near
                const float bs = MODE == KEY_SCORE && a.bias && id >= 0 ? a.bias[id] : 0.f;
                const float bu = __shfl_up_sync(ALL, bs, 1);
                if (lane > 0) close = close && !(xs == xu && bs == bu);
                // those equal to the last place come after it, but before a place in
                // question that turns out to be smaller: with any passed over, such a
                // token is done again (kept beside the list, for route_resolve, they would
                // cost 16 to 27 registers and with them a CTA an SM)
                uint32_t w = after, rest[LIST + 1];
#pragma unroll
                for (int i = 0; i <= LIST; ++i) rest[i] = list[i];
                const float xl = __shfl_sync(ALL, xs, a.k - 1), bl = __shfl_sync(ALL, bs, a.k - 1);
                bool border = false, equal = false;
                while (w && (float)((last >> kIdxBits) - (w >> kIdxBits)) <= near_) {
                    const int e = kIdxMask - (int)(w & kIdxMask);
                    border = !(IO<T>::to_f(row[e]) == xl && (MODE == KEY_SCORE && a.bias ? a.bias[e] : 0.f) == bl);
                    if (border) break;
                    equal = true;
                    if (rest[0] == w) {
#pragma unroll
                        for (int i = 0; i < LIST; ++i) rest[i] = rest[i + 1];
                        --left;
                    }
                    if (PL > LIST && __any_sync(ALL, left == 0)) {
                        again = true;
                        break;
                    }
                    w = __reduce_max_sync(ALL, rest[0]);
                }
                if (!again && (border || __any_sync(ALL, close && lane > 0)))
                    again = equal || !route_resolve<T, PL, LIST>(a, row, lane, mine, last, rest, left, near_, &id, &xs);
            }
            if (again) {
                id = route_exact<T, PL>(a, row, lane);
                xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
            }
        } else if (again) {
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
            w = have ? route_sigmoid(xs) : 0.f;
        }
        if (a.renorm) {
            const float sum = warp_sum_all(w);
            w = sum > 1e-30f ? __fdividef(w, sum) : sum == 0.f ? 0.f : w / sum;
        }
        if (lane < a.k) {
            a.weights[t * a.k + lane] = w * a.scale;
            a.ids[t * a.k + lane] = have ? id : -1;
        }
    }
}

// ---------------------------------------------------------------------------
// Up to 8 places of up to 256 experts (and 8 groups): eight lanes a token, four
// tokens a warp, so that what passes between lanes is done for four at once.  A
// lane takes its experts in chunks of eight, sorts each chunk's keys and keeps the
// eight largest (the larger of entry i of one list and entry 7 - i of the other
// are the eight largest of both, and three stages of exchanges sort them); three
// merges of the same kind join the lanes.  65536 x 256 bf16 in 8 groups: 38 us, a
// warp a token 65; without groups and bias 23 and 34.  Bound by instructions, 320 a
// token (the keys' exponentials and sorting networks most of them), and by the
// last turn: 3.4 of four.  (Taking tokens from a counter instead: no change.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ void exchange(uint32_t &a, uint32_t &b) {
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
// list: the 8 largest of two descending lists of 8, descending.
__device__ __forceinline__ void merge8(uint32_t (&list)[8], const uint32_t (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) list[i] = max(list[i], o[7 - i]);
#pragma unroll
    for (int d = 4; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) exchange(list[i], list[i + d]);
}
// Over the eight lanes of a token.
__device__ __forceinline__ uint32_t oct_max(uint32_t v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ uint32_t oct_min(uint32_t v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float oct_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename T> __device__ __forceinline__ uint4 no_expert() {  // a pack of -inf
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}

template <typename T, int NC, int MODE>
__global__ void __launch_bounds__(kRouteThreads, 4) route_oct_kernel(const RouteArgs a) {
    constexpr uint32_t ALL = 0xffffffffu;
    constexpr int PL = 8 * NC;
    // SCORE: the biases in fixed point, a lane's 8 NC together and 4 apart from the
    // next lane's (the lanes' 16-byte loads fall on different banks)
    __shared__ __align__(16) float base_of[MODE == KEY_SCORE ? 8 * (PL + 4) : 1];
    __shared__ float range[2];
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    const int g = l >> a.oct_log_lanes, first = g * a.group_size + (l & ((1 << a.oct_log_lanes) - 1)) * a.oct_per_lane;
    const int n = g < a.groups ? max(0, min(a.oct_per_lane, (g + 1) * a.group_size - first)) : 0;
    const bool limited = a.top_groups < a.groups;
    const uint32_t index = (uint32_t)(kIdxMask - first);
    float S = 262143.f, near_bias = 0.f;
    int zero = 0;           // what a missing second of a group counts
    bool zero_far = false;  // beyond what sums hold
    bool odd_bias = false;  // infinite or NaN ones
    bool wild = false;      // their range is beyond binary32: every token is done again
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (MODE == KEY_SCORE) {
        if (threadIdx.x < 32) {
            float lo = INFINITY, hi = -INFINITY;
            for (int e = lane; e < a.experts; e += 32) {
                const float b = a.bias ? a.bias[e] : 0.f;
                if (fabsf(b) < INFINITY) {
                    lo = fminf(lo, b);
                    hi = fmaxf(hi, b);
                } else {
                    odd_bias = true;
                }
            }
            lo = from_ordered32(__reduce_min_sync(ALL, ordered32(lo)));
            hi = from_ordered32(__reduce_max_sync(ALL, ordered32(hi)));
            if (!(hi >= lo)) lo = hi = 0.f;  // no expert has a finite bias
            if (lane == 0) {
                range[0] = lo;
                range[1] = hi;
            }
        }
        odd_bias = __syncthreads_or(odd_bias);
        const float lo = range[0], hi = range[1];
        S = 4194300.f / (1.f + (hi - lo));
        wild = !(hi - lo < INFINITY);
        // the rounding of base: half a step of its size, relative to 2^23
        near_bias = 1.2e-7f * (fabsf(lo) + fabsf(hi)) * S + 1.f;
        const float z = rintf(fmaf(-lo, S, 2.f));
        zero_far = !(fabsf(z) < kZeroMost);
        zero = zero_far ? 0 : (int)z;
        if (threadIdx.x < 8) {
            for (int i = 0; i < PL; ++i)
                base_of[l * (PL + 4) + i] =
                    i < n ? fmaf((a.bias ? a.bias[first + i] : 0.f) - lo, S, 8388610.f) : -INFINITY;
        }
        __syncthreads();
    }
    const int64_t step = (int64_t)gridDim.x * (kRouteThreads / 8);
    for (int64_t t0 = (int64_t)blockIdx.x * (kRouteThreads / 8) + (threadIdx.x >> 5) * 4; t0 < a.tokens; t0 += step) {
        const bool real = t0 + sub < a.tokens;
        const int64_t t = real ? t0 + sub : a.tokens - 1;
        const T *row = static_cast<const T *>(a.x) + t * a.ldx;
        // a lane's logits: whole packs, or one by one
        constexpr int W = 8 / IO<T>::V;  // packs a chunk
        auto fetch = [&](int c, uint4 (&raw)[W]) {
            if (a.oct_wide) {
#pragma unroll
                for (int w = 0; w < W; ++w)
                    raw[w] = n > 0 ? *reinterpret_cast<const uint4 *>(row + first + c * 8 + w * IO<T>::V) : no_expert<T>();
            } else {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = c * 8 + i < n ? IO<T>::to_f(row[first + c * 8 + i]) : -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) raw[w] = IO<T>::pack(v + w * IO<T>::V);
            }
        };
        auto unpack = [&](const uint4 (&raw)[W], float (&x)[8]) {
#pragma unroll
            for (int w = 0; w < W; ++w) IO<T>::unpack(raw[w], x + w * IO<T>::V);
        };
        auto chunk = [&](int c, float (&x)[8]) {
            uint4 raw[W];
            fetch(c, raw);
            unpack(raw, x);
        };
        // the softmax' maximum and sum, where they are needed; binary32 logits' largest
        float m = 0.f, d = 1.f, inv = 1.f;
        if (MODE == KEY_LOGIT || (a.softmax && a.need_sum)) {
            m = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                float x[8];
                chunk(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, x[i]);
            }
            m = oct_max(m);
        }
        const float top = m;
        if (a.softmax && a.need_sum) {
            m = m == -INFINITY ? 0.f : m;
            d = 0.f;
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                float x[8];
                chunk(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) d += route_exp2((x[i] - m) * kRouteLog2e);
            }
            d = group_sum_all<8>(d);
            inv = 1.f / d;
        }
        if (a.scores && real) {
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                float x[8];
                chunk(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c * 8 + i < n)
                        a.scores[t * a.experts + first + c * 8 + i] =
                            x[i] == -INFINITY ? 0.f : a.softmax ? expf(x[i] - m) / d : 1.f / (1.f + expf(-x[i]));
            }
        }
        // keys, largest first; 0: not available
        uint32_t list[8];
        float near_ = MODE == KEY_LOGIT ? 2.f : 0.f;  // keys no further apart than this are in question
        bool again = wild;                            // the whole token is
        float odd_sum = 0.f;                          // NaN or infinity where a logit is, but for overflow
        if constexpr (MODE == KEY_SCORE)
            // as in route_fwd_kernel; the sum is at most 8 NC + 3 additions deep
            near_ = 2.f * (S * (a.softmax ? (6e-7f + 6e-8f * (PL + 3)) * inv : 3e-7f) + near_bias);
#pragma unroll
        for (int i = 0; i < 8; ++i) list[i] = 0u;
        uint4 coming[W];
        fetch(0, coming);
        // (one copy of the loop's code: four did not fit the instruction cache)
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
            float x[8];
            uint32_t key[8];
            unpack(coming, x);
            if (c + 1 < NC) fetch(c + 1, coming);
            if constexpr (MODE != KEY_SCORE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) odd_sum += x[i];
            }
            if constexpr (MODE == KEY_WHOLE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t b = ordered32(x[i]) >> 16;
                    if (std::is_same<T, __half>::value) {  // binary16 keeps more bits than a binary32's upper half
                        b = __half_as_ushort(__float2half_rn(x[i] + 0.f));
                        b = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
                    }
                    key[i] = x[i] > -INFINITY ? (b << kIdxBits) + (index - (c * 8 + i)) : 0u;
                }
            } else if constexpr (MODE == KEY_LOGIT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = fmaxf(fmaf(x[i] - top, S, 8388608.f + 4194303.f), 8388609.f);
                    key[i] = x[i] > -INFINITY ? (__float_as_uint(q) << kIdxBits) + (index - (c * 8 + i)) : 0u;
                }
                again = top == INFINITY;
            } else {
                float odd = 0.f, base[8];  // odd: NaN or inf where a logit is
                const float4 b0 = *reinterpret_cast<const float4 *>(&base_of[l * (PL + 4) + c * 8]),
                             b1 = *reinterpret_cast<const float4 *>(&base_of[l * (PL + 4) + c * 8 + 4]);
                base[0] = b0.x, base[1] = b0.y, base[2] = b0.z, base[3] = b0.w;
                base[4] = b1.x, base[5] = b1.y, base[6] = b1.z, base[7] = b1.w;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    odd += x[i];
                    const float s = a.softmax ? route_exp2((x[i] - m) * kRouteLog2e) * inv
                                              : route_rcp(1.f + route_exp2(x[i] * -kRouteLog2e));
                    key[i] = (__float_as_uint(fmaf(s, S, base[i])) << kIdxBits) + (index - (c * 8 + i));
                }
                // experts that a lane has not, and those that are not available
                if (__any_sync(ALL, !(fabsf(odd) < INFINITY)) || odd_bias) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!(x[i] > -INFINITY) || !(base[i] > 0.f) || !(d < INFINITY)) key[i] = 0u;
                        again = again || x[i] == INFINITY || base[i] == INFINITY;
                    }
                }
            }
            sort_desc<8>(key);
            merge8(list, key);
        }
        if (limited) {
            uint32_t b1 = list[0] >> kIdxBits, b2 = list[1] >> kIdxBits;
            for (int o = 1; o < 1 << a.oct_log_lanes; o <<= 1) {
                const uint32_t c1 = __shfl_xor_sync(ALL, b1, o), c2 = __shfl_xor_sync(ALL, b2, o);
                b2 = max(min(b1, c1), max(b2, c2));
                b1 = max(b1, c1);
            }
            // sum and then the lower group first; + 1: groups without an expert are
            // still groups
            const bool two = MODE == KEY_SCORE && a.group_top > 1, is = g < a.groups;
            if (two) again = again || (zero_far && b1 && !b2);
            const uint32_t sum = two ? pair_worth(b1, b2, zero) : b1 + 1u;
            const uint32_t worth = is ? sum * 32u + (uint32_t)(31 - g) : 0u;
            int rank = 0;
            for (int h = 0; h < a.groups; ++h)
                rank += __shfl_sync(ALL, worth, (lane & 24) | h << a.oct_log_lanes) > worth;
            const bool keep = is && rank < a.top_groups;
            if constexpr (MODE != KEY_WHOLE) {
                const uint32_t least = oct_min(keep ? worth : ALL), most = oct_max(keep ? 0u : worth);
                // too near; or a kept group owes its place to a logit below the range
                const bool low = MODE == KEY_LOGIT && keep && b1 == 1u;
                again = again || (float)(least / 32u - most / 32u) <= (two ? 2.f : 1.f) * near_ || low;
            }
            if (!keep) {
#pragma unroll
                for (int i = 0; i < 8; ++i) list[i] = 0u;
            }
        }
        // a softmax of a NaN or of infinity is NaN for every expert (keys of scores
        // show that themselves)
        if (MODE != KEY_SCORE && a.softmax && __any_sync(ALL, !(odd_sum < INFINITY))) {
            bool bad = false;
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                float x[8];
                chunk(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) bad = bad || !(x[i] < INFINITY);
            }
            if (__ballot_sync(ALL, bad) & 0xffu << (lane & 24)) {
                again = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) list[i] = 0u;
            }
        }
        uint32_t own[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) own[i] = list[i];
#pragma unroll
        for (int o = 1; o < 8; o *= 2) {
            uint32_t other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(ALL, list[i], o);
            merge8(list, other);
        }
        // place l
        uint32_t mine;
        {
            const uint32_t p = l & 4 ? list[4] : list[0], q = l & 4 ? list[5] : list[1], u = l & 4 ? list[6] : list[2],
                           v = l & 4 ? list[7] : list[3];
            const uint32_t w = l & 2 ? u : p, z = l & 2 ? v : q;
            mine = l & 1 ? z : w;
        }
        const uint32_t last = __shfl_sync(ALL, mine, (lane & 24) | (a.k - 1));
        if (l >= a.k) mine = 0u;
        int id = mine ? kIdxMask - (int)(mine & kIdxMask) : -1;
        float xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
        if constexpr (MODE != KEY_WHOLE) {
            // the first one left out: the largest below the last place
            uint32_t after = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) after = max(after, own[i] < last ? own[i] : 0u);
            after = oct_max(after);
            // a lane that has all its eight among the places may hold the next
            again = again || (PL > 8 && last && own[7] >= last);
            const uint32_t up = __shfl_up_sync(ALL, mine, 1);
            bool close = l > 0 && mine && (float)((up >> kIdxBits) - (mine >> kIdxBits)) <= near_;
            bool border = after && (float)((last >> kIdxBits) - (after >> kIdxBits)) <= near_;
            if (__any_sync(ALL, close || border)) {
                // equal logits with equal biases are equal, not near
                const float bs = MODE == KEY_SCORE && a.bias && id >= 0 ? a.bias[id] : 0.f;
                const float xu = __shfl_up_sync(ALL, xs, 1), bu = __shfl_up_sync(ALL, bs, 1);
                close = close && !(xs == xu && bs == bu);
                const float xl = __shfl_sync(ALL, xs, (lane & 24) | (a.k - 1)), bl = __shfl_sync(ALL, bs, (lane & 24) | (a.k - 1));
                // those equal to the last place come after it, but before a place in
                // question that turns out to be smaller
                const bool equal = border;
                while (__any_sync(ALL, border)) {
                    if (border) {
                        const int e = kIdxMask - (int)(after & kIdxMask);
                        again = again || !(IO<T>::to_f(row[e]) == xl && (MODE == KEY_SCORE && a.bias ? a.bias[e] : 0.f) == bl);
                    }
                    const uint32_t below = after;
                    after = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) after = max(after, own[i] < below ? own[i] : 0u);
                    after = oct_max(after);
                    again = again || (PL > 8 && border && own[7] && own[7] >= below);
                    border = border && after && (float)((last >> kIdxBits) - (after >> kIdxBits)) <= near_;
                }
                again = again || (close && (equal || (a.softmax && a.by_score)));
                if (!(a.softmax && a.by_score) && __any_sync(ALL, close)) {
                    // the places in their order, one expert a lane
                    uint64_t key = 0;
                    if (id >= 0) key = ordered_pair(a.by_score ? route_choice(a, xs, id, 0.f, Pair{1.f, 0.f}) : Pair{xs, 0.f});
                    int rank = 0, src = lane;
                    for (int p = 0; p < 8; ++p) {
                        const uint64_t o = __shfl_sync(ALL, key, (lane & 24) | p);
                        const int oe = __shfl_sync(ALL, id, (lane & 24) | p);
                        rank += o > key || (o == key && oe < id);
                    }
                    if (id < 0) rank = l;
                    for (int p = 0; p < 8; ++p)
                        if (__shfl_sync(ALL, rank, (lane & 24) | p) == l) src = (lane & 24) | p;
                    id = __shfl_sync(ALL, id, src);
                    xs = __shfl_sync(ALL, xs, src);
                }
            }
            for (uint32_t who = __ballot_sync(ALL, again && real); who;) {
                const int of = __ffs(who) - 1 >> 3;
                who &= ~(0xffu << of * 8);
                const T *r = static_cast<const T *>(a.x) + (t0 + of) * a.ldx;
                const int e = __shfl_sync(ALL, route_exact<T, 8>(a, r, lane), l);
                if (sub == of) {
                    id = l < a.k ? e : -1;
                    xs = id >= 0 ? IO<T>::to_f(row[id]) : -INFINITY;
                }
            }
        }
        float w;
        if (a.softmax) {
            if (a.renorm) m = oct_max(id >= 0 ? xs : -INFINITY);
            w = id < 0 ? 0.f : a.renorm ? expf(xs - m) : expf(xs - m) / d;
        } else {
            w = id >= 0 ? route_sigmoid(xs) : 0.f;
        }
        if (a.renorm) {
            const float sum = group_sum_all<8>(w);
            w = sum > 1e-30f ? __fdividef(w, sum) : sum == 0.f ? 0.f : w / sum;
        }
        if (real && l < a.k) {
            a.weights[t * a.k + l] = w * a.scale;
            a.ids[t * a.k + l] = id;
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient of the logits.  With d_i the gradient of chosen weight i times
// scale, s the scores and g the gradient of all of them (dscores, or 0),
//   softmax  dx = s (ds - sum ds s),   sigmoid  dx = ds s (1 - s),
// where ds is g plus, for each place i of an expert, d_i.  Renormalised weights w_i =
// s_i / S, S the chosen scores' sum, have ds_i = (d_i - sum_j d_j w_j) / S, whose sum
// with s over the chosen is 0, so that their part of dx is
//   softmax  w_i (d_i - sum_j d_j w_j),   sigmoid  that times 1 - s_i,
// without a division by S, which may be 0 or subnormal where the weights are
// ordinary numbers: w comes from the largest of the chosen, as exp(x - largest),
// sigmoid that / (1 + exp(x)) below 0.  Sigmoids that are all 0 have weights of 0
// and no such part.
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
        // the chosen score, its slope in the logit, and a sigmoid's 1 - s
        float s, slope, rest = 1.f;
        if (a.softmax) {
            s = slope = id >= 0 ? expf(xs - m) * inv : 0.f;
        } else {
            const float e = expf(-fabsf(xs)), q = 1.f / (1.f + e);
            s = id >= 0 ? (xs < 0.f ? e * q : q) : 0.f;
            rest = xs < 0.f ? q : e * q;
            slope = id >= 0 ? e * q * q : 0.f;
        }
        // dw: the weights' part of dx; dot: a softmax' sum of ds s without that
        float dot = 0.f;
        if (a.renorm) {
            // w from s where the row's largest is among the chosen (of sigmoids: one of
            // 1/2 and more), else from the differences to the chosen ones' largest
            const float top = from_ordered32(__reduce_max_sync(ALL, ordered32(id >= 0 ? xs : -INFINITY)));
            float w = s;
            if (!(top >= m)) {
                const bool none = a.softmax ? top == -INFINITY : expf(top) == 0.f;
                w = id >= 0 && !none ? expf(xs - top) * rest : 0.f;
            }
            const float sum = warp_sum_all(w);
            // (one expert alone has a weight of 1, exactly, and no gradient)
            w = sum == 0.f ? 0.f : w == sum ? 1.f : w * (1.f / sum);
            dw = w * (dw - warp_sum_all(dw * w)) * rest;
        } else {
            if (a.softmax) dot = dw * s;
            dw *= slope;
        }
        if (a.softmax) {
#pragma unroll
            for (int i = 0; i < PL; ++i) dot = fmaf(g[i], x[i], dot);
            dot = warp_sum_all(dot);
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
        if (id >= 0 && lane == __ffs(same) - 1) out[id] = IO<T>::from_f(fmaf(slope, gs - dot, dw));
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (route_<type>.cu).
// ---------------------------------------------------------------------------
template <typename K>
cudaError_t launch_route_k(K kernel, const RouteArgs &a, int per_cta, int pl, int sms, cudaStream_t s, Plan *p) {
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), kRouteThreads, 0, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t need = (a.tokens + per_cta - 1) / per_cta, most = (int64_t)sms * per_sm;
    p->kind = PLAN_WARP;
    p->threads = kRouteThreads;
    p->packs = pl;
    p->groups = per_cta;
    return launch_row(kernel, (unsigned)(need < most ? need : most), (unsigned)kRouteThreads, 0, s, a);
}

template <typename T, int PL> cudaError_t launch_route_n(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    constexpr int LOGIT = sizeof(T) == 2 ? KEY_WHOLE : KEY_LOGIT;
    auto kernel = back ? route_bwd_kernel<T, PL> : a.by_score ? route_fwd_kernel<T, PL, KEY_SCORE> : route_fwd_kernel<T, PL, LOGIT>;
    return launch_route_k(kernel, a, kRouteThreads / 32, PL, sms, s, p);
}
template <typename T, int NC> cudaError_t launch_route_oct(const RouteArgs &a, int sms, cudaStream_t s, Plan *p) {
    constexpr int LOGIT = sizeof(T) == 2 ? KEY_WHOLE : KEY_LOGIT;
    auto kernel = a.by_score ? route_oct_kernel<T, NC, KEY_SCORE> : route_oct_kernel<T, NC, LOGIT>;
    return launch_route_k(kernel, a, kRouteThreads / 8, 8 * NC, sms, s, p);
}

template <typename T> cudaError_t launch_route_t(const RouteArgs &a, bool back, int sms, cudaStream_t s, Plan *p) {
    if (!back && a.oct_per_lane) {
        if (a.oct_per_lane <= 8) return launch_route_oct<T, 1>(a, sms, s, p);
        if (a.oct_per_lane <= 16) return launch_route_oct<T, 2>(a, sms, s, p);
        return launch_route_oct<T, 4>(a, sms, s, p);
    }
    const int n = back ? (a.experts + 31) / 32 : a.per_lane;
    if (n <= 2) return launch_route_n<T, 2>(a, back, sms, s, p);
    if (n <= 4) return launch_route_n<T, 4>(a, back, sms, s, p);
    if (n <= 8) return launch_route_n<T, 8>(a, back, sms, s, p);
    if (n <= 16) return launch_route_n<T, 16>(a, back, sms, s, p);
    return launch_route_n<T, 32>(a, back, sms, s, p);
}

}  // namespace nrm
