// qk.cuh -- RMSNorm of each head's query and key with the position rotation
// behind it, and the gradient.  For a token at position p and a head's row x of
// D entries, with r = 1/sqrt(mean x^2 + eps) and y = x r w, the first `rot`
// entries turn in pairs (a, b) by the pair's angle, c and s its cosine and sine
// from row p of a table; the others stay y:
//
//   out_a = y_a c - y_b s        out_b = y_b c + y_a s
//
// Backward: g = dout turned by -angle, u = g w, and
//
//   dx = r (u - x r^2 mean(u x))        dw = sum over tokens and heads of g x r
//
// r comes from x again (which has to be read anyway), so the forward leaves
// nothing behind.  Two numbers are summed over a row, so a row belongs to a
// few lanes: 2 VE PP entries each, arranged so that both entries of a pair are
// in the same lane and a row needs no exchange but the sums.  The lanes' angles
// depend on the token alone and stay in registers over its heads.  HBM bounds
// it: each row once in, once out (backward: two in, one out).  16384 tokens x 40
// heads x 128 bf16: 58.8 us forward, 85 % of the measured copy rate, and 8192 of
// them 51 us backward, 73 %: there the registers of the weights' gradients leave 16
// warps an SM, whose loads in flight are too few.
//
// A token whose position lies outside the table takes no part: its rows are not
// read, its outputs and gradients are 0.
#pragma once

#include <cstdint>
#include <type_traits>

#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

// VE consecutive values in one access of 2 to 16 bytes, aligned to its size; in
// registers as H pairs for the packed binary32 arithmetic (VE = 1: the second of
// the pair is 0).
template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = unsigned short; };
template <typename T> struct Two16;
template <> struct Two16<__half> {
    __device__ __forceinline__ static float2 wide(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
    __device__ __forceinline__ static uint32_t narrow(float2 v) {
        const __half2 h = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <> struct Two16<__nv_bfloat16> {
    __device__ __forceinline__ static float2 wide(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t narrow(float2 v) {
        const __nv_bfloat162 h = __float22bfloat162_rn(v);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

template <typename T, int VE> struct Pk {
    static constexpr int BYTES = VE * (int)sizeof(T), H = VE > 1 ? VE / 2 : 1;
    using Raw = typename RawOf<BYTES>::type;
    union Words {
        Raw r;
        uint32_t w[BYTES >= 4 ? BYTES / 4 : 1];
        __device__ __forceinline__ Words() {}
    };
    // coherent: an output may replace its input in place
    __device__ __forceinline__ static Raw load(const T *p) {
        if constexpr (BYTES == 16) return ld_once(p);
        return *reinterpret_cast<const Raw *>(p);
    }
    __device__ __forceinline__ static void store(T *p, const float2 *f) {
        if constexpr (VE == 1) {
            *p = IO<T>::from_f(f[0].x);
        } else {
            Words w;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w.w[2 * i] = __float_as_uint(f[i].x);
                    w.w[2 * i + 1] = __float_as_uint(f[i].y);
                } else {
                    w.w[i] = Two16<T>::narrow(f[i]);
                }
            }
            if constexpr (BYTES == 16) st_stream(p, w.r);
            else *reinterpret_cast<Raw *>(p) = w.r;
        }
    }
    __device__ __forceinline__ static void unpack(const Raw &r, float2 *f) {
        if constexpr (VE == 1) {
            f[0] = make_float2(IO<T>::to_f(*reinterpret_cast<const T *>(&r)), 0.f);
        } else {
            Words w;
            w.r = r;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if constexpr (sizeof(T) == 4) f[i] = make_float2(__uint_as_float(w.w[2 * i]), __uint_as_float(w.w[2 * i + 1]));
                else f[i] = Two16<T>::wide(w.w[i]);
            }
        }
    }
    __device__ __forceinline__ static Raw all(float v) {
        if constexpr (VE == 1) {
            const T t = IO<T>::from_f(v);
            return *reinterpret_cast<const Raw *>(&t);
        } else {
            Words w;
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i) {
                if constexpr (sizeof(T) == 4) w.w[i] = __float_as_uint(v);
                else w.w[i] = Two16<T>::narrow(f2(v));
            }
            return w.r;
        }
    }
};

// N consecutive binary32 numbers of the table, aligned to min(N, 4) of them.
template <int N> __device__ __forceinline__ void ld_angles(const float *p, float *f) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
            f[i] = v.x;
            f[i + 1] = v.y;
            f[i + 2] = v.z;
            f[i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
        f[0] = v.x;
        f[1] = v.y;
    } else {
        f[0] = __ldg(p);
    }
}

// What a lane holds of a row: PP slots of two packs each, a and b.
//   CROSS   an entry of a pairs with the same one of b (halves; or neighbours
//           with packs of one entry); the entries that do not turn fill the
//           slots behind
//   else    the pairs are neighbours inside a pack
// Offsets of packs the row does not have are -1; with FULL it has them all.
template <int VE, int PP, bool CROSS, bool FULL> struct Slots {
    int a[PP], b[PP];
    __device__ __forceinline__ Slots(int l, int lanes, const QkArgs &q) {
        const int D = q.D, half = q.half;
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const int j = l + p * lanes;
            if (CROSS && VE == 1 && q.near) {
                a[p] = 2 * j < D ? 2 * j : -1;
                b[p] = 2 * j + 1 < D ? 2 * j + 1 : -1;
            } else {
                const int turn = CROSS ? half / VE : 0, still = D / VE - 2 * turn, first = (still + 1) / 2;
                const int i = j - turn;
                a[p] = i < 0 ? j * VE : i < first ? (2 * turn + i) * VE : -1;
                b[p] = i < 0 ? (j + turn) * VE : first + i < still ? (2 * turn + first + i) * VE : -1;
            }
        }
    }
    __device__ __forceinline__ bool has_a(int p) const { return FULL || a[p] >= 0; }
    __device__ __forceinline__ bool has_b(int p) const { return FULL || b[p] >= 0; }
    // Cosines and sines of one token; packs that do not turn get 1 and 0.  CROSS: one
    // pair of numbers for two entries of a and of b; else the angles of a's pairs,
    // then those of b's.
    static constexpr int H = VE > 1 ? VE / 2 : 1;
    __device__ __forceinline__ void angles(const QkArgs &q, int64_t pos, float2 (&c)[PP][H], float2 (&s)[PP][H]) const {
        const float *row = q.table + pos * (2 * q.half);
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            float cc[2 * H], ss[2 * H];
            cc[2 * H - 1] = ss[2 * H - 1] = 0.f;
            if constexpr (CROSS) {
                // the pair's first entry is a: its angle is a's place among the
                // first halves, or half its place among neighbours
                const int at = VE == 1 && q.near ? a[p] >> 1 : a[p];
                const bool on = has_a(p) && has_b(p) && at < q.half;
                get<VE>(row, at, on, q.half, cc, ss);
            } else {
                get<VE / 2>(row, a[p] / 2, has_a(p) && a[p] < 2 * q.half, q.half, cc, ss);
                get<VE / 2>(row, b[p] / 2, has_b(p) && b[p] < 2 * q.half, q.half, cc + VE / 2, ss + VE / 2);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                c[p][i] = make_float2(cc[2 * i], cc[2 * i + 1]);
                s[p][i] = make_float2(ss[2 * i], ss[2 * i + 1]);
            }
        }
    }
    template <int N>
    __device__ __forceinline__ static void get(const float *row, int at, bool on, int half, float *c, float *s) {
        if (on) {
            ld_angles<N>(row + at, c);
            ld_angles<N>(row + half + at, s);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                c[i] = 1.f;
                s[i] = 0.f;
            }
        }
    }
};

// Turn a slot by its angles, or (BACK) by the negative ones.
template <int VE, bool CROSS, bool BACK>
__device__ __forceinline__ void turn(float2 *a, float2 *b, const float2 *c, const float2 *s) {
    constexpr int H = VE > 1 ? VE / 2 : 1;
    if constexpr (CROSS) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 x = a[i], y = b[i], n = make_float2(-s[i].x, -s[i].y);
            a[i] = __ffma2_rn(x, c[i], __fmul2_rn(y, BACK ? s[i] : n));
            b[i] = __ffma2_rn(y, c[i], __fmul2_rn(x, BACK ? n : s[i]));
        }
    } else {
        auto one = [](float2 &v, float c, float s) {
            const float x = v.x, y = v.y, t = BACK ? -s : s;
            v.x = fmaf(x, c, -(y * t));
            v.y = fmaf(y, c, x * t);
        };
        // angle i of a slot is half a pair of numbers: a's come first
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int k = i, m = H + i;
            one(a[i], k % 2 ? c[k / 2].y : c[k / 2].x, k % 2 ? s[k / 2].y : s[k / 2].x);
            one(b[i], m % 2 ? c[m / 2].y : c[m / 2].x, m % 2 ? s[m / 2].y : s[m / 2].x);
        }
    }
}

constexpr int kQkThreads = 256;

// The heads [h0, h1) of one token and one side.
struct QkItem {
    int64_t token;
    int h0, h1;
};
__device__ __forceinline__ QkItem qk_item(int64_t id, int64_t total, int items, int heads, int of) {
    QkItem it;
    it.token = total <= 0xffffffffll ? (int64_t)((uint32_t)id / (uint32_t)items) : id / items;
    it.h0 = (int)(id - it.token * items) * heads;
    it.h1 = min(it.h0 + heads, of);
    return it;
}

// One row's packs of a lane, as they are in memory.
template <typename T, int VE, int PP> struct QkRow {
    typename Pk<T, VE>::Raw a[PP], b[PP];
    template <typename S> __device__ __forceinline__ void load(const T *row, const S &at) {
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            if (at.has_a(p)) a[p] = Pk<T, VE>::load(row + at.a[p]);
            else a[p] = Pk<T, VE>::all(0.f);
            if (at.has_b(p)) b[p] = Pk<T, VE>::load(row + at.b[p]);
            else b[p] = Pk<T, VE>::all(0.f);
        }
    }
};
template <typename T, int VE, int PP, typename S>
__device__ __forceinline__ void qk_store(T *row, const S &at, const float2 (&a)[PP][Pk<T, VE>::H],
                                         const float2 (&b)[PP][Pk<T, VE>::H]) {
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        if (at.has_a(p)) Pk<T, VE>::store(row + at.a[p], a[p]);
        if (at.has_b(p)) Pk<T, VE>::store(row + at.b[p], b[p]);
    }
}
// Zeros for the rows h, h + R, .. below h1.
template <typename T, int VE, int PP, typename S>
__device__ __forceinline__ void qk_zeros(T *out, int64_t stride, int h, int h1, int R, const S &at) {
    float2 zero[PP][Pk<T, VE>::H];
#pragma unroll
    for (int p = 0; p < PP; ++p)
#pragma unroll
        for (int i = 0; i < Pk<T, VE>::H; ++i) zero[p][i] = f2(0.f);
    for (; h < h1; h += R) qk_store<T, VE, PP>(out + h * stride, at, zero, zero);
}
// The weights of a lane's entries (none: ones).
template <typename T, int VE, int PP, typename S>
__device__ __forceinline__ void qk_weights(const void *w, const S &at, QkRow<T, VE, PP> &r) {
#pragma unroll
    for (int p = 0; p < PP; ++p) r.a[p] = r.b[p] = Pk<T, VE>::all(1.f);
    if (w) r.load(static_cast<const T *>(w), at);
}
// Sum over the lanes of a row: 2^LL of them, or (LL < 0) `lanes`.
template <int LL> __device__ __forceinline__ float qk_sum(float v, int lanes) {
    if constexpr (LL >= 0) {
        return group_sum_all<1 << (LL > 0 ? LL : 0)>(v);
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

// Rows a lane has on its way at once, forward.  With 80 registers and three CTAs
// an SM two rows are ahead of four with 108 and two (16384 x 40 x 128 bf16 58.8 us
// and 59.8, f32 8192 x 20 x 128 27.0 and 29.7); pairs inside a pack need more
// registers, there four rows are (8192 x 32 x 128 24.2 us and 26.5), and so without a
// constant number of lanes, where an item costs more beside its rows (8192 x 32 x
// 80, half of it turned, 28.1 us and 32.0).
template <int VE, int PP, bool CROSS, int ES, int LL>
constexpr int kQkFwdRows = PP > 1 || ES == 4 || (CROSS && LL >= 0) ? 2 : 4;

// Forward.  One warp an item of U times 32 / lanes rows, all of whose loads are in
// flight together.  LL >= 0: every lane of 2^LL has its two packs.
template <typename T, int VE, int PP, bool CROSS, int LL, int U>
__global__ void __launch_bounds__(kQkThreads, PP > 1 ? 1 : U == 2 ? 3 : 2) qk_fwd_kernel(const QkArgs q, const int log_lanes,
                                                                             const int q_items, const int items) {
    using P = Pk<T, VE>;
    constexpr int H = P::H;
    const int lane = threadIdx.x & 31, lanes = LL >= 0 ? 1 << (LL > 0 ? LL : 0) : 1 << log_lanes, l = lane & (lanes - 1),
              sub = lane / lanes, R = 32 / lanes;
    const Slots<VE, PP, CROSS, (LL >= 0)> at(l, lanes, q);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = q.tokens * items, step = (int64_t)gridDim.x * (kQkThreads / 32);
    for (int64_t id = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); id < total; id += step) {
        QkItem it = qk_item(id, total, items, R * U, 0);
        const bool keys = it.h0 >= q_items * (R * U);
        const QkSide &sd = q.side[keys];
        if (keys) it.h0 -= q_items * (R * U);
        it.h1 = min(it.h0 + R * U, sd.heads);
        const int64_t pos = q.pos[it.token];
        const T *x = static_cast<const T *>(sd.x) + it.token * sd.xt + (it.h0 + sub) * sd.xh;
        T *out = static_cast<T *>(sd.out) + it.token * sd.ot + (it.h0 + sub) * sd.oh;
        if (pos < 0 || pos >= q.max_pos) {
            qk_zeros<T, VE, PP>(out - (it.h0 + sub) * sd.oh, sd.oh, it.h0 + sub, it.h1, R, at);
            continue;
        }
        const int n = it.h1 - it.h0;  // rows
        QkRow<T, VE, PP> rows[U], w;
#pragma unroll
        for (int u = 0; u < U; ++u)
            // a row past the last is not loaded, and counts nowhere
            if (u * R + sub < n) rows[u].load(x + u * R * sd.xh, at);
        float2 c[PP][H], s[PP][H];
        at.angles(q, pos, c, s);
        qk_weights<T, VE, PP>(sd.w, at, w);
        // Weights and angles in one: with ca = w_a c, sb = w_b s, cb = w_b c, sa =
        // w_a s a row turns as r (a ca - b sb), r (b cb + a sa).  Pairs inside a pack
        // take them one after the other.
        float2 wa[PP][H], wb[PP][H], sa[PP][H], sb[PP][H];
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            P::unpack(w.a[p], wa[p]);
            P::unpack(w.b[p], wb[p]);
            if constexpr (CROSS) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    sa[p][i] = __fmul2_rn(wa[p][i], s[p][i]);
                    sb[p][i] = __fmul2_rn(wb[p][i], make_float2(-s[p][i].x, -s[p][i].y));
                    wa[p][i] = __fmul2_rn(wa[p][i], c[p][i]);
                    wb[p][i] = __fmul2_rn(wb[p][i], c[p][i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * R >= n) break;
            float2 a[PP][H], b[PP][H], ss = f2(0.f);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                P::unpack(rows[u].a[p], a[p]);
                P::unpack(rows[u].b[p], b[p]);
#pragma unroll
                for (int i = 0; i < H; ++i) ss = __ffma2_rn(a[p][i], a[p][i], __ffma2_rn(b[p][i], b[p][i], ss));
            }
            const float2 r = f2(rsqrtf(fmaf(qk_sum<LL>(ss.x + ss.y, lanes), q.invD, q.eps)));
#pragma unroll
            for (int p = 0; p < PP; ++p) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 x = __fmul2_rn(a[p][i], r), y = __fmul2_rn(b[p][i], r);
                    if constexpr (CROSS) {
                        a[p][i] = __ffma2_rn(x, wa[p][i], __fmul2_rn(y, sb[p][i]));
                        b[p][i] = __ffma2_rn(y, wb[p][i], __fmul2_rn(x, sa[p][i]));
                    } else {
                        a[p][i] = __fmul2_rn(x, wa[p][i]);
                        b[p][i] = __fmul2_rn(y, wb[p][i]);
                    }
                }
                if constexpr (!CROSS) turn<VE, CROSS, false>(a[p], b[p], c[p], s[p]);
            }
            if (u * R + sub < n) qk_store<T, VE, PP>(out + u * R * sd.oh, at, a, b);
        }
    }
}

// Backward.  The grid is resident at once; every warp goes over a share of the
// queries' items, then of the keys', a row a lane group at a time, the next one's
// packs on their way, with the weight's gradient of its entries in registers.
// The CTA joins those (rows of a warp by shuffles, warps in shared memory, both
// in a fixed order) and leaves one partial row for each of the two, [CTA][2][D];
// qk_fold_kernel adds those up.
template <typename T, int VE, int PP, bool CROSS, int LL>
__global__ void __launch_bounds__(kQkThreads, PP > 1 ? 1 : 2) qk_bwd_kernel(const QkArgs q, const int log_lanes,
                                                                             const int heads_q, const int heads_k) {
    using P = Pk<T, VE>;
    constexpr int NW = kQkThreads / 32, H = P::H;
    extern __shared__ float join[];  // [NW][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5,
              lanes = LL >= 0 ? 1 << (LL > 0 ? LL : 0) : 1 << log_lanes, l = lane & (lanes - 1), sub = lane / lanes,
              R = 32 / lanes;
    const Slots<VE, PP, CROSS, (LL >= 0)> at(l, lanes, q);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = (int64_t)gridDim.x * NW;
    int64_t id = (int64_t)blockIdx.x * NW + warp;
    for (int keys = 0; keys < 2; ++keys) {
        const QkSide &sd = q.side[keys];
        if (sd.heads == 0) break;
        const int heads = keys ? heads_k : heads_q, items = (sd.heads + heads - 1) / heads;
        const int64_t total = q.tokens * items;
        QkRow<T, VE, PP> w;
        qk_weights<T, VE, PP>(sd.w, at, w);
        float2 dwa[PP][H], dwb[PP][H];
#pragma unroll
        for (int p = 0; p < PP; ++p)
#pragma unroll
            for (int i = 0; i < H; ++i) dwa[p][i] = dwb[p][i] = f2(0.f);
        // the next item whose token takes part (the others get their zeros); the
        // position of the one after is on its way
        auto token_at = [&](int64_t i) { return q.pos[qk_item(i, total, items, heads, 0).token]; };
        int64_t coming = id < total ? token_at(id) : -1;
        auto next_live = [&](QkItem &it, int64_t &pos) {
            while (id < total) {
                it = qk_item(id, total, items, heads, sd.heads);
                pos = coming;
                id += step;
                if (id < total) coming = token_at(id);
                if (pos >= 0 && pos < q.max_pos) return true;
                qk_zeros<T, VE, PP>(static_cast<T *>(sd.out) + it.token * sd.ot, sd.oh, it.h0 + sub, it.h1, R, at);
            }
            return false;
        };
        QkItem it, next;
        int64_t pos, pos_n;
        QkRow<T, VE, PP> xr, gr;
        float2 c[PP][H], s[PP][H];
        auto load = [&](const QkItem &i, int h) {
            if (h < i.h1) {
                xr.load(static_cast<const T *>(sd.x) + i.token * sd.xt + h * sd.xh, at);
                gr.load(static_cast<const T *>(sd.dy) + i.token * sd.dt + h * sd.dh, at);
            }
        };
        if (next_live(it, pos)) {
            load(it, it.h0 + sub);
            at.angles(q, pos, c, s);
            bool more = next_live(next, pos_n);
            for (int hb = it.h0;;) {
                const bool last = hb + R >= it.h1, on = hb + sub < it.h1;
                float2 a[PP][H], b[PP][H], ua[PP][H], ub[PP][H], va[H], vb[H], ss = f2(0.f), ux = f2(0.f);
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    P::unpack(xr.a[p], a[p]);
                    P::unpack(xr.b[p], b[p]);
                    P::unpack(gr.a[p], ua[p]);
                    P::unpack(gr.b[p], ub[p]);
                }
                if (!last) load(it, hb + R + sub);
                else if (more) load(next, next.h0 + sub);
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    turn<VE, CROSS, true>(ua[p], ub[p], c[p], s[p]);
                    P::unpack(w.a[p], va);
                    P::unpack(w.b[p], vb);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        ss = __ffma2_rn(a[p][i], a[p][i], __ffma2_rn(b[p][i], b[p][i], ss));
                        ux = __ffma2_rn(__fmul2_rn(ua[p][i], va[i]), a[p][i],
                                        __ffma2_rn(__fmul2_rn(ub[p][i], vb[i]), b[p][i], ux));
                    }
                }
                if (last && more) at.angles(q, pos_n, c, s);
                const float sum = qk_sum<LL>(ss.x + ss.y, lanes), dot = qk_sum<LL>(ux.x + ux.y, lanes);
                const float r = rsqrtf(fmaf(sum, q.invD, q.eps));
                const float2 rr = f2(r), m = f2(-(r * (dot * q.invD)));
                if (on) {
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        P::unpack(w.a[p], va);
                        P::unpack(w.b[p], vb);
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            // x r, whose product with r mean(u x) is x r^2 mean(u x)
                            const float2 ha = __fmul2_rn(a[p][i], rr), hb2 = __fmul2_rn(b[p][i], rr);
                            dwa[p][i] = __ffma2_rn(ua[p][i], ha, dwa[p][i]);
                            dwb[p][i] = __ffma2_rn(ub[p][i], hb2, dwb[p][i]);
                            a[p][i] = __fmul2_rn(__ffma2_rn(ha, m, __fmul2_rn(ua[p][i], va[i])), rr);
                            b[p][i] = __fmul2_rn(__ffma2_rn(hb2, m, __fmul2_rn(ub[p][i], vb[i])), rr);
                        }
                    }
                    qk_store<T, VE, PP>(static_cast<T *>(sd.out) + it.token * sd.ot + (hb + sub) * sd.oh, at, a, b);
                }
                hb += R;
                if (last) {
                    if (!more) break;
                    it = next;
                    hb = it.h0;
                    more = next_live(next, pos_n);
                }
            }
        }
        id -= total;
        if (q.part) {
            auto join_one = [&](float v, int i) {
                for (int o = 16; o >= lanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (sub == 0 && i >= 0) join[warp * q.D + i] = v;
            };
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    join_one(i % 2 ? dwa[p][i / 2].y : dwa[p][i / 2].x, at.has_a(p) ? at.a[p] + i : -1);
                    join_one(i % 2 ? dwb[p][i / 2].y : dwb[p][i / 2].x, at.has_b(p) ? at.b[p] + i : -1);
                }
            __syncthreads();
            for (int i = threadIdx.x; i < q.D; i += kQkThreads) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k) v += join[k * q.D + i];
                q.part[((int64_t)blockIdx.x * 2 + keys) * q.D + i] = v;
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (qk_<type>.cu).
// ---------------------------------------------------------------------------
inline int qk_log_lanes(const QkArgs &q, int ve, int pp, bool cross) {
    int slots;
    if (cross && !q.near) {
        const int turn = q.half / ve, still = q.D / ve - 2 * turn;
        slots = turn + (still + 1) / 2;
    } else {
        slots = (q.D / ve + 1) / 2;
    }
    int log = 0;
    while ((1 << log) * pp < slots) ++log;
    return log;  // at most 5 by the choice of pp
}

template <typename T, int VE, int PP, bool CROSS, int LL>
cudaError_t launch_qk_one(const QkArgs &q, int log, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const int R = 32 >> log;
    p->kind = PLAN_WARP;
    p->threads = kQkThreads;
    p->packs = VE;
    p->groups = 1 << log;
    if (!back) {
        constexpr int U = kQkFwdRows<VE, PP, CROSS, (int)sizeof(T), LL>;
        const int heads = R * U;
        const int q_items = (q.side[0].heads + heads - 1) / heads, items = q_items + (q.side[1].heads + heads - 1) / heads;
        const int64_t n = (q.tokens * items + kQkThreads / 32 - 1) / (kQkThreads / 32);
        return launch_row(qk_fwd_kernel<T, VE, PP, CROSS, LL, U>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff),
                          (unsigned)kQkThreads, 0, s, q, log, q_items, items);
    }
    constexpr int NW = kQkThreads / 32;
    auto kernel = qk_bwd_kernel<T, VE, PP, CROSS, LL>;
    const size_t smem = (size_t)NW * q.D * 4;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), kQkThreads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t most = (int64_t)sms * per_sm;
    if (most > kDropMaxParts) most = kDropMaxParts;
    // heads an item: as many steps as leave every warp some items
    auto heads = [&](int n) {
        const int steps = (n + R - 1) / R;
        int at_once = steps < 4 ? steps : 4;
        while (at_once > 1 && q.tokens * ((steps + at_once - 1) / at_once) < most * NW * 4) at_once = (at_once + 1) / 2;
        return at_once * R;
    };
    const int heads_q = heads(q.side[0].heads), heads_k = q.side[1].heads ? heads(q.side[1].heads) : 1;
    const int64_t work = q.tokens * ((q.side[0].heads + heads_q - 1) / heads_q + (q.side[1].heads + heads_k - 1) / heads_k);
    const int64_t need = (work + NW - 1) / NW, n = need < most ? need : most;
    *parts = n;
    return launch_row(kernel, (unsigned)n, (unsigned)kQkThreads, smem, s, q, log, heads_q, heads_k);
}

// Rows whose packs fill a power of two of lanes have kernels of their own.
template <typename T, int VE, int PP, bool CROSS>
cudaError_t launch_qk_lanes(const QkArgs &q, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const int log = qk_log_lanes(q, VE, PP, CROSS);
    const bool full = 2 * VE * PP << log == q.D && (!CROSS || !q.near) && (!CROSS || (q.D / VE - 2 * (q.half / VE)) % 2 == 0);
    if constexpr (VE == IO<T>::V && PP == 1) {
        constexpr int L = VE == 8 ? 2 : 3;  // D = 64, 128, 256
        if (full && log == L) return launch_qk_one<T, VE, PP, CROSS, L>(q, log, back, sms, s, p, parts);
        if (full && log == L + 1) return launch_qk_one<T, VE, PP, CROSS, L + 1>(q, log, back, sms, s, p, parts);
        if (full && log == L + 2) return launch_qk_one<T, VE, PP, CROSS, L + 2>(q, log, back, sms, s, p, parts);
    }
    return launch_qk_one<T, VE, PP, CROSS, -1>(q, log, back, sms, s, p, parts);
}

// ve: the widest access that every row, weight and table row allows.  Rows of
// more than 64 entries a lane-pair of that width take several slots a lane.
template <typename T>
cudaError_t launch_qk_t(const QkArgs &q, int ve, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const bool wide = q.D > 64 * ve;  // more than 32 lanes of one slot
    if constexpr (IO<T>::V == 8) {
        if (ve == 8)
            return q.near ? launch_qk_lanes<T, 8, 1, false>(q, back, sms, s, p, parts)
                          : launch_qk_lanes<T, 8, 1, true>(q, back, sms, s, p, parts);
    }
    if (ve == 4) {
        if (q.near)
            return wide ? launch_qk_lanes<T, 4, 2, false>(q, back, sms, s, p, parts)
                        : launch_qk_lanes<T, 4, 1, false>(q, back, sms, s, p, parts);
        return wide ? launch_qk_lanes<T, 4, 2, true>(q, back, sms, s, p, parts)
                    : launch_qk_lanes<T, 4, 1, true>(q, back, sms, s, p, parts);
    }
    if (ve == 2) {
        if (q.near)
            return wide ? launch_qk_lanes<T, 2, 4, false>(q, back, sms, s, p, parts)
                        : launch_qk_lanes<T, 2, 1, false>(q, back, sms, s, p, parts);
        return wide ? launch_qk_lanes<T, 2, 4, true>(q, back, sms, s, p, parts)
                    : launch_qk_lanes<T, 2, 1, true>(q, back, sms, s, p, parts);
    }
    return wide ? launch_qk_lanes<T, 1, 8, true>(q, back, sms, s, p, parts)
                : launch_qk_lanes<T, 1, 1, true>(q, back, sms, s, p, parts);
}

}  // namespace nrm
