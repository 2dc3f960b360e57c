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
// it: each row once in, once out (backward: two in, one out).
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

// VE consecutive values in one access of 2 to 16 bytes, aligned to its size.
template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = unsigned short; };

template <typename T, int VE> struct Pk {
    static constexpr int BYTES = VE * (int)sizeof(T);
    using Raw = typename RawOf<BYTES>::type;
    union Words {
        Raw r;
        T t[VE];
        __device__ __forceinline__ Words() {}
    };
    // coherent: an output may replace its input in place
    __device__ __forceinline__ static Raw load(const T *p) {
        if constexpr (BYTES == 16) return ld_once(p);
        return *reinterpret_cast<const Raw *>(p);
    }
    __device__ __forceinline__ static void store(T *p, const float *f) {
        Words w;
#pragma unroll
        for (int i = 0; i < VE; ++i) w.t[i] = IO<T>::from_f(f[i]);
        if constexpr (BYTES == 16) st_stream(p, w.r);
        else *reinterpret_cast<Raw *>(p) = w.r;
    }
    __device__ __forceinline__ static void unpack(const Raw &r, float *f) {
        Words w;
        w.r = r;
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = IO<T>::to_f(w.t[i]);
    }
    __device__ __forceinline__ static Raw all(float v) {
        Words w;
#pragma unroll
        for (int i = 0; i < VE; ++i) w.t[i] = IO<T>::from_f(v);
        return w.r;
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
// Offsets of packs the row does not have are -1; angle -1 does not turn.
template <int VE, int PP, bool CROSS> struct Slots {
    int a[PP], b[PP];
    __device__ __forceinline__ Slots(int l, int lanes, const QkArgs &q) {
        const int D = q.D, half = q.half;
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const int j = l + p * lanes;
            if (CROSS && q.near) {  // VE = 1
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
    // cosines and sines of one token; packs that do not turn get 1 and 0
    __device__ __forceinline__ void angles(const QkArgs &q, int64_t pos, float (&c)[PP][VE], float (&s)[PP][VE]) const {
        const float *row = q.table + pos * (2 * q.half);
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            if constexpr (CROSS) {
                // the pair's first entry is a: its angle is a's place among the
                // first halves, or half its place among neighbours
                const int at = q.near ? a[p] >> 1 : a[p];
                const bool on = a[p] >= 0 && b[p] >= 0 && at < q.half;
                get<VE>(row, at, on, q.half, c[p], s[p]);
            } else {
                get<VE / 2>(row, a[p] / 2, a[p] >= 0 && a[p] < 2 * q.half, q.half, c[p], s[p]);
                get<VE / 2>(row, b[p] / 2, b[p] >= 0 && b[p] < 2 * q.half, q.half, c[p] + VE / 2, s[p] + VE / 2);
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

// Turn a slot by its angles (sign = 1) or back (sign = -1).
template <int VE, bool CROSS>
__device__ __forceinline__ void turn(float *a, float *b, const float *c, const float *s, float sign) {
    if constexpr (CROSS) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float t = sign * s[i], x = a[i], y = b[i];
            a[i] = fmaf(x, c[i], -(y * t));
            b[i] = fmaf(y, c[i], x * t);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const float t = sign * s[i], x = a[2 * i], y = a[2 * i + 1];
            a[2 * i] = fmaf(x, c[i], -(y * t));
            a[2 * i + 1] = fmaf(y, c[i], x * t);
            const float u = sign * s[VE / 2 + i], z = b[2 * i], w = b[2 * i + 1];
            b[2 * i] = fmaf(z, c[VE / 2 + i], -(w * u));
            b[2 * i + 1] = fmaf(w, c[VE / 2 + i], z * u);
        }
    }
}

constexpr int kQkThreads = 256;

// Forward.  One warp an item: `heads` heads of the queries or of the keys of one
// token, 32 / lanes rows at a time, U such steps' loads in flight together.
template <typename T, int VE, int PP, bool CROSS, int U>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(const QkArgs q, const int log_lanes, const int heads,
                                                            const int q_items, const int items) {
    using P = Pk<T, VE>;
    const int lane = threadIdx.x & 31, lanes = 1 << log_lanes, l = lane & (lanes - 1), sub = lane >> log_lanes,
              R = 32 >> log_lanes;
    const Slots<VE, PP, CROSS> at(l, lanes, q);
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = q.tokens * items, step = (int64_t)gridDim.x * (kQkThreads / 32);
    for (int64_t id = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); id < total; id += step) {
        const int64_t token = total <= 0xffffffffll ? (int64_t)((uint32_t)id / (uint32_t)items) : id / items;
        const int item = (int)(id - token * items);
        const bool keys = item >= q_items;
        const QkSide &sd = q.side[keys];
        const int h0 = (keys ? item - q_items : item) * heads, h1 = min(h0 + heads, sd.heads);
        const int64_t pos = q.pos[token];
        const bool live = pos >= 0 && pos < q.max_pos;
        const T *x = static_cast<const T *>(sd.x) + token * sd.xt;
        T *out = static_cast<T *>(sd.out) + token * sd.ot;
        const T *w = static_cast<const T *>(sd.w);
        typename P::Raw wa[PP], wb[PP];
        float c[PP][VE], s[PP][VE];
        if (live) {
            at.angles(q, pos, c, s);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                wa[p] = w && at.a[p] >= 0 ? P::load(w + at.a[p]) : P::all(1.f);
                wb[p] = w && at.b[p] >= 0 ? P::load(w + at.b[p]) : P::all(1.f);
            }
        }
        for (int hb = h0; hb < h1; hb += R * U) {
            typename P::Raw ra[U][PP], rb[U][PP];
            if (live) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = hb + u * R + sub;
                    const T *row = x + h * sd.xh;
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        ra[u][p] = rb[u][p] = P::all(0.f);
                        if (h < h1 && at.a[p] >= 0) ra[u][p] = P::load(row + at.a[p]);
                        if (h < h1 && at.b[p] >= 0) rb[u][p] = P::load(row + at.b[p]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = hb + u * R + sub;
                T *row = out + h * sd.oh;
                float a[PP][VE], b[PP][VE], ss = 0.f;
                if (live) {
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        P::unpack(ra[u][p], a[p]);
                        P::unpack(rb[u][p], b[p]);
#pragma unroll
                        for (int i = 0; i < VE; ++i) ss = fmaf(a[p][i], a[p][i], fmaf(b[p][i], b[p][i], ss));
                    }
                    for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(fmaf(ss, q.invD, q.eps));
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        float wf[VE];
                        P::unpack(wa[p], wf);
#pragma unroll
                        for (int i = 0; i < VE; ++i) a[p][i] = a[p][i] * r * wf[i];
                        P::unpack(wb[p], wf);
#pragma unroll
                        for (int i = 0; i < VE; ++i) b[p][i] = b[p][i] * r * wf[i];
                        turn<VE, CROSS>(a[p], b[p], c[p], s[p], 1.f);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < PP; ++p)
#pragma unroll
                        for (int i = 0; i < VE; ++i) a[p][i] = b[p][i] = 0.f;
                }
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    if (h < h1 && at.a[p] >= 0) P::store(row + at.a[p], a[p]);
                    if (h < h1 && at.b[p] >= 0) P::store(row + at.b[p], b[p]);
                }
            }
        }
    }
}

// Backward.  The grid is resident at once; every warp goes over a share of the
// queries' items, then of the keys', with the weight's gradient of its entries
// in registers, which the CTA joins (rows of a warp by shuffles, warps in
// shared memory, both in a fixed order) and leaves as one partial row for each
// of the two, [CTA][2][D]; qk_fold_kernel adds those up.
template <typename T, int VE, int PP, bool CROSS, int U>
__global__ void __launch_bounds__(kQkThreads) qk_bwd_kernel(const QkArgs q, const int log_lanes, const int heads) {
    using P = Pk<T, VE>;
    constexpr int NW = kQkThreads / 32;
    extern __shared__ float join[];  // [NW][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = 1 << log_lanes, l = lane & (lanes - 1),
              sub = lane >> log_lanes, R = 32 >> log_lanes;
    const Slots<VE, PP, CROSS> at(l, lanes, q);
    pdl_wait();
    pdl_launch_dependents();
    for (int keys = 0; keys < 2; ++keys) {
        const QkSide &sd = q.side[keys];
        if (sd.heads == 0) continue;
        const int items = (sd.heads + heads - 1) / heads;
        const T *w = static_cast<const T *>(sd.w);
        typename P::Raw wa[PP], wb[PP];
        float dwa[PP][VE], dwb[PP][VE];
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            wa[p] = w && at.a[p] >= 0 ? P::load(w + at.a[p]) : P::all(1.f);
            wb[p] = w && at.b[p] >= 0 ? P::load(w + at.b[p]) : P::all(1.f);
#pragma unroll
            for (int i = 0; i < VE; ++i) dwa[p][i] = dwb[p][i] = 0.f;
        }
        const int64_t total = q.tokens * items, step = (int64_t)gridDim.x * NW;
        for (int64_t id = (int64_t)warp * gridDim.x + blockIdx.x; id < total; id += step) {
            const int64_t token = total <= 0xffffffffll ? (int64_t)((uint32_t)id / (uint32_t)items) : id / items;
            const int h0 = (int)(id - token * items) * heads, h1 = min(h0 + heads, sd.heads);
            const int64_t pos = q.pos[token];
            const bool live = pos >= 0 && pos < q.max_pos;
            const T *x = static_cast<const T *>(sd.x) + token * sd.xt, *dy = static_cast<const T *>(sd.dy) + token * sd.dt;
            T *out = static_cast<T *>(sd.out) + token * sd.ot;
            float c[PP][VE], s[PP][VE];
            if (live) at.angles(q, pos, c, s);
            for (int hb = h0; hb < h1; hb += R * U) {
                typename P::Raw xa[U][PP], xb[U][PP], ga[U][PP], gb[U][PP];
                if (live) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int h = hb + u * R + sub;
                        const T *xr = x + h * sd.xh, *gr = dy + h * sd.dh;
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            xa[u][p] = xb[u][p] = ga[u][p] = gb[u][p] = P::all(0.f);
                            if (h < h1 && at.a[p] >= 0) {
                                xa[u][p] = P::load(xr + at.a[p]);
                                ga[u][p] = P::load(gr + at.a[p]);
                            }
                            if (h < h1 && at.b[p] >= 0) {
                                xb[u][p] = P::load(xr + at.b[p]);
                                gb[u][p] = P::load(gr + at.b[p]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = hb + u * R + sub;
                    const bool on = h < h1;
                    T *row = out + h * sd.oh;
                    float a[PP][VE], b[PP][VE], ua[PP][VE], ub[PP][VE];
                    if (live) {
                        float ss = 0.f, ux = 0.f;
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            P::unpack(xa[u][p], a[p]);
                            P::unpack(xb[u][p], b[p]);
                            P::unpack(ga[u][p], ua[p]);
                            P::unpack(gb[u][p], ub[p]);
                            turn<VE, CROSS>(ua[p], ub[p], c[p], s[p], -1.f);
                            float va[VE], vb[VE];
                            P::unpack(wa[p], va);
                            P::unpack(wb[p], vb);
#pragma unroll
                            for (int i = 0; i < VE; ++i) {
                                ss = fmaf(a[p][i], a[p][i], fmaf(b[p][i], b[p][i], ss));
                                ux = fmaf(ua[p][i] * va[i], a[p][i], fmaf(ub[p][i] * vb[i], b[p][i], ux));
                            }
                        }
                        for (int o = lanes >> 1; o > 0; o >>= 1) {
                            ss += __shfl_xor_sync(0xffffffffu, ss, o);
                            ux += __shfl_xor_sync(0xffffffffu, ux, o);
                        }
                        const float r = rsqrtf(fmaf(ss, q.invD, q.eps));
                        const float m = on ? r * (r * (ux * q.invD)) : 0.f;
#pragma unroll
                        for (int p = 0; p < PP; ++p) {
                            float va[VE], vb[VE];
                            P::unpack(wa[p], va);
                            P::unpack(wb[p], vb);
#pragma unroll
                            for (int i = 0; i < VE; ++i) {
                                // rows past the last are zeros with r = 1/sqrt(eps): no share
                                if (on) {
                                    dwa[p][i] = fmaf(ua[p][i], a[p][i] * r, dwa[p][i]);
                                    dwb[p][i] = fmaf(ub[p][i], b[p][i] * r, dwb[p][i]);
                                }
                                a[p][i] = r * fmaf(ua[p][i], va[i], -(a[p][i] * m));
                                b[p][i] = r * fmaf(ub[p][i], vb[i], -(b[p][i] * m));
                            }
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < PP; ++p)
#pragma unroll
                            for (int i = 0; i < VE; ++i) a[p][i] = b[p][i] = 0.f;
                    }
#pragma unroll
                    for (int p = 0; p < PP; ++p) {
                        if (on && at.a[p] >= 0) P::store(row + at.a[p], a[p]);
                        if (on && at.b[p] >= 0) P::store(row + at.b[p], b[p]);
                    }
                }
            }
        }
        if (q.part) {
#pragma unroll
            for (int p = 0; p < PP; ++p) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    for (int o = 16; o >= lanes; o >>= 1) {
                        dwa[p][i] += __shfl_xor_sync(0xffffffffu, dwa[p][i], o);
                        dwb[p][i] += __shfl_xor_sync(0xffffffffu, dwb[p][i], o);
                    }
                    if (sub == 0) {
                        if (at.a[p] >= 0) join[warp * q.D + at.a[p] + i] = dwa[p][i];
                        if (at.b[p] >= 0) join[warp * q.D + at.b[p] + i] = dwb[p][i];
                    }
                }
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

template <typename T, int VE, int PP, bool CROSS>
cudaError_t launch_qk_one(const QkArgs &q, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const int log = qk_log_lanes(q, VE, PP, CROSS), R = 32 >> log;
    constexpr int REG = VE * PP * (int)sizeof(T) / 16 > 0 ? VE * PP * (int)sizeof(T) / 16 : 1;  // 32-byte slots a row
    p->kind = PLAN_WARP;
    p->threads = kQkThreads;
    p->packs = VE;
    p->groups = 1 << log;
    if (!back) {
        constexpr int U = REG > 1 ? 2 : 4;
        const int heads = R * U;
        const int q_items = (q.side[0].heads + heads - 1) / heads, items = q_items + (q.side[1].heads + heads - 1) / heads;
        const int64_t n = (q.tokens * items + kQkThreads / 32 - 1) / (kQkThreads / 32);
        return launch_row(qk_fwd_kernel<T, VE, PP, CROSS, U>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff),
                          (unsigned)kQkThreads, 0, s, q, log, heads, q_items, items);
    }
    constexpr int U = REG > 1 ? 1 : 2;
    const int heads = R * U;
    auto kernel = qk_bwd_kernel<T, VE, PP, CROSS, U>;
    const size_t smem = (size_t)(kQkThreads / 32) * q.D * 4;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), kQkThreads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t n = (int64_t)sms * per_sm;
    const int most = q.side[0].heads > q.side[1].heads ? q.side[0].heads : q.side[1].heads;
    const int64_t need = (q.tokens * ((most + heads - 1) / heads) + kQkThreads / 32 - 1) / (kQkThreads / 32);
    if (n > need) n = need;
    if (n > kDropMaxParts) n = kDropMaxParts;
    if (n < 1) n = 1;
    *parts = n;
    return launch_row(kernel, (unsigned)n, (unsigned)kQkThreads, smem, s, q, log, heads);
}

// ve: the widest access that every row, weight and table row allows.  Rows of
// more than 64 entries a lane-pair of that width take several slots a lane.
template <typename T>
cudaError_t launch_qk_t(const QkArgs &q, int ve, bool back, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const bool wide = q.D > 64 * ve;  // more than 32 lanes of one slot
    if constexpr (IO<T>::V == 8) {
        if (ve == 8)
            return q.near ? launch_qk_one<T, 8, 1, false>(q, back, sms, s, p, parts)
                          : launch_qk_one<T, 8, 1, true>(q, back, sms, s, p, parts);
    }
    if (ve == 4) {
        if (q.near)
            return wide ? launch_qk_one<T, 4, 2, false>(q, back, sms, s, p, parts)
                        : launch_qk_one<T, 4, 1, false>(q, back, sms, s, p, parts);
        return wide ? launch_qk_one<T, 4, 2, true>(q, back, sms, s, p, parts)
                    : launch_qk_one<T, 4, 1, true>(q, back, sms, s, p, parts);
    }
    if (ve == 2) {
        if (q.near)
            return wide ? launch_qk_one<T, 2, 4, false>(q, back, sms, s, p, parts)
                        : launch_qk_one<T, 2, 1, false>(q, back, sms, s, p, parts);
        return wide ? launch_qk_one<T, 2, 4, true>(q, back, sms, s, p, parts)
                    : launch_qk_one<T, 2, 1, true>(q, back, sms, s, p, parts);
    }
    return wide ? launch_qk_one<T, 1, 8, true>(q, back, sms, s, p, parts)
                : launch_qk_one<T, 1, 1, true>(q, back, sms, s, p, parts);
}

}  // namespace nrm
