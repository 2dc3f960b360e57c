// logits_top.cuh -- the log-probability of one target per row of logits with the
// row's entropy and its k largest alternatives, and the gradient of all three.
// With s the inverse temperature, c = s log2(e), m the row's maximum and
// x_j = (z_j - m) c,
//
//   d = sum_j 2^x_j,  A = sum_j 2^x_j x_j
//   lp_j = s (z_j - m) - log d          logp = lp_target
//   H = -sum_j p_j lp_j = log d - log(2) A / d
//
// all in the one pass that the log-probability alone takes (logits.cuh): A is
// rescaled like d, and moves by d times the shift when the maximum does.  The k
// largest logits (ties: the lowest index first) come out of the same pass.  A
// thread keeps the maximum of each group of packs it has seen.  At the row's
// end the k-th largest of some threads' own maxima, T (a row of one warp: of its
// lanes'; of a CTA: of each warp's four or eight largest), is a lower bound of the
// k-th largest logit, for k threads' maxima are k logits; so only groups whose
// maximum reaches T can hold one of the k largest, and there are hardly more than
// k of those.  A CTA reads them again, from L2; their logits from T on go, as
// 64-bit keys (value, then lower index first), into a sorted list of 32 that each
// warp keeps one entry a lane, and an entry's rank among all lists is its place.
// (One warp ranks the logits from T on without lists, up to 256 of them.)  Where
// many logits equal T (masked by one finite value, say) the groups are in index
// order, and later ones of no larger maximum are left out.
//
// The gradient for g of logp, h of H and a_i of the alternatives' lp:
//   dz_j = s (g [j = target] + sum_i a_i [j = id_i] - p_j (g + sum_i a_i + h (lp_j + H)))
#pragma once

#include "logits.cuh"

namespace nrm {

__device__ __forceinline__ uint32_t top_ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 counts as 0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float top_value(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t kTopNone = 0x007fffffu;  // of -inf: nothing up to it is a candidate

// A key: larger values first, then lower indices.  0: none.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t index) {
    return (uint64_t)top_ordered(v) << 32 | (uint32_t)~index;
}
__device__ __forceinline__ bool top_finite(float v) { return v > -INFINITY; }  // not NaN either

// One warp's sorted list: lane i holds the (i+1)-th largest key it was given.
struct TopList {
    uint64_t key = 0;
    // the keys of the lanes that offer one
    __device__ __forceinline__ void offer(bool on, uint64_t mine, int k, int lane) {
        uint64_t least = __shfl_sync(0xffffffffu, key, k - 1);
        uint32_t who = __ballot_sync(0xffffffffu, on && mine > least);
        while (who) {
            const int src = __ffs(who) - 1;
            const uint64_t v = __shfl_sync(0xffffffffu, mine, src);
            const uint32_t above = __ballot_sync(0xffffffffu, key > v);  // a prefix of the lanes
            const uint64_t up = __shfl_up_sync(0xffffffffu, key, 1);
            const int at = __popc(above);
            key = lane < at ? key : lane == at ? v : up;
            least = __shfl_sync(0xffffffffu, key, k - 1);
            who &= who - 1;
            who &= __ballot_sync(0xffffffffu, mine > least);
        }
    }
};

// Candidates in shared memory, in no order: one key is one logit, so the places
// that their ranks give them do not depend on it.
constexpr int kTopCand = 256;
__device__ __forceinline__ void top_add(bool on, uint64_t key, uint64_t *cand, int *n) {
    if (on) {
        const int at = atomicAdd(n, 1);
        if (at < kTopCand) cand[at] = key;
    }
}
__device__ __forceinline__ int top_rank(const uint64_t *cand, int n, uint64_t v) {
    int place = 0, i = 0;
    for (; i + 4 <= n; i += 4) {
        const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(cand + i), q = *reinterpret_cast<const ulonglong2 *>(cand + i + 2);
        place += (p.x > v) + (p.y > v) + (q.x > v) + (q.y > v);
    }
    for (; i < n; ++i) place += cand[i] > v;
    return place;
}
// By `threads` threads, of which this is t: `put` takes the first k places, 0 where
// there is none.
template <typename F>
__device__ __forceinline__ void top_ranks(const uint64_t *cand, int n, int k, int t, int threads, F put) {
    for (int i = t; i < n; i += threads) {
        const uint64_t v = cand[i];
        const int place = top_rank(cand, n, v);
        if (place < k) put(place, v);
    }
    if (t >= n && t < k) put(t, 0);
}

// (maximum, sum, A) of a set of logits.
struct RowEnt {
    float m, d, a;
};
// The same around another maximum M >= m.
__device__ __forceinline__ void ent_to(RowEnt &r, float M, float c) {
    if (M > r.m) {
        if (r.m > -INFINITY) {
            const float x = fmaxf((r.m - M) * c, -300.f), f = exp2_fast(x);
            r.a = f * fmaf(r.d, x, r.a);
            r.d *= f;
        }
        r.m = M;
    }
}
// A term 2^x x is 0 from 2^-126 on; -inf times 0 is not.
__device__ __forceinline__ float ent_x(float x) { return fmaxf(x, -200.f); }

// Add a set of packs to (d, A) around m (packs_sum with the second sum).  CLAMP:
// logits of -inf may be among them.
template <typename T, int PK, bool CLAMP>
__device__ __forceinline__ void packs_ent_any(const uint4 (&raw)[PK], RowEnt &r, float c) {
    constexpr int H = IO2<T>::H;
    const Shift s(r.m, c);
    float2 d = f2(0.f), a = f2(0.f);
    if (!s.direct) {
#pragma unroll
        for (int k = 0; k < PK; ++k) {
            float2 v[H];
            IO2<T>::unpack(raw[k], v);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float2 x = __ffma2_rn(v[h], f2(c), f2(-s.b));
                const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                d = __fadd2_rn(d, e);
                if (CLAMP) x = make_float2(ent_x(x.x), ent_x(x.y));
                a = __ffma2_rn(e, x, a);
            }
        }
        const float sum = d.x + d.y;
        // what the rounding of b leaves of every x
        const float rest = r.m == -INFINITY ? 0.f : -fmaf(r.m, c, -s.b);
        r.a += s.left * fmaf(sum, rest, a.x + a.y);
        r.d += s.left * sum;
        return;
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
        for (int h = 0; h < H; ++h) {
            const float2 x = make_float2((v[h].x - r.m) * c, (v[h].y - r.m) * c);
            const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
            d = __fadd2_rn(d, e);
            a = __ffma2_rn(e, make_float2(ent_x(x.x), ent_x(x.y)), a);
        }
    }
    r.a += a.x + a.y;
    r.d += d.x + d.y;
}
// The clamp is one instruction a logit of seven: left out until a thread finds its
// A without a value, which -inf leaves (0 times -inf); then the packs at hand are
// taken again.
template <typename T, int PK>
__device__ __forceinline__ void packs_ent(const uint4 (&raw)[PK], RowEnt &r, float c, bool &clamp) {
    const RowEnt before = r;
    if (!clamp) {
        packs_ent_any<T, PK, false>(raw, r, c);
        clamp = __any_sync(0xffffffffu, r.a != r.a);
        if (!clamp) return;
        r = before;
    }
    packs_ent_any<T, PK, true>(raw, r, c);
}
__device__ __forceinline__ void one_ent(float z, RowEnt &r, float c) {
    if (z > r.m) ent_to(r, z, c);
    const float x = (z - (r.m == -INFINITY ? 0.f : r.m)) * c, e = exp2_fast(x);
    r.d += e;
    r.a = fmaf(e, ent_x(x), r.a);
}
// Over a warp's lanes: every lane gets the same bits.
__device__ __forceinline__ RowEnt lanes_ent(RowEnt r, float c) {
    float M = r.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    ent_to(r, M, c);
    return RowEnt{M, warp_sum_all(r.d), warp_sum_all(r.a)};
}

// The outputs of a row that has a distribution, or has not (`empty`).
__device__ __forceinline__ void top_row(const TopArgs &t, int64_t row, const RowEnt &r, float za) {
    const bool empty = r.m == -INFINITY && r.d == 0.f;
    const float logd = empty ? -INFINITY : -log_prob(r.m, r.m, r.d, t.a.scale).hi;
    if (t.a.logp) t.a.logp[row] = empty ? -INFINITY : log_prob(za, r.m, r.d, t.a.scale).hi;
    if (t.entropy) t.entropy[row] = empty ? 0.f : fmaf(-0.693147181f, r.a / r.d, logd);
    if (t.a.stats) {
        t.a.stats[2 * row] = r.m;
        t.a.stats[2 * row + 1] = logd;
    }
}
// By one thread or by lanes of a warp: a row that takes no part.
__device__ __forceinline__ void top_no_row(const TopArgs &t, int64_t row) {
    if (t.a.logp) t.a.logp[row] = 0.f;
    if (t.entropy) t.entropy[row] = 0.f;
    if (t.a.stats) t.a.stats[2 * row] = t.a.stats[2 * row + 1] = 0.f;
    for (int i = 0; i < t.k; ++i) {
        t.ids[row * t.k + i] = -1;
        t.top[row * t.k + i] = 0.f;
    }
}
__device__ __forceinline__ void top_place(const TopArgs &t, int64_t row, int place, uint64_t key, const RowEnt &r) {
    t.ids[row * t.k + place] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
    t.top[row * t.k + place] = key ? log_prob(top_value((uint32_t)(key >> 32)), r.m, r.d, t.a.scale).hi : -INFINITY;
}

// ---------------------------------------------------------------------------
// Rows of up to 32 PK packs: one warp a row, the row in its registers.
// ---------------------------------------------------------------------------
template <typename T, int PK, int MINB>
__global__ void __launch_bounds__(128, MINB) logit_top_warp_kernel(const TopArgs ta) {
    constexpr int V = IO<T>::V;
    __shared__ __align__(16) uint64_t cand[4][kTopCand];
    __shared__ int count[4];
    const LogitArgs &a = ta.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = ta.k;
    pdl_wait();
    pdl_launch_dependents();
    const float c = a.scale * kLog2e;
    for (int64_t row = (int64_t)blockIdx.x * 4 + warp; row < a.rows; row += (int64_t)gridDim.x * 4) {
        const int64_t tgt = a.target[row];
        if (tgt < 0 || tgt >= a.V) {
            if (lane == 0) top_no_row(ta, row);
            continue;
        }
        const RowView<T> w(a, row, 0, 0, lane);
        const float za = IO<T>::to_f(w.z[tgt]);
        const bool has = lane < w.ns;
        const float zs = has ? IO<T>::to_f(w.z[w.sc]) : -INFINITY;
        uint4 raw[PK];
#pragma unroll
        for (int p = 0; p < PK; ++p) {
            raw[p] = no_pack<T>();
            if (p * 32 < w.mine) raw[p] = ld_once(w.body + p * 32 * V);
        }
        RowEnt r{packs_max<PK>(raw, T()), 0.f, 0.f};
        bool clamp = false;
        packs_ent<T, PK>(raw, r, c, clamp);
        float tm = r.m;
        if (has) {
            one_ent(zs, r, c);
            tm = fmaxf(tm, zs);
        }
        r = lanes_ent(r, c);
        if (lane == 0) top_row(ta, row, r, za);
        if (k == 0) continue;
        // T: the k-th largest of the lanes' maxima, to 16 bits downwards
        const uint32_t om = top_ordered(tm) >> 16;
        uint32_t T16 = 0;
#pragma unroll
        for (int b = 15; b >= 0; --b) {
            const uint32_t t = T16 | 1u << b;
            if (__popc(__ballot_sync(0xffffffffu, om >= t)) >= k) T16 = t;
        }
        const uint32_t T32 = T16 << 16 > kTopNone ? T16 << 16 : kTopNone + 1u;
        // (a prefix below that of the lowest finite value stands for it: compared as
        // values, NaN and -inf fail)
        const float low = fmaxf(top_value(T32), -3.4028235e38f);
        if (lane == 0) count[warp] = 0;
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PK; ++p) {
            float f[V];
            IO<T>::unpack(raw[p], f);
            float pm = f[0];
#pragma unroll
            for (int i = 1; i < V; ++i) pm = fmaxf(pm, f[i]);
            if (!(pm >= low)) continue;
            const uint32_t at = (uint32_t)(w.head + (lane + p * 32) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) top_add(f[i] >= low, top_key(f[i], at + i), cand[warp], &count[warp]);
        }
        top_add(has && zs >= low, top_key(zs, (uint32_t)w.sc), cand[warp], &count[warp]);
        __syncwarp();
        const int n = count[warp];
        if (n <= kTopCand) {
            top_ranks(cand[warp], n, k, lane, 32, [&](int place, uint64_t key) { top_place(ta, row, place, key, r); });
            __syncwarp();
            continue;
        }
        // many more than k (ties): a sorted list of the largest so far
        TopList list;
#pragma unroll 1
        for (int p = 0; p < PK; ++p) {
            uint4 q = raw[0];
#pragma unroll
            for (int j = 1; j < PK; ++j)
                if (j == p) q = raw[j];
            float f[V];
            IO<T>::unpack(q, f);
            const uint32_t at = (uint32_t)(w.head + (lane + p * 32) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) list.offer(f[i] >= low, top_key(f[i], at + i), k, lane);
        }
        list.offer(has && zs >= low, top_key(zs, (uint32_t)w.sc), k, lane);
        if (lane < k) top_place(ta, row, lane, list.key, r);
    }
}

// ---------------------------------------------------------------------------
// Any row: a CTA, or the CTAs of a cluster with a slice of the packs each, goes
// over it in segments of TH x PK packs, the next segment on its way into shared
// memory meanwhile.  4096 x 131072 bf16, a quarter of the rows out: without
// alternatives 126 us, 94 % of the measured copy rate; with 20 150 us.  A row's
// selection (three barriers, the found groups' way from L2) is a CTA's own time,
// which the other three CTAs of its SM stream through.
// ---------------------------------------------------------------------------
constexpr int kTopGroups = 8;  // a thread's groups: their maxima wait in shared memory

template <typename T> struct TopSlice {
    const T *z, *body;
    int head, tail, p0, mine, packs, ns;
    int64_t sc;
    __device__ __forceinline__ TopSlice(const LogitArgs &a, int64_t row, int rank, int cs, int t) {
        z = static_cast<const T *>(a.z) + row * a.ldz;
        const RowCut<T> cut = cut_row(z, a.V);
        head = cut.head;
        tail = cut.tail;
        p0 = (int)((int64_t)cut.packs * rank / cs);
        packs = (int)((int64_t)cut.packs * (rank + 1) / cs) - p0;
        body = z + head + (int64_t)p0 * IO<T>::V;
        mine = packs - t;
        ns = rank == 0 ? head + tail : 0;
        sc = t < head ? t : a.V - tail + (t - head);
    }
};

// What the CTA's warps share.  The arrays of two alternate between rows.
template <int NW> struct TopShared {
    RowEnt slot[2][NW];
    __align__(16) uint32_t tops[2][32];     // each warp's 32 / NW largest
    __align__(16) uint64_t cand[kTopCand];  // room for every warp's list
    float target[2], ends[2][16];           // the target's logit; the row's scalar elements
    uint64_t pub_keys[2][32];
    RowEnt pub[2];
    int groups_found[2], cands[2], per_group[kTopGroups];
};

// A found group's elements, PASS a lane (a group's packs are TH apart), four groups
// in flight: `use` gets each value and its column.
template <typename T, int TH, int PK, typename F>
__device__ __forceinline__ void top_scan(const TopSlice<T> &w, const unsigned short *found, int n, int per, F use) {
    constexpr int NW = TH / 32, V = IO<T>::V, PASS = PK * V / 32;
    static_assert(PASS >= 1, "a group has an element for each lane");
    const int lane = threadIdx.x & 31;
    for (int i0 = threadIdx.x >> 5; i0 < n; i0 += 4 * NW) {
        for (int sub = 0; sub < per; ++sub) {
            float f[4][PASS];
            int idx[4][PASS];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * NW;
                const int code = i < n ? found[i] : 0, g = code / TH, th = code % TH;
#pragma unroll
                for (int q = 0; q < PASS; ++q) {
                    const int e = q * 32 + lane, pack = ((g * per + sub) * PK + e / V) * TH + th;
                    f[j][q] = -INFINITY;
                    idx[j][q] = (int)((uint32_t)w.head + (uint32_t)(w.p0 + pack) * V + e % V);
                    if (i < n && pack < w.packs) f[j][q] = IO<T>::to_f(w.z[idx[j][q]]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < PASS; ++q)
                    if (i0 + j * NW < n) use(f[j][q], (uint32_t)idx[j][q]);
        }
    }
}

template <typename T, int TH, int PK, int MINB>
__global__ void __launch_bounds__(TH, MINB) logit_top_kernel(const TopArgs ta, const int cs, const int batch) {
    constexpr int V = IO<T>::V;
    constexpr int NW = TH / 32, TOPS = 32 / NW;
    static_assert(kTopCand >= 32 * NW, "room for every warp's list");
    constexpr uint32_t ALL = 0xffffffffu;
    extern __shared__ __align__(16) uint4 next_row[];                                     // [PK][TH]
    float *const group_max = reinterpret_cast<float *>(next_row + PK * TH);               // [kTopGroups][TH]
    unsigned short *const found = reinterpret_cast<unsigned short *>(group_max + kTopGroups * TH);  // [kTopGroups * TH]
    __shared__ TopShared<NW> sh;
    const LogitArgs &a = ta.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, k = ta.k;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    pdl_wait();
    pdl_launch_dependents();
    const float c = a.scale * kLog2e;
    int parity = 1;
    bool clamp = false;
    if (t == 0) sh.groups_found[0] = sh.cands[0] = 0;  // the first row's barrier is ahead of their first use
    const int64_t first = (int64_t)(blockIdx.x / cs) * batch, step = (int64_t)(gridDim.x / cs) * batch;
    for (int64_t r0 = first; r0 < a.rows; r0 += step) {
        const bool have = lane < batch && r0 + lane < a.rows;
        const int64_t my_target = have ? a.target[r0 + lane] : -1;
        const bool takes_part = my_target >= 0 && my_target < a.V;
        uint32_t live = __ballot_sync(ALL, takes_part);
        if (rank == 0 && t < 32 && have && !takes_part) top_no_row(ta, r0 + lane);
        float zn = 0.f;  // the next row's scalar element
        auto fetch = [&](int64_t row, int seg) {
            const TopSlice<T> w(a, row, rank, cs, t);
            if (seg == 0 && t < w.ns) zn = IO<T>::to_f(w.z[w.sc]);
#pragma unroll
            for (int p = 0; p < PK; ++p) {
                const int at = (seg * PK + p) * TH;
                cp_async16_if(at < w.mine, &next_row[p * TH + t], w.body + (int64_t)(at + t) * V);
            }
        };
        if (live) fetch(r0 + __ffs(live) - 1, 0);
        while (live) {
            const int at = __ffs(live) - 1;
            const int64_t row = r0 + at, tgt = __shfl_sync(ALL, my_target, at);
            live &= live - 1;
            parity ^= 1;
            const TopSlice<T> w(a, row, rank, cs, t);
            if (t < w.ns) sh.ends[parity][t] = zn;
            if (t == 0) sh.target[parity] = IO<T>::to_f(w.z[tgt]);
            const int segs = w.packs > 0 ? (w.packs - 1) / (TH * PK) + 1 : 1;
            int log_per = 0;  // segments of a group: 2^log_per
            while ((segs - 1) >> log_per >= kTopGroups) ++log_per;
            RowEnt r{-INFINITY, 0.f, 0.f};
            for (int seg = 0; seg < segs; ++seg) {
                cp_async_wait();
                uint4 raw[PK];
#pragma unroll
                for (int p = 0; p < PK; ++p) {
                    raw[p] = no_pack<T>();
                    if ((seg * PK + p) * TH < w.mine) raw[p] = next_row[p * TH + t];
                }
                float m = packs_max<PK>(raw, T());
                // the maximum is there, so the packs have left shared memory
                asm volatile("" : "+f"(m)::"memory");
                if (seg + 1 < segs)
                    fetch(row, seg + 1);
                else if (live)
                    fetch(r0 + __ffs(live) - 1, 0);
                float &gm = group_max[(seg >> log_per) * TH + t];
                gm = seg & ((1 << log_per) - 1) ? fmaxf(gm, m) : m;
                ent_to(r, m, c);
                packs_ent<T, PK>(raw, r, c, clamp);
            }
            const int group = ((segs - 1) >> log_per) + 1, per = 1 << log_per;
            float tm = -INFINITY;
            if (k > 0)
                for (int g = 0; g < group; ++g) tm = fmaxf(tm, group_max[g * TH + t]);
            if (t < w.ns) {
                const float zs = sh.ends[parity][t];
                one_ent(zs, r, c);
                tm = fmaxf(tm, zs);
            }
            r = lanes_ent(r, c);
            if (lane == 0) sh.slot[parity][warp] = r;
            if (k > 0) {
                uint32_t v = top_ordered(tm);
#pragma unroll
                for (int i = 0; i < TOPS; ++i) {
                    const uint32_t m = __reduce_max_sync(ALL, v);
                    if (lane == i) sh.tops[parity][warp * TOPS + i] = m;
                    if (lane == __ffs(__ballot_sync(ALL, v == m)) - 1) v = 0u;
                }
            }
            __syncthreads();
            if (k > 0) {
                // T: the k-th of those 32, maxima of as many threads.  (The k-th of their
                // different values is one redux.max each, but 16-bit logits have many
                // equal ones: 4096 x 131072 bf16 with 20 alternatives 169 us.)
                uint32_t T32;
                {
                    const uint32_t v = sh.tops[parity][lane];
                    int place = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 o = reinterpret_cast<const uint4 *>(sh.tops[parity])[i];
                        place += (o.x > v || (o.x == v && 4 * i < lane)) + (o.y > v || (o.y == v && 4 * i + 1 < lane)) +
                                 (o.z > v || (o.z == v && 4 * i + 2 < lane)) + (o.w > v || (o.w == v && 4 * i + 3 < lane));
                    }
                    T32 = __shfl_sync(ALL, v, __ffs(__ballot_sync(ALL, place == k - 1)) - 1);
                    if (T32 <= kTopNone) T32 = kTopNone + 1u;
                }
                for (int g = 0; g < group; ++g)
                    if (top_ordered(group_max[g * TH + t]) >= T32)
                        found[atomicAdd(&sh.groups_found[parity], 1)] = (unsigned short)(g * TH + t);
                __syncthreads();
                int n = sh.groups_found[parity], cut = group;
                if (n > kTopCand) {
                    // Many more than k (ties): groups up to `cut` hold k candidates, and later
                    // ones count only with a larger maximum.
                    __syncthreads();
                    if (t < kTopGroups) sh.per_group[t] = 0;
                    if (t == 0) sh.groups_found[parity] = 0;
                    __syncthreads();
                    for (int g = 0; g < group; ++g) {
                        const uint32_t who = __ballot_sync(ALL, top_ordered(group_max[g * TH + t]) >= T32);
                        if (who && lane == 0) atomicAdd(&sh.per_group[g], __popc(who));
                    }
                    __syncthreads();
                    int sum = 0;
                    for (int g = 0; g < group && sum < k; ++g) {
                        sum += sh.per_group[g];
                        cut = g + 1;
                    }
                    for (int g = 0; g < cut; ++g)
                        if (top_ordered(group_max[g * TH + t]) >= T32)
                            found[atomicAdd(&sh.groups_found[parity], 1)] = (unsigned short)(g * TH + t);
                    __syncthreads();
                    n = sh.groups_found[parity];
                }
                TopList list;
                while (true) {
                    top_scan<T, TH, PK>(w, found, n, per, [&](float f, uint32_t at) {
                        list.offer(top_finite(f) && top_ordered(f) >= T32, top_key(f, at), k, lane);
                    });
                    // the row's ends at last: the tail's columns are above all groups', so it
                    // may not raise the bound for them
                    if (warp == 0 && cut == group) {
                        const float zs = t < w.ns ? sh.ends[parity][t] : -INFINITY;
                        list.offer(top_finite(zs), top_key(zs, (uint32_t)w.sc), k, lane);
                    }
                    // the warps' lists, one behind the other
                    const uint32_t held = __ballot_sync(ALL, list.key != 0);
                    int base = 0;
                    if (lane == 0 && held) base = atomicAdd(&sh.cands[parity], __popc(held));
                    base = __shfl_sync(ALL, base, 0);
                    if (list.key) sh.cand[base + lane] = list.key;
                    if (t == 0) sh.groups_found[parity ^ 1] = sh.cands[parity ^ 1] = 0;  // the next row's
                    __syncthreads();
                    if (cut == group) break;
                    // the rest, from the k-th key on
                    const int nc = sh.cands[parity];
                    if (t < nc && top_rank(sh.cand, nc, sh.cand[t]) == k - 1) sh.pub_keys[parity][k - 1] = sh.cand[t];
                    __syncthreads();
                    const uint32_t kth = (uint32_t)(sh.pub_keys[parity][k - 1] >> 32);
                    if (t == 0) sh.groups_found[parity] = sh.cands[parity] = 0;
                    __syncthreads();
                    for (; cut < group; ++cut)
                        if (top_ordered(group_max[cut * TH + t]) > kth)
                            found[atomicAdd(&sh.groups_found[parity], 1)] = (unsigned short)(cut * TH + t);
                    __syncthreads();
                    n = sh.groups_found[parity];
                }
            }
            // The row's outputs, by the threads that find a candidate.  (For one warp
            // alone, while the others go on, the compiler spilled 53 registers a row.)
            // A warp without one goes on to the next row, whose first barrier is ahead
            // of what it would overwrite.
            {
                r = lanes_ent(lane < NW ? sh.slot[parity][lane] : RowEnt{-INFINITY, 0.f, 0.f}, c);
                const int nc = k > 0 ? sh.cands[parity] : 0;
                if (cs == 1) {
                    if (t == 0) top_row(ta, row, r, sh.target[parity]);
                    top_ranks(sh.cand, nc, k, t, TH, [&](int place, uint64_t key) { top_place(ta, row, place, key, r); });
                } else {
                    if (t == 0) sh.pub[parity] = r;
                    top_ranks(sh.cand, nc, k, t, TH, [&](int place, uint64_t key) { sh.pub_keys[parity][place] = key; });
                }
            }
            if (cs > 1) {
                __syncwarp();
                cluster_arrive();
                cluster_wait();
                if (rank == 0) {
                    // every CTA's sums and list
                    if (t == 0) sh.cands[parity] = 0;
                    __syncthreads();
                    uint64_t v = 0;
                    if (warp < cs && lane < k) {
                        const float2 u = ld_dsmem(reinterpret_cast<const float2 *>(&sh.pub_keys[parity][lane]), (uint32_t)warp);
                        v = (uint64_t)__float_as_uint(u.y) << 32 | __float_as_uint(u.x);
                    }
                    if (v) sh.cand[atomicAdd(&sh.cands[parity], 1)] = v;
                    r = RowEnt{-INFINITY, 0.f, 0.f};
                    if (lane < cs) {
                        r.m = ld_dsmem(&sh.pub[parity].m, (uint32_t)lane);
                        r.d = ld_dsmem(&sh.pub[parity].d, (uint32_t)lane);
                        r.a = ld_dsmem(&sh.pub[parity].a, (uint32_t)lane);
                    }
                    r = lanes_ent(r, c);
                    if (t == 0) top_row(ta, row, r, sh.target[parity]);
                    __syncthreads();
                    top_ranks(sh.cand, sh.cands[parity], k, t, TH, [&](int place, uint64_t key) { top_place(ta, row, place, key, r); });
                }
            }
        }
    }
    if (cs > 1) {
        // stay resident until the first rank has read this CTA's list
        cluster_arrive();
        cluster_wait();
    }
}

// ---------------------------------------------------------------------------
// The gradient: element-wise from the forward's statistics, tiles of 4 x TH
// packs of a row.  The entries of the target and the alternatives are written
// once more, whole, each by the thread that wrote its pack just now, from the
// logit that it still has in its registers (dlogits may replace the logits); every
// warp has the names, one a lane, and looks at those in its tile.  2048 x 131072
// bf16: 151 us, 92 % of the measured copy rate; with the names in shared memory and
// barriers around the tile's stores 161.
// ---------------------------------------------------------------------------
template <typename T> struct TopSlope {
    float s, top, logd, gsum, h, gh;  // gh: gsum + h H
    // -s p (gsum + h (lp + H)); p = 0 from lp = -88 on
    __device__ __forceinline__ float one(float z) const {
        const float lp = fmaf(z - top, s, -logd);
        return -s * exp2_fast(lp * kLog2e) * fmaf(h, fmaxf(lp, -100.f), gh);
    }
    __device__ __forceinline__ uint4 pack(const uint4 &raw) const {
        constexpr int H = IO2<T>::H;
        float2 v[H];
        IO2<T>::unpack(raw, v);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 lp = __ffma2_rn(__fadd2_rn(v[i], f2(-top)), f2(s), f2(-logd));
            float2 p = __fmul2_rn(lp, f2(kLog2e));
            p.x = exp2_fast(p.x);
            p.y = exp2_fast(p.y);
            const float2 q = __ffma2_rn(f2(h), make_float2(fmaxf(lp.x, -100.f), fmaxf(lp.y, -100.f)), f2(gh));
            v[i] = __fmul2_rn(__fmul2_rn(p, f2(-s)), q);
        }
        return IO2<T>::pack(v);
    }
};

// Value e of a thread's packs, e = pack * V + its place.
template <typename T, int U> __device__ __forceinline__ float pick(const uint4 (&raw)[U], int e) {
    constexpr int V = IO<T>::V, PER = V / 4;
    const int word = e / PER;
    uint32_t w = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (word == 4 * u) w = raw[u].x;
        if (word == 4 * u + 1) w = raw[u].y;
        if (word == 4 * u + 2) w = raw[u].z;
        if (word == 4 * u + 3) w = raw[u].w;
    }
    float f[V];
    IO<T>::unpack(make_uint4(w, w, w, w), f);
    return PER == 2 && e % 2 ? f[1] : f[0];
}

template <typename T, int TH>
__global__ void __launch_bounds__(256) logit_top_grad_kernel(const TopArgs ta, const int tiles) {
    constexpr int G = 256 / TH, V = IO<T>::V, U = 4;
    constexpr uint32_t ALL = 0xffffffffu;
    const LogitArgs &a = ta.a;
    const int t = threadIdx.x % TH, lane = threadIdx.x & 31, k = ta.k;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = a.rows * tiles;
    for (int64_t id = (int64_t)blockIdx.x * G + threadIdx.x / TH; id < total; id += (int64_t)gridDim.x * G) {
        const int64_t row = total <= 0xffffffffll ? (int64_t)((uint32_t)id / (uint32_t)tiles) : id / tiles;
        const int tile = (int)(id - row * tiles);
        const T *Z = static_cast<const T *>(a.z) + row * a.ldz;
        T *D = static_cast<T *>(a.dz) + row * a.lddz;
        const int64_t tgt = a.target[row];
        TopSlope<T> f;
        f.s = a.scale;
        f.top = a.stats_in[2 * row];
        f.logd = a.stats_in[2 * row + 1];
        const bool live = tgt >= 0 && tgt < a.V && f.logd != -INFINITY;
        const float g = live && a.dlogp ? a.dlogp[row] : 0.f;
        // the alternatives, one a lane (a column fits 32 bits); -1: none
        const int64_t named = live && lane < k && ta.dtop ? ta.ids_in[row * k + lane] : -1;
        const int name = named >= 0 && named < a.V ? (int)named : -1;
        const float al = name >= 0 ? ta.dtop[row * k + lane] : 0.f;
        f.h = live && ta.dentropy ? ta.dentropy[row] : 0.f;
        f.gsum = g + warp_sum_all(al);
        f.gh = f.h != 0.f ? fmaf(f.h, ta.entropy_in[row], f.gsum) : f.gsum;
        const bool any = __any_sync(ALL, al != 0.f) || g != 0.f || f.h != 0.f;
        const RowCut<T> cut = cut_row(Z, a.V);
        const T *body = Z + cut.head;
        T *out = D + cut.head;
        const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const int base = tile * (TH * U), p0 = base + t;
        const int ns = tile == 0 ? cut.head + cut.tail : 0;
        const int64_t sc = t < cut.head ? t : a.V - cut.tail + (t - cut.head);
        if (!any) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * TH < cut.packs) st_pack(out + (int64_t)(p0 + u * TH) * V, make_uint4(0, 0, 0, 0), wide);
            if (t < ns) D[sc] = IO<T>::from_f(0.f);
            continue;
        }
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p0 + u * TH < cut.packs) raw[u] = ld_once(body + (int64_t)(p0 + u * TH) * V);
        const float zs = t < ns ? IO<T>::to_f(Z[sc]) : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p0 + u * TH < cut.packs) st_pack(out + (int64_t)(p0 + u * TH) * V, f.pack(raw[u]), wide);
        if (t < ns) D[sc] = IO<T>::from_f(f.one(zs));
        // the columns of this tile that have a name: the target, and those of the
        // alternatives that are not the target
        const int c0 = cut.head + base * V, c1 = (int)min((int64_t)cut.head + (int64_t)(base + TH * U) * V, a.V - cut.tail);
        auto here = [&](int j) { return (j >= c0 && j < c1) || (tile == 0 && (j < cut.head || j >= a.V - cut.tail)); };
        auto write = [&](int j, float part) {
            if (j >= cut.head && j < a.V - cut.tail) {
                const int e = j - c0, p = e / V;  // of the tile
                if (p % TH == t) D[j] = IO<T>::from_f(fmaf(f.s, part, f.one(pick<T, U>(raw, p / TH * V + e % V))));
            } else if (t < ns && sc == j) {
                D[j] = IO<T>::from_f(fmaf(f.s, part, f.one(zs)));
            }
        };
        const int it = (int)tgt;
        if (here(it)) write(it, g + warp_sum_all(name == it ? al : 0.f));
        uint32_t left = __ballot_sync(ALL, name >= 0 && name != it && here(name));
        while (left) {
            const int j = __shfl_sync(ALL, name, __ffs(left) - 1);
            left &= ~__ballot_sync(ALL, name == j);
            write(j, warp_sum_all(name == j ? al : 0.f));
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (logits_<type>.cu).
// ---------------------------------------------------------------------------
template <typename T, int PK, int MINB> cudaError_t launch_top_warp(const TopArgs &a, cudaStream_t s, Plan *p) {
    p->kind = PLAN_WARP;
    p->threads = 128;
    p->packs = PK;
    const int64_t n = (a.a.rows + 3) / 4;
    return launch_row(logit_top_warp_kernel<T, PK, MINB>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff), 128u, 0, s, a);
}
template <typename T, int TH, int PK, int MINB>
cudaError_t launch_top_cta(const TopArgs &a, int cs, int sms, cudaStream_t s, Plan *p) {
    constexpr size_t smem = (size_t)PK * TH * 16 + (size_t)kTopGroups * TH * 6;
    auto kernel = logit_top_kernel<T, TH, PK, MINB>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), TH, smem, &per_sm);
    if (e != cudaSuccess) return e;
    p->kind = cs > 1 ? PLAN_CLUSTER : PLAN_CTA;
    p->threads = TH;
    p->packs = PK;
    p->groups = cs > 1 ? cs : 0;
    const int64_t batch = rows_per_batch(a.a.rows, (int64_t)sms * per_sm / cs, 1);
    return launch_clusters(kernel, (a.a.rows + batch - 1) / batch, cs, TH, smem, s, a, cs, (int)batch);
}

// Device times of bf16 with 20 alternatives, inputs beyond L2, all of them of this
// form of the kernels.  Rows of up to 512 packs by a warp, where rows are many: 8192 x
// 4000 45 us, by CTAs of 128 threads 92, of 256 137 (with 32 alternatives, whose lower
// bound is the least of the lanes' maxima, 103 and 122 by CTAs of 128); 8192 x 1000
// 17.5 and 91.  Then CTAs of 128 up to 4096 packs, for what a row costs beside its packs
// is paid by each warp: 4096 x 8000 47 us, by CTAs of 256 77; 4096 x 32000 88 and 93.
// Longer rows keep more in flight by 256: 4096 x 131072 149, by 128 173; the two meet
// above the border (4096 x 50257 136, by 128 124).  A row over two or more CTAs while
// they do not cover the SMs twice, so that a few long rows are not one SM's each: 200 x
// 32000 13.6 us by two and 22 by four, but 10.6 by one, so that this border, too, is
// not where the two meet; beyond it the second list a row costs more than it gives
// (f32 513 x 50001 26.5 us, by two CTAs 32).
template <typename T> cudaError_t launch_logit_top_t(const TopArgs &a, int sms, cudaStream_t s, Plan *p) {
    const int64_t packs = a.a.V / IO<T>::V;
    if (packs <= 32 * 4) return launch_top_warp<T, 4, 8>(a, s, p);
    if (packs <= 32 * 16 && a.a.rows >= 2 * (int64_t)sms)
        return packs <= 32 * 8 ? launch_top_warp<T, 8, 6>(a, s, p) : launch_top_warp<T, 16, 4>(a, s, p);
    int cs = 1;
    while (cs < 8 && a.a.rows * cs < 2 * (int64_t)sms && packs >= 2 * cs * 256) cs *= 2;
    if (cs == 1 && packs <= 4096) return launch_top_cta<T, 128, 8, 8>(a, 1, sms, s, p);
    return launch_top_cta<T, 256, 8, 4>(a, cs, sms, s, p);
}

template <typename T, int TH> cudaError_t launch_top_grad_g(const TopArgs &a, cudaStream_t s) {
    constexpr int G = 256 / TH;
    const int64_t packs = a.a.V / IO<T>::V + 1;
    const int64_t tiles = (packs + 4 * TH - 1) / (4 * TH);
    const int64_t n = (a.a.rows * tiles + G - 1) / G;
    return launch_row(logit_top_grad_kernel<T, TH>, (unsigned)(n < 0x7fffffff ? n : 0x7fffffff), 256u, 0, s, a, (int)tiles);
}
template <typename T> cudaError_t launch_logit_top_grad_t(const TopArgs &a, cudaStream_t s) {
    return a.a.V / IO<T>::V <= 512 ? launch_top_grad_g<T, 32>(a, s) : launch_top_grad_g<T, 256>(a, s);
}

}  // namespace nrm
