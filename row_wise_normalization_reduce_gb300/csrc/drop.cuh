// drop.cuh -- dropout from a counter-based generator, and the residual path
// built on it:
//
//   dropout            y = d(x)
//   dropout+add+RMS    h = residual + d(x) (rounded),  y = h * rstd * w
//   its backward       dresidual = dh,  dx = d(dh),  dw = sum_rows dy * h * rstd
//
// with d(v) = v * scale where the mask keeps the element and +0 elsewhere.
//
// Generator: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011).  Key = the 64-bit seed, counter =
// (column / 8, row, offset lo, offset hi).  The four output words are eight
// 16-bit numbers, low half first, one per column of the block; an element is
// kept when its number is at least T = round(65536 p).  16 bits per element
// (p to 2^-17) cost one generator call per 16 bytes of a 16-bit row: about
// 40 integer instructions per 8 elements, which stays under the time HBM
// needs for them; 32 bits per element would double that.  The mask depends on
// (seed, offset, row, column) alone -- not on types, strides or launch shapes
// -- so the backward makes it again instead of reading it.
//
// Work is cut into chunks of 256 columns, one warp each; lane l always
// computes generator block l of the chunk (columns 8 l .. 8 l + 7) and holds 8
// of the chunk's elements, placed so that its global accesses coalesce:
//   MAP_V8  16-bit types, 16-byte aligned rows: columns 8 l + j, one 16-byte access
//   MAP_V4  binary32, 16-byte aligned rows: columns 4 l + j and 128 + 4 l + j
//   MAP_S   any N and alignment: columns 32 j + l, eight scalar accesses
// For the last two the keep bits of a chunk travel by warp shuffles.
#pragma once

#include <cstdint>

#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

enum Map { MAP_V8 = 0, MAP_V4 = 1, MAP_S = 2 };
template <typename T> constexpr int vec_map() { return sizeof(T) == 2 ? MAP_V8 : MAP_V4; }
constexpr int kChunk = 256;

// The offset words of this call: the host's plus the device counter's value.
struct DropCtr {
    uint32_t lo, hi;
};
__device__ __forceinline__ DropCtr drop_ctr(const DropArgs &d) {
    uint64_t o = d.offset;
    if (d.offset_dev) o += (uint64_t)*d.offset_dev;
    return DropCtr{(uint32_t)o, (uint32_t)(o >> 32)};
}

// One generator block.
__device__ __forceinline__ uint4 drop_block(const DropArgs &d, const DropCtr &o, uint32_t block,
                                            uint32_t row) {
    uint32_t a = block, b = row, c = o.lo, e = o.hi;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ d.key[2 * r];
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ e ^ d.key[2 * r + 1];
        e = (uint32_t)p;
    }
    return make_uint4(a, b, c, e);
}

// Which of a lane's 8 elements are kept.  MAP_V8 keeps the block's words (the
// lane's elements are its own block); the others hold 8 bits gathered from
// the lanes that computed them.
template <int MAP> struct Keep {
    uint32_t bits;
    __device__ __forceinline__ bool operator()(int j, uint32_t) const { return (bits >> j) & 1u; }
};
template <> struct Keep<MAP_V8> {
    uint32_t w[4];
    __device__ __forceinline__ bool operator()(int j, uint32_t bar) const {
        return (j & 1 ? w[j >> 1] : w[j >> 1] << 16) > bar;
    }
};

// The keep set of chunk `chunk` of `row` (the whole warp calls it).
template <int MAP>
__device__ __forceinline__ Keep<MAP> drop_keep(const DropArgs &d, const DropCtr &o, int64_t chunk,
                                               int64_t row) {
    const int lane = threadIdx.x & 31;
    const uint4 w = drop_block(d, o, (uint32_t)(chunk * 32) + lane, (uint32_t)row);
    Keep<MAP> k;
    if constexpr (MAP == MAP_V8) {
        k.w[0] = w.x; k.w[1] = w.y; k.w[2] = w.z; k.w[3] = w.w;
    } else {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            mine |= (uint32_t)((j & 1 ? v[j >> 1] : v[j >> 1] << 16) > d.bar) << j;
        if constexpr (MAP == MAP_V4) {
            // pack p of the chunk is half (p & 1) of block p / 2
            const int sh = (lane & 1) * 4;
            const uint32_t lo = __shfl_sync(0xffffffffu, mine, lane >> 1) >> sh;
            const uint32_t hi = __shfl_sync(0xffffffffu, mine, 16 + (lane >> 1)) >> sh;
            k.bits = (lo & 15u) | (hi & 15u) << 4;
        } else {
            uint32_t b = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                b |= (__shfl_sync(0xffffffffu, mine, 4 * j + (lane >> 3)) >> (lane & 7) & 1u) << j;
            k.bits = b;
        }
    }
    return k;
}

// A lane's 8 elements of one chunk, in the storage type.
template <typename T> struct Frag {
    uint32_t r[2 * sizeof(T)];
};

// Streaming 16-byte load that stays coherent (an output may be the input).
__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Column of element j of this lane in a chunk.
template <int MAP> __device__ __forceinline__ int frag_col(int j) {
    const int lane = threadIdx.x & 31;
    return MAP == MAP_V8 ? 8 * lane + j : MAP == MAP_V4 ? 4 * lane + (j & 3) + 32 * (j & 4) : 32 * j + lane;
}

// p: the chunk's first element; left: columns from there to the row's end
// (any value; lanes past it hold zeros and store nothing).
template <typename T, int MAP, bool KEEP_CACHED = false>
__device__ __forceinline__ void frag_load(Frag<T> &f, const T *p, int64_t left) {
    const int lane = threadIdx.x & 31;
    if constexpr (MAP == MAP_V8) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (8 * lane < left) v = KEEP_CACHED ? ld_param(p + 8 * lane) : ld_once(p + 8 * lane);
        f.r[0] = v.x; f.r[1] = v.y; f.r[2] = v.z; f.r[3] = v.w;
    } else if constexpr (MAP == MAP_V4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 v = make_uint4(0, 0, 0, 0);
            const int c = 128 * h + 4 * lane;
            if (c < left) v = KEEP_CACHED ? ld_param(p + c) : ld_once(p + c);
            f.r[4 * h] = v.x; f.r[4 * h + 1] = v.y; f.r[4 * h + 2] = v.z; f.r[4 * h + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 2) {
        const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
        unsigned short e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = 32 * j + lane < left ? q[32 * j + lane] : (unsigned short)0;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.r[j] = (uint32_t)e[2 * j] | (uint32_t)e[2 * j + 1] << 16;
    } else {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) f.r[j] = 32 * j + lane < left ? q[32 * j + lane] : 0u;
    }
}

template <typename T, int MAP>
__device__ __forceinline__ void frag_store(const Frag<T> &f, T *p, int64_t left) {
    const int lane = threadIdx.x & 31;
    if constexpr (MAP == MAP_V8) {
        if (8 * lane < left) st_stream(p + 8 * lane, make_uint4(f.r[0], f.r[1], f.r[2], f.r[3]));
    } else if constexpr (MAP == MAP_V4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 128 * h + 4 * lane;
            if (c < left)
                st_stream(p + c, make_uint4(f.r[4 * h], f.r[4 * h + 1], f.r[4 * h + 2], f.r[4 * h + 3]));
        }
    } else if constexpr (sizeof(T) == 2) {
        unsigned short *q = reinterpret_cast<unsigned short *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (32 * j + lane < left) q[32 * j + lane] = (unsigned short)(f.r[j >> 1] >> 16 * (j & 1));
    } else {
        uint32_t *q = reinterpret_cast<uint32_t *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (32 * j + lane < left) q[32 * j + lane] = f.r[j];
    }
}

// Elements (2 i, 2 i + 1) as binary32 pairs, and back with one rounding each.
template <typename T> __device__ __forceinline__ void frag_unpack(const Frag<T> &f, float2 v[4]) {
    IO2<T>::unpack(make_uint4(f.r[0], f.r[1], f.r[2], f.r[3]), v);
    if constexpr (sizeof(T) == 4) IO2<T>::unpack(make_uint4(f.r[4], f.r[5], f.r[6], f.r[7]), v + 2);
}
template <typename T> __device__ __forceinline__ Frag<T> frag_pack(const float2 v[4]) {
    Frag<T> f;
    const uint4 a = IO2<T>::pack(v);
    f.r[0] = a.x; f.r[1] = a.y; f.r[2] = a.z; f.r[3] = a.w;
    if constexpr (sizeof(T) == 4) {
        const uint4 b = IO2<T>::pack(v + 2);
        f.r[4] = b.x; f.r[5] = b.y; f.r[6] = b.z; f.r[7] = b.w;
    }
    return f;
}

// d(v) of 8 elements: the product rounded to binary32, or +0 (a select, so a
// dropped infinity or NaN leaves nothing behind).
template <int MAP>
__device__ __forceinline__ void drop_apply(const DropArgs &d, const Keep<MAP> &k, float2 v[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = __fmul2_rn(v[i], f2(d.scale));
        v[i].x = k(2 * i, d.bar) ? s.x : 0.f;
        v[i].y = k(2 * i + 1, d.bar) ? s.y : 0.f;
    }
}

// L2 prefetch of one row, its ends rounded inward to 16 bytes.
template <typename T> __device__ __forceinline__ void prefetch_row(const T *p, int64_t n) {
    const uintptr_t lo = (reinterpret_cast<uintptr_t>(p) + 15) & ~(uintptr_t)15;
    const uintptr_t hi = reinterpret_cast<uintptr_t>(p + n) & ~(uintptr_t)15;
    if (hi > lo) prefetch_l2_bulk(reinterpret_cast<const void *>(lo), (uint32_t)(hi - lo));
}

// ---------------------------------------------------------------------------
// Dropout alone: element-wise, bound by HBM (one read, one write).  Chunks of
// the whole tensor are numbered row by row; a warp takes U at a time, loads
// issued before the generator runs.
// ---------------------------------------------------------------------------
template <typename T, int MAP, int U>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs d, const T *x, const int64_t ldx,
                                                      T *y, const int64_t ldy, const int64_t rows,
                                                      const int64_t N, const int64_t cpr) {
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(d);
    const int64_t total = rows * cpr;
    const int64_t step = (int64_t)gridDim.x * 8 * U;
    for (int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * U; first < total; first += step) {
        Frag<T> f[U];
        int64_t row[U], c[U];
        row[0] = total <= 0xffffffffll ? (int64_t)((uint32_t)first / (uint32_t)cpr) : first / cpr;
        c[0] = first - row[0] * cpr;
#pragma unroll
        for (int u = 1; u < U; ++u) {
            const bool wrap = c[u - 1] + 1 == cpr;
            c[u] = wrap ? 0 : c[u - 1] + 1;
            row[u] = row[u - 1] + wrap;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row[u] < rows)
                frag_load<T, MAP>(f[u], x + row[u] * ldx + c[u] * kChunk, N - c[u] * kChunk);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < rows) {
                float2 v[4];
                frag_unpack<T>(f[u], v);
                if (d.on) drop_apply<MAP>(d, drop_keep<MAP>(d, o, c[u], row[u]), v);
                frag_store<T, MAP>(frag_pack<T>(v), y + row[u] * ldy + c[u] * kChunk, N - c[u] * kChunk);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Forward of the residual path, register plan: a group of GT threads per row
// (a warp, or the whole CTA), the row in registers, x and the residual read
// once.
// ---------------------------------------------------------------------------
template <typename T, int GT, int U, int MAP>
__global__ void __launch_bounds__(GT < 128 ? 128 : GT) drop_add_rms_kernel(const DropRmsArgs a,
                                                                          const int64_t pf) {
    constexpr int CTA = GT < 128 ? 128 : GT, NW = GT / 32, G = CTA / GT;
    __shared__ float slot[2][NW];
    const int warp = (threadIdx.x % GT) >> 5;
    const bool lead = threadIdx.x % GT == 0;
    const int N = (int)a.N;
    const T *X = static_cast<const T *>(a.x), *R = static_cast<const T *>(a.res);
    const T *W = static_cast<const T *>(a.w);
    T *H = static_cast<T *>(a.h), *Y = static_cast<T *>(a.y);
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(a.d);
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / GT; row < a.rows;
         row += (int64_t)gridDim.x * G, parity ^= 1) {
        if (pf > 0 && lead && row + pf < a.rows) {
            prefetch_row(X + (row + pf) * a.ldx, N);
            prefetch_row(R + (row + pf) * a.ldr, N);
        }
        Frag<T> fx[U], fr[U], fw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * NW + warp) * kChunk;
            frag_load<T, MAP>(fx[u], X + row * a.ldx + c, N - c);
            frag_load<T, MAP>(fr[u], R + row * a.ldr + c, N - c);
        }
        float2 acc = f2(0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = u * NW + warp, c = ch * kChunk;
            float2 v[4], r[4];
            Keep<MAP> k;
            if (a.d.on) k = drop_keep<MAP>(a.d, o, ch, row);
            frag_unpack<T>(fx[u], v);
            frag_unpack<T>(fr[u], r);
            if (a.d.on) drop_apply<MAP>(a.d, k, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r[i]);
            fr[u] = frag_pack<T>(v);  // the stream's value: the norm is of this rounding
            frag_store<T, MAP>(fr[u], H + row * a.ldh + c, N - c);
            frag_unpack<T>(fr[u], v);
            // columns past the row's end hold zeros and add nothing
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __ffma2_rn(v[i], v[i], acc);
            if (W) frag_load<T, MAP, true>(fw[u], W + c, N - c);
        }
        float ss = acc.x + acc.y;
        ss = GT == 32 ? warp_sum_all(ss) : cta_sum_all<NW>(ss, slot[parity]);
        const float rstd = rsqrtf(fmaf(ss, a.invN, a.eps));
        if (lead && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * NW + warp) * kChunk;
            float2 v[4], w[4];
            frag_unpack<T>(fr[u], v);
            if (W) frag_unpack<T>(fw[u], w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __fmul2_rn(v[i], f2(rstd));
                if (W) v[i] = __fmul2_rn(v[i], w[i]);
            }
            frag_store<T, MAP>(frag_pack<T>(v), Y + row * a.ldy + c, N - c);
        }
    }
}

// Rows longer than the register plan holds: the sum of squares while h is
// written, then h read again (each lane re-reads what it wrote) for y.
template <typename T, int MAP>
__global__ void __launch_bounds__(512) drop_add_rms_long_kernel(const DropRmsArgs a) {
    constexpr int NW = 16;
    __shared__ float slot[2][NW];
    const int warp = threadIdx.x >> 5;
    const T *X = static_cast<const T *>(a.x), *R = static_cast<const T *>(a.res);
    const T *W = static_cast<const T *>(a.w);
    T *H = static_cast<T *>(a.h), *Y = static_cast<T *>(a.y);
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(a.d);
    const int64_t chunks = (a.N + kChunk - 1) / kChunk;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        float2 acc = f2(0.f);
        for (int64_t ch = warp; ch < chunks; ch += NW) {
            const int64_t c = ch * kChunk;
            Frag<T> fx, fr;
            frag_load<T, MAP>(fx, X + row * a.ldx + c, a.N - c);
            frag_load<T, MAP>(fr, R + row * a.ldr + c, a.N - c);
            float2 v[4], r[4];
            frag_unpack<T>(fx, v);
            frag_unpack<T>(fr, r);
            if (a.d.on) drop_apply<MAP>(a.d, drop_keep<MAP>(a.d, o, ch, row), v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r[i]);
            fr = frag_pack<T>(v);
            frag_store<T, MAP>(fr, H + row * a.ldh + c, a.N - c);
            frag_unpack<T>(fr, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __ffma2_rn(v[i], v[i], acc);
        }
        const float ss = cta_sum_all<NW>(acc.x + acc.y, slot[parity]);
        const float rstd = rsqrtf(fmaf(ss, a.invN, a.eps));
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int64_t ch = warp; ch < chunks; ch += NW) {
            const int64_t c = ch * kChunk;
            Frag<T> fh, fw;
            float2 v[4], w[4];
            frag_load<T, MAP>(fh, H + row * a.ldh + c, a.N - c);
            if (W) frag_load<T, MAP, true>(fw, W + c, a.N - c);
            frag_unpack<T>(fh, v);
            if (W) frag_unpack<T>(fw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __fmul2_rn(v[i], f2(rstd));
                if (W) v[i] = __fmul2_rn(v[i], w[i]);
            }
            frag_store<T, MAP>(frag_pack<T>(v), Y + row * a.ldy + c, a.N - c);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  With k = -rstd^3 / N * sum_j dy_j w_j h_j (one row-wide sum):
//   dh = rstd * dy * w + k * h + dh_up
// ---------------------------------------------------------------------------
// The outputs of one lane's 8 elements of a row, and their share of dw.
template <typename T, int MAP>
__device__ __forceinline__ void drop_bwd_chunk(const DropRmsBwdArgs &a, const DropCtr &o, int64_t row,
                                               int64_t ch, const Frag<T> &fd, const Frag<T> &fh,
                                               const Frag<T> &fu, const Frag<T> &fw, float rstd,
                                               float k, float2 dw[4]) {
    const int64_t c = ch * kChunk;
    float2 dy[4], h[4], t[4];
    frag_unpack<T>(fd, dy);
    frag_unpack<T>(fh, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 e = __fmul2_rn(dy[i], f2(rstd));
        dw[i] = __ffma2_rn(e, h[i], dw[i]);
        dy[i] = e;
    }
    if (a.w) {
        frag_unpack<T>(fw, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) dy[i] = __fmul2_rn(dy[i], t[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) dy[i] = __ffma2_rn(h[i], f2(k), dy[i]);
    if (a.up) {
        frag_unpack<T>(fu, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) dy[i] = __fadd2_rn(dy[i], t[i]);
    }
    if (a.dres) frag_store<T, MAP>(frag_pack<T>(dy), static_cast<T *>(a.dres) + row * a.lddr + c, a.N - c);
    if (a.dx) {
        if (a.d.on) drop_apply<MAP>(a.d, drop_keep<MAP>(a.d, o, ch, row), dy);
        frag_store<T, MAP>(frag_pack<T>(dy), static_cast<T *>(a.dx) + row * a.lddx + c, a.N - c);
    }
}

// Register plan: persistent groups of GT threads, a row at a time; a thread's
// columns are the same in every row, so dw accumulates in registers and each
// CTA leaves one row of partial sums (folded in order by dw_fold_kernel: no
// atomics, the same bits every time).
template <typename T, int GT, int U, int MAP>
__global__ void __launch_bounds__(GT < 128 ? 128 : GT) drop_add_rms_bwd_kernel(const DropRmsBwdArgs a) {
    constexpr int CTA = GT < 128 ? 128 : GT, NW = GT / 32, G = CTA / GT;
    __shared__ float slot[2][NW];
    __shared__ float part[G > 1 ? G - 1 : 1][G > 1 ? U * kChunk : 1];
    const int warp = (threadIdx.x % GT) >> 5;
    const int N = (int)a.N;
    const T *DY = static_cast<const T *>(a.dy), *H = static_cast<const T *>(a.h);
    const T *UP = static_cast<const T *>(a.up), *W = static_cast<const T *>(a.w);
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(a.d);
    Frag<T> fw[U];
    float2 dw[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * NW + warp) * kChunk;
        if (W) frag_load<T, MAP, true>(fw[u], W + c, N - c);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[u][i] = f2(0.f);
    }
    const int64_t step = (int64_t)gridDim.x * G;
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / GT; row < a.rows; row += step, parity ^= 1) {
        if (threadIdx.x % GT == 0 && row + step < a.rows) {
            prefetch_row(DY + (row + step) * a.lddy, N);
            prefetch_row(H + (row + step) * a.ldh, N);
            if (UP) prefetch_row(UP + (row + step) * a.ldu, N);
        }
        Frag<T> fd[U], fh[U], fu[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * NW + warp) * kChunk;
            frag_load<T, MAP>(fd[u], DY + row * a.lddy + c, N - c);
            frag_load<T, MAP>(fh[u], H + row * a.ldh + c, N - c);
            if (UP) frag_load<T, MAP>(fu[u], UP + row * a.ldu + c, N - c);
        }
        const float rstd = a.rstd[row];
        float2 acc = f2(0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 dy[4], h[4], w[4];
            frag_unpack<T>(fd[u], dy);
            frag_unpack<T>(fh[u], h);
            if (W) frag_unpack<T>(fw[u], w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (W) dy[i] = __fmul2_rn(dy[i], w[i]);
                acc = __ffma2_rn(dy[i], h[i], acc);
            }
        }
        float dot = acc.x + acc.y;
        dot = GT == 32 ? warp_sum_all(dot) : cta_sum_all<NW>(dot, slot[parity]);
        // rstd^3 can leave binary32 where rstd * (rstd * dot) * rstd does not
        const float k = -(rstd * dot) * a.invN * rstd * rstd;
#pragma unroll
        for (int u = 0; u < U; ++u)
            drop_bwd_chunk<T, MAP>(a, o, row, u * NW + warp, fd[u], fh[u], fu[u], fw[u], rstd, k, dw[u]);
    }
    if (!a.dw) return;
    if constexpr (G > 1) {
        // the CTA's groups meet in shared memory, added in group order
        const int g = threadIdx.x / GT;
        if (g > 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    part[g - 1][u * kChunk + frag_col<MAP>(j)] = j & 1 ? dw[u][j >> 1].y : dw[u][j >> 1].x;
        }
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                for (int q = 0; q < G - 1; ++q) {
                    float &s = j & 1 ? dw[u][j >> 1].y : dw[u][j >> 1].x;
                    s += part[q][u * kChunk + frag_col<MAP>(j)];
                }
    }
    float *P = a.part + (int64_t)blockIdx.x * a.N;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (u * NW + warp) * kChunk + frag_col<MAP>(j);
            if (c < N) P[c] = j & 1 ? dw[u][j >> 1].y : dw[u][j >> 1].x;
        }
}

// Long rows: the row sums first (k per row into the workspace) ...
template <typename T, int MAP>
__global__ void __launch_bounds__(512) drop_bwd_dot_kernel(const DropRmsBwdArgs a) {
    constexpr int NW = 16;
    __shared__ float slot[2][NW];
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    const int64_t chunks = (a.N + kChunk - 1) / kChunk;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        float2 acc = f2(0.f);
        for (int64_t ch = warp; ch < chunks; ch += NW) {
            const int64_t c = ch * kChunk;
            Frag<T> fd, fh, fw;
            frag_load<T, MAP>(fd, static_cast<const T *>(a.dy) + row * a.lddy + c, a.N - c);
            frag_load<T, MAP>(fh, static_cast<const T *>(a.h) + row * a.ldh + c, a.N - c);
            if (a.w) frag_load<T, MAP, true>(fw, static_cast<const T *>(a.w) + c, a.N - c);
            float2 dy[4], h[4], w[4];
            frag_unpack<T>(fd, dy);
            frag_unpack<T>(fh, h);
            if (a.w) frag_unpack<T>(fw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (a.w) dy[i] = __fmul2_rn(dy[i], w[i]);
                acc = __ffma2_rn(dy[i], h[i], acc);
            }
        }
        const float dot = cta_sum_all<NW>(acc.x + acc.y, slot[parity]);
        const float rstd = a.rstd[row];
        if (threadIdx.x == 0) a.k[row] = -(rstd * dot) * a.invN * rstd * rstd;
    }
}

// ... then columns: a warp owns one chunk of columns and walks its split of
// the rows, so dw accumulates in registers as in the register plan.
template <typename T, int MAP>
__global__ void __launch_bounds__(256) drop_bwd_cols_kernel(const DropRmsBwdArgs a, const int64_t rows_per) {
    pdl_wait();
    const DropCtr o = drop_ctr(a.d);
    const int64_t chunks = (a.N + kChunk - 1) / kChunk;
    const int64_t ch = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), c = ch * kChunk;
    if (ch >= chunks) return;
    Frag<T> fw;
    if (a.w) frag_load<T, MAP, true>(fw, static_cast<const T *>(a.w) + c, a.N - c);
    float2 dw[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
    const int64_t r0 = (int64_t)blockIdx.y * rows_per;
    const int64_t r1 = r0 + rows_per < a.rows ? r0 + rows_per : a.rows;
    for (int64_t row = r0; row < r1; ++row) {
        Frag<T> fd, fh, fu;
        frag_load<T, MAP>(fd, static_cast<const T *>(a.dy) + row * a.lddy + c, a.N - c);
        frag_load<T, MAP>(fh, static_cast<const T *>(a.h) + row * a.ldh + c, a.N - c);
        if (a.up) frag_load<T, MAP>(fu, static_cast<const T *>(a.up) + row * a.ldu + c, a.N - c);
        drop_bwd_chunk<T, MAP>(a, o, row, ch, fd, fh, fu, fw, a.rstd[row], a.k[row], dw);
    }
    if (!a.dw) return;
    float *P = a.part + (int64_t)blockIdx.y * a.N;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t col = c + frag_col<MAP>(j);
        if (col < a.N) P[col] = j & 1 ? dw[j >> 1].y : dw[j >> 1].x;
    }
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (drop_<type>.cu).
// ---------------------------------------------------------------------------
template <typename T, int MAP>
cudaError_t launch_dropout_m(const DropoutArgs &a, int sms, cudaStream_t s) {
    constexpr int U = 4;
    const int64_t cpr = (a.N + kChunk - 1) / kChunk;
    int64_t ctas = (a.rows * cpr + 8 * U - 1) / (8 * U);
    const int64_t most = (int64_t)sms * 64;
    if (ctas > most) ctas = most;
    return launch_row(dropout_kernel<T, MAP, U>, (unsigned)ctas, 256u, 0, s, a.d,
                      static_cast<const T *>(a.x), a.ldx, static_cast<T *>(a.y), a.ldy, a.rows, a.N, cpr);
}
template <typename T> cudaError_t launch_dropout_t(const DropoutArgs &a, bool vec, int sms, cudaStream_t s) {
    return vec ? launch_dropout_m<T, vec_map<T>()>(a, sms, s) : launch_dropout_m<T, MAP_S>(a, sms, s);
}

template <typename T, int GT, int U, int MAP>
cudaError_t launch_drop_fwd_k(const DropRmsArgs &a, int sms, cudaStream_t s, Plan *p) {
    constexpr int CTA = GT < 128 ? 128 : GT, G = CTA / GT;
    auto kernel = drop_add_rms_kernel<T, GT, U, MAP>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), CTA, 0, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t need = (a.rows + G - 1) / G;
    p->kind = GT == 32 ? PLAN_WARP : PLAN_CTA;
    p->threads = CTA;
    p->packs = U * 2 * (int)sizeof(T) / 4;
    return launch_row(kernel, (unsigned)(need < 0x7fffffff ? need : 0x7fffffff), (unsigned)CTA, 0, s, a,
                      (int64_t)sms * per_sm * G);
}

// The group and its share of the row: at least 128 threads a row where rows
// are few (latency), a warp a row where they are many.
template <typename T, int MAP>
cudaError_t launch_drop_fwd_m(const DropRmsArgs &a, bool longrow, int sms, cudaStream_t s, Plan *p) {
    const int64_t C = (a.N + kChunk - 1) / kChunk;
    if (!longrow) {
        if (C <= 4 && a.rows >= 4 * (int64_t)sms) {
            if (C <= 1) return launch_drop_fwd_k<T, 32, 1, MAP>(a, sms, s, p);
            if (C <= 2) return launch_drop_fwd_k<T, 32, 2, MAP>(a, sms, s, p);
            return launch_drop_fwd_k<T, 32, 4, MAP>(a, sms, s, p);
        }
        if (C <= 4) return launch_drop_fwd_k<T, 128, 1, MAP>(a, sms, s, p);
        if (C <= 8) return launch_drop_fwd_k<T, 128, 2, MAP>(a, sms, s, p);
        if (C <= 16) return launch_drop_fwd_k<T, 256, 2, MAP>(a, sms, s, p);
        if (C <= 32) return launch_drop_fwd_k<T, 512, 2, MAP>(a, sms, s, p);
        if (C <= 64) return launch_drop_fwd_k<T, 1024, 2, MAP>(a, sms, s, p);
    }
    p->kind = PLAN_GENERIC;
    p->threads = 512;
    p->packs = 1;
    return launch_row(drop_add_rms_long_kernel<T, MAP>, (unsigned)(a.rows < 0x7fffffff ? a.rows : 0x7fffffff),
                      512u, 0, s, a);
}
template <typename T>
cudaError_t launch_drop_fwd_t(const DropRmsArgs &a, bool vec, bool longrow, int sms, cudaStream_t s, Plan *p) {
    return vec ? launch_drop_fwd_m<T, vec_map<T>()>(a, longrow, sms, s, p)
               : launch_drop_fwd_m<T, MAP_S>(a, longrow, sms, s, p);
}

template <typename T, int GT, int U, int MAP>
cudaError_t launch_drop_bwd_k(const DropRmsBwdArgs &a, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    constexpr int CTA = GT < 128 ? 128 : GT, G = CTA / GT;
    auto kernel = drop_add_rms_bwd_kernel<T, GT, U, MAP>;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), CTA, 0, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t ctas = (a.rows + G - 1) / G;
    if (ctas > (int64_t)sms * per_sm) ctas = (int64_t)sms * per_sm;
    if (ctas > kDropMaxParts) ctas = kDropMaxParts;
    p->kind = GT == 32 ? PLAN_WARP : PLAN_CTA;
    p->threads = CTA;
    p->packs = U * 2 * (int)sizeof(T) / 4;
    *parts = ctas;
    return launch_row(kernel, (unsigned)ctas, (unsigned)CTA, 0, s, a);
}

template <typename T, int MAP>
cudaError_t launch_drop_bwd_m(const DropRmsBwdArgs &a, bool longrow, int sms, cudaStream_t s, Plan *p,
                              int64_t *parts) {
    const int64_t C = (a.N + kChunk - 1) / kChunk;
    if (!longrow) {
        if (C <= 4 && a.rows >= 4 * (int64_t)sms) {
            if (C <= 1) return launch_drop_bwd_k<T, 32, 1, MAP>(a, sms, s, p, parts);
            if (C <= 2) return launch_drop_bwd_k<T, 32, 2, MAP>(a, sms, s, p, parts);
            return launch_drop_bwd_k<T, 32, 4, MAP>(a, sms, s, p, parts);
        }
        if (C <= 4) return launch_drop_bwd_k<T, 128, 1, MAP>(a, sms, s, p, parts);
        if (C <= 8) return launch_drop_bwd_k<T, 128, 2, MAP>(a, sms, s, p, parts);
        if (C <= 16) return launch_drop_bwd_k<T, 256, 2, MAP>(a, sms, s, p, parts);
        if (C <= 32) return launch_drop_bwd_k<T, 512, 2, MAP>(a, sms, s, p, parts);
    }
    p->kind = PLAN_GENERIC;
    p->threads = 256;
    p->packs = 1;
    cudaError_t e = launch_row(drop_bwd_dot_kernel<T, MAP>,
                               (unsigned)(a.rows < 0x7fffffff ? a.rows : 0x7fffffff), 512u, 0, s, a);
    if (e != cudaSuccess) return e;
    const int64_t gx = (C + 7) / 8;
    int64_t split = ((int64_t)sms * 8 + gx - 1) / gx;
    if (split > kDropMaxParts) split = kDropMaxParts;
    if (split > a.rows) split = a.rows;
    const int64_t per = (a.rows + split - 1) / split;
    split = (a.rows + per - 1) / per;
    *parts = split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)split);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, drop_bwd_cols_kernel<T, MAP>, a, per);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <typename T>
cudaError_t launch_drop_bwd_t(const DropRmsBwdArgs &a, bool vec, bool longrow, int sms, cudaStream_t s,
                              Plan *p, int64_t *parts) {
    return vec ? launch_drop_bwd_m<T, vec_map<T>()>(a, longrow, sms, s, p, parts)
               : launch_drop_bwd_m<T, MAP_S>(a, longrow, sms, s, p, parts);
}

}  // namespace nrm
