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
//   MAP_V  rows of whole 16-byte packs on 16-byte boundaries: one 16-byte
//          access (16-bit types: columns 8 l + j) or two (binary32: columns
//          4 l + j and 128 + 4 l + j)
//   MAP_A  any N, rows at any element alignment that all tensors share (odd N,
//          contiguous): the same accesses on the 16-byte grid, so a lane's
//          columns are those of MAP_V minus the row's `shift` (its start
//          behind the grid, in elements).  A pack that a row's end cuts is
//          read whole where it lies between the tensor's first and last
//          element (its other half is the neighbouring row's) and trimmed,
//          and written element by element.  A lane's columns straddle two
//          generator blocks: its own and its lower neighbour's, by shuffle.
//   MAP_S  tensors that differ in alignment: columns 32 j + l, eight scalar
//          accesses, the keep bits gathered by shuffles
#pragma once

#include <cstdint>
#include <type_traits>

#include "nrm_device.cuh"
#include "nrm_internal.h"
#include "row_kernels.cuh"  // launch_row

namespace nrm {

constexpr int kChunk = 256;
constexpr int kRowWarps = 4;  // rows (warps) per CTA of the warp plans
constexpr int kBwdWarps = 16;  // the most warps a CTA of the backward's register plan has

// The offset words of this call: the host's plus the device counter's value.
struct DropCtr {
    uint32_t lo, hi;
};
__device__ __forceinline__ DropCtr drop_ctr(const DropArgs &d) {
    uint64_t o = d.offset;
    if (d.offset_dev) o += (uint64_t)*d.offset_dev;
    return DropCtr{(uint32_t)o, (uint32_t)(o >> 32)};
}

// What the generator's first two rounds make of the call's and the row's
// words alone (2 of its 20 products).
struct DropRow {
    uint32_t x1, x2, x3, e2;
};
__device__ __forceinline__ DropRow drop_row(const DropArgs &d, const DropCtr &o, int64_t row) {
    const uint64_t q1 = (uint64_t)o.lo * 0xCD9E8D57u;
    const uint64_t p2 = (uint64_t)((uint32_t)(q1 >> 32) ^ (uint32_t)row ^ d.key[0]) * 0xD2511F53u;
    return DropRow{o.hi ^ d.key[1], (uint32_t)q1 ^ d.key[2], (uint32_t)(p2 >> 32) ^ d.key[3], (uint32_t)p2};
}

// One generator block of a row.
__device__ __forceinline__ uint4 drop_block(const DropArgs &d, const DropRow &r, uint32_t block) {
    const uint64_t p1 = (uint64_t)block * 0xD2511F53u;
    const uint64_t q2 = (uint64_t)((uint32_t)(p1 >> 32) ^ r.x1) * 0xCD9E8D57u;
    uint32_t a = (uint32_t)(q2 >> 32) ^ r.x2, b = (uint32_t)q2, c = r.x3 ^ (uint32_t)p1, e = r.e2;
#pragma unroll
    for (int i = 2; i < 10; ++i) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ d.key[2 * i];
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ e ^ d.key[2 * i + 1];
        e = (uint32_t)p;
    }
    return make_uint4(a, b, c, e);
}

// Which of a lane's 8 elements are kept: the words of its own block (16-bit
// types, MAP_V), or 8 bits gathered from the lanes that computed them.
template <typename T, int MAP> struct Keep {
    static constexpr bool WORDS = MAP == MAP_V && sizeof(T) == 2;
    uint32_t w[WORDS ? 4 : 1];
    __device__ __forceinline__ bool operator()(int j, uint32_t bar) const {
        if constexpr (WORDS)
            return (j & 1 ? w[j >> 1] : w[j >> 1] << 16) > bar;
        else
            return (w[0] >> j) & 1u;
    }
};

// The 8 keep bits of a block, bit j for number j.  Two numbers are compared
// with T at a time: with H the halves' top bits, (x | H) - (T & ~H) borrows
// nothing across the halves, and its top bit says x & ~H >= T & ~H.
__device__ __forceinline__ uint32_t keep_byte(const uint4 &w, const DropArgs &d) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t ge[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t e = (x[i] | 0x80008000u) - d.low2;
        ge[i] = (d.top ? x[i] & e : x[i] | e) & d.any2;
    }
    // the halves' bits to places 2 i and 2 i + 16, then together
    const uint32_t t = ge[0] >> 15 | ge[1] >> 13 | ge[2] >> 11 | ge[3] >> 9;
    return (t | t >> 15) & 0xffu;
}

// The keep sets of one row's neighbouring chunks, in order from `chunk` (the
// whole warp calls).
template <typename T, int MAP> struct Masks {
    const DropArgs &d;
    DropRow r;
    uint32_t block;  // this lane's next block
    uint32_t prev;   // MAP_A: the byte of the block before the warp's next chunk
    int shift;

    __device__ __forceinline__ Masks(const DropArgs &d_, const DropCtr &o, int64_t row, int64_t chunk, int shift_)
        : d(d_), r(drop_row(d_, o, row)), block((uint32_t)(chunk * 32) + (threadIdx.x & 31)), prev(0), shift(shift_) {
        // columns before the row's first are nobody's: chunk 0 needs none
        if (MAP == MAP_A && shift && chunk > 0)
            prev = keep_byte(drop_block(d, r, (uint32_t)(chunk * 32) - 1), d);
    }
    // The byte of this lane's next block, and the keep set of a chunk from its
    // lanes' bytes.
    __device__ __forceinline__ uint32_t next_byte() {
        const uint32_t m = keep_byte(drop_block(d, r, block), d);
        block += 32;
        return m;
    }
    __device__ __forceinline__ Keep<T, MAP> window(uint32_t mine) {
        static_assert(!Keep<T, MAP>::WORDS && MAP != MAP_S, "shifted or binary32 rows");
        const int lane = threadIdx.x & 31;
        Keep<T, MAP> k;
        // columns 8 l - 8 .. 8 l + 7, then the window at -shift
        uint32_t two = mine << 8;
        if (MAP == MAP_A) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, mine, 1);
            two |= lane ? up : prev;
            prev = __shfl_sync(0xffffffffu, mine, 31);
        }
        const int sh = 8 - (MAP == MAP_A ? shift : 0);
        if constexpr (sizeof(T) == 2) {
            k.w[0] = two >> sh;
        } else {
            // pack p of the chunk starts at half (p & 1) of block p / 2
            const int at = sh + (lane & 1) * 4;
            const uint32_t lo = __shfl_sync(0xffffffffu, two, lane >> 1) >> at;
            const uint32_t hi = __shfl_sync(0xffffffffu, two, 16 + (lane >> 1)) >> at;
            k.w[0] = (lo & 15u) | (hi & 15u) << 4;
        }
        return k;
    }
    // The next U keep sets; the generator's chains of all of them first, side by
    // side: the shuffles in between would set them one behind the other (dropout
    // 4096 x 5001 bf16 21.2 us against 23.5; the fused kernels have no registers
    // for it).
    template <int U> __device__ __forceinline__ void all(Keep<T, MAP> (&k)[U]) {
        uint32_t b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) b[u] = next_byte();
#pragma unroll
        for (int u = 0; u < U; ++u) k[u] = window(b[u]);
    }
    __device__ __forceinline__ Keep<T, MAP> next() {
        if constexpr (Keep<T, MAP>::WORDS) {
            const uint4 w = drop_block(d, r, block);
            block += 32;
            Keep<T, MAP> k;
            k.w[0] = w.x; k.w[1] = w.y; k.w[2] = w.z; k.w[3] = w.w;
            return k;
        } else if constexpr (MAP == MAP_S) {
            const int lane = threadIdx.x & 31;
            const uint32_t mine = next_byte();
            Keep<T, MAP> k;
            k.w[0] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                k.w[0] |= (__shfl_sync(0xffffffffu, mine, 4 * j + (lane >> 3)) >> (lane & 7) & 1u) << j;
            return k;
        } else {
            return window(next_byte());
        }
    }
};

// A lane's 8 elements of one chunk, in the storage type.
template <typename T> struct Frag {
    uint32_t r[2 * sizeof(T)];
};

// Place of element j of this lane in a chunk (its column, plus the shift for
// MAP_A).
template <typename T, int MAP> __device__ __forceinline__ int frag_col(int j) {
    const int lane = threadIdx.x & 31;
    return MAP == MAP_S ? 32 * j + lane : sizeof(T) == 2 ? 8 * lane + j : 4 * lane + (j & 3) + 32 * (j & 4);
}

// A row's place on the 16-byte grid: elements from the grid to its start.
template <typename T, int MAP> __device__ __forceinline__ int row_shift(const void *row) {
    return MAP == MAP_A ? (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T)) : 0;
}

// What of a chunk belongs to the row: places head (inclusive) to left
// (exclusive; may be <= 0 or beyond the chunk).
struct Part {
    int head, left;
};
// chunk ch of a row of n elements.
__device__ __forceinline__ Part chunk_part(int64_t ch, int64_t n, int shift) {
    const int64_t left = n + shift - ch * kChunk;
    return Part{ch == 0 ? shift : 0, left < kChunk ? (int)left : kChunk};
}

// Element e (0 .. sizeof-wise V - 1) of a pack as its bits.
template <typename T> using Bits = typename std::conditional<sizeof(T) == 2, unsigned short, uint32_t>::type;

template <typename T> constexpr int kPacks = sizeof(T) / 2;  // 16-byte packs of a fragment (MAP_V, MAP_A)

// Place of a fragment's pack h in its chunk.
template <typename T> __device__ __forceinline__ int pack_at(int h) {
    const int lane = threadIdx.x & 31;
    return sizeof(T) == 2 ? 8 * lane : 128 * h + 4 * lane;
}

// Which of a pack's elements belong to the part, bit j for element j.
template <typename T> __device__ __forceinline__ uint32_t cut_bits(int c, Part b) {
    constexpr int V = IO<T>::V;
    const int lo = b.head - c, hi = b.left - c;
    uint32_t m = (1u << V) - 1u;
    if (lo > 0) m = lo < V ? m >> lo << lo : 0u;
    if (hi < V) m &= hi > 0 ? (1u << hi) - 1u : 0u;
    return m;
}
// Elements of a cut pack, one by one; the others are zeros, and are not stored.
template <typename T> __device__ __forceinline__ uint4 cut_load(const T *p, int c, Part b) {
    constexpr int V = IO<T>::V;
    const Bits<T> *q = reinterpret_cast<const Bits<T> *>(p);
    uint32_t e[V];
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = c + j >= b.head && c + j < b.left ? (uint32_t)q[j] : 0u;
    if constexpr (V == 8)
        return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    else
        return make_uint4(e[0], e[1], e[2], e[3]);
}
template <typename T> __device__ __forceinline__ void cut_store(T *p, uint32_t bits, const uint4 &v) {
    constexpr int V = IO<T>::V;
    Bits<T> *q = reinterpret_cast<Bits<T> *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (bits >> j & 1u) q[j] = (Bits<T>)(V == 8 ? w[j >> 1] >> 16 * (j & 1) : w[j]);
}

// How a lane reaches its elements of U neighbouring chunks of a row: which of
// its packs the row has whole, and which in part.  The same for all rows of
// one shift.
template <typename T, int MAP, int U> struct Access {
    static constexpr int H = MAP == MAP_S ? 1 : kPacks<T>;
    uint32_t whole, some;  // bit u * H + h; `some` includes the whole ones
    uint32_t bits;         // MAP_A: the elements of a cut pack, in the byte of its chunk (a
                           // chunk's second pack, binary32: the upper half of it)
    int64_t ch0, n;
    int shift;

    __device__ __forceinline__ Access(int64_t ch0_, int64_t n_, int shift_)
        : whole(0), some(0), bits(0), ch0(ch0_), n(n_), shift(shift_) {
        if constexpr (MAP != MAP_S) {
            if ((MAP == MAP_V || ch0 > 0) && n + shift - ch0 * kChunk >= U * kChunk) {  // inside the row
                whole = some = (1u << (U * H)) - 1u;
                return;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Part b = part(u);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int c = pack_at<T>(h);
                    const bool s = c < b.left && c + IO<T>::V > b.head;
                    some |= (uint32_t)s << (u * H + h);
                    if (MAP == MAP_A) bits |= cut_bits<T>(c, b) << (8 * u + 4 * h);
                    whole |= (uint32_t)(s && c >= b.head && c + IO<T>::V <= b.left) << (u * H + h);
                }
            }
        }
    }
    __device__ __forceinline__ Part part(int u) const { return chunk_part(ch0 + u, n, shift); }
    // Element 0 of this lane in chunk 0 of the run, behind the row's first.
    __device__ __forceinline__ int64_t first() const {
        return ch0 * kChunk - shift + (MAP == MAP_S ? (int)(threadIdx.x & 31) : pack_at<T>(0));
    }
    // Packs that may be read whole in this row: a cut one reaches up to V - 1
    // elements into the rows before or after.  That stays inside the tensor
    // when as many lie on that side; rows are at least n elements apart.
    __device__ __forceinline__ uint32_t readable(int64_t row, int64_t rows) const {
        if (MAP != MAP_A) return whole;
        constexpr int V = IO<T>::V;
        const int over = (int)((V - ((uint32_t)n + shift) % V) % V);  // places behind the row in its last pack
        // rows that hold as many elements as are needed on a side
        const int before = n >= V ? shift > 0 : (shift + (int)n - 1) / (int)n;
        const int behind = n >= V ? over > 0 : (over + (int)n - 1) / (int)n;
        return row >= before && row + behind < rows ? some : whole;
    }

    // p: the row's element first().
    template <bool KEEP_CACHED = false>
    __device__ __forceinline__ void load(Frag<T> &f, const T *p, int u, uint32_t read) const {
        if constexpr (MAP == MAP_S) {
            const Part b = part(u);
            const int lane = threadIdx.x & 31;
            const Bits<T> *q = reinterpret_cast<const Bits<T> *>(p) + u * kChunk;
            uint32_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = 32 * j + lane < b.left ? (uint32_t)q[32 * j] : 0u;
#pragma unroll
            for (int j = 0; j < 2 * (int)sizeof(T); ++j)
                f.r[j] = sizeof(T) == 2 ? e[2 * j & 7] | e[(2 * j + 1) & 7] << 16 : e[j];
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t bit = 1u << (u * H + h);
                const T *q = p + u * kChunk + 128 * h;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (read & bit)
                    v = KEEP_CACHED ? ld_param(q) : ld_once(q);
                else if (MAP == MAP_A && (some & bit))
                    v = cut_load<T>(q, pack_at<T>(h), part(u));
                f.r[4 * h] = v.x; f.r[4 * h + 1] = v.y; f.r[4 * h + 2] = v.z; f.r[4 * h + 3] = v.w;
            }
        }
    }
    // Zeros in the places of a loaded fragment that are not the row's.
    __device__ __forceinline__ void trim(Frag<T> &f, int u) const {
        if constexpr (MAP == MAP_A) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t bit = 1u << (u * H + h);
                if ((some & ~whole) & bit) {
                    const uint32_t m = bits >> (8 * u + 4 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (sizeof(T) == 2)
                            f.r[i] &= (m >> (2 * i) & 1u ? 0xffffu : 0u) | (m >> (2 * i + 1) & 1u ? 0xffff0000u : 0u);
                        else if (!(m >> i & 1u))
                            f.r[(4 * h + i) % (2 * sizeof(T))] = 0u;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void store(const Frag<T> &f, T *p, int u) const {
        if constexpr (MAP == MAP_S) {
            const Part b = part(u);
            const int lane = threadIdx.x & 31;
            Bits<T> *q = reinterpret_cast<Bits<T> *>(p) + u * kChunk;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (32 * j + lane < b.left)
                    q[32 * j] = (Bits<T>)(sizeof(T) == 2 ? f.r[j >> 1] >> 16 * (j & 1) : f.r[j % (2 * sizeof(T))]);
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t bit = 1u << (u * H + h);
                T *q = p + u * kChunk + 128 * h;
                const uint4 v = make_uint4(f.r[4 * h], f.r[4 * h + 1], f.r[4 * h + 2], f.r[4 * h + 3]);
                if (whole & bit)
                    st_stream(q, v);
                else if (MAP == MAP_A && (some & bit))
                    cut_store<T>(q, bits >> (8 * u + 4 * h), v);
            }
        }
    }
};

// The weights of a lane's columns.  Their vector has an alignment of its own:
// element by element unless both are on the grid.
template <typename T, int MAP, int U>
__device__ __forceinline__ void frag_param(Frag<T> &f, const T *w, const Access<T, MAP, U> &at, int u) {
    if (MAP != MAP_A || (at.shift == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0)) {
        at.template load<true>(f, w + at.first(), u, at.whole);
    } else {
        const Part b = at.part(u);
        const Bits<T> *q = reinterpret_cast<const Bits<T> *>(w) + ((at.ch0 + u) * kChunk - at.shift);
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = frag_col<T, MAP>(j);
            e[j] = c >= b.head && c < b.left ? (uint32_t)q[c] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 2 * (int)sizeof(T); ++j) f.r[j] = sizeof(T) == 2 ? e[2 * j & 7] | e[(2 * j + 1) & 7] << 16 : e[j];
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
template <typename T, int MAP>
__device__ __forceinline__ void drop_apply(const DropArgs &d, const Keep<T, MAP> &k, float2 v[4]) {
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
// Dropout alone: element-wise, one read and one write.  A warp's item is U
// neighbouring chunks of one row; all loads are issued before the generator
// runs.  At 8192 x 8192 bf16 the generator's integer products and the ALU work
// of the selects take 60 % of their pipes' time, so the kernel needs its
// warps: five CTAs per SM (48 registers) 42.9 us, four 46.4, two 48.9, six
// (spills) 54.9.
// ---------------------------------------------------------------------------
template <typename T, int MAP, int U>
__global__ void __launch_bounds__(256, (MAP == MAP_V && sizeof(T) == 2 ? 5 : 3))
    dropout_kernel(const DropArgs d, const T *x, const int64_t ldx, T *y, const int64_t ldy, const int64_t rows,
                   const int64_t N, const uint32_t per_row) {
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(d);
    const int64_t total = rows * per_row;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < total; item += step) {
        const int64_t row = total <= 0xffffffffll ? (int64_t)((uint32_t)item / per_row) : item / per_row;
        const int64_t ch = (item - row * per_row) * U;
        const Access<T, MAP, U> at(ch, N, row_shift<T, MAP>(x + row * ldx));
        const T *p = x + row * ldx + at.first();
        T *q = y + row * ldy + at.first();
        Frag<T> f[U];
        const uint32_t read = at.readable(row, rows);
#pragma unroll
        for (int u = 0; u < U; ++u) at.load(f[u], p, u, read);
        if (d.on) {
            Masks<T, MAP> m(d, o, row, ch, at.shift);
            Keep<T, MAP> k[U];
            if constexpr (MAP == MAP_A) m.all(k);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 v[4];
                frag_unpack<T>(f[u], v);
                if (MAP != MAP_A) k[u] = m.next();
                drop_apply<T, MAP>(d, k[u], v);
                f[u] = frag_pack<T>(v);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) at.store(f[u], q, u);
    }
}

// Sum over the CTA's warps (nw of them), returned to every thread; `slot` as
// for cta_sum_all.
__device__ __forceinline__ float warps_sum_all(float v, float *slot, int nw) {
    const int lane = threadIdx.x & 31;
    v = warp_sum_all(v);
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum_all(lane < nw ? slot[lane] : 0.f);
}

// ---------------------------------------------------------------------------
// Forward of the residual path, register plan: a row per warp (WARP) or per
// CTA of as many warps as the row has U chunks; the row in registers, x and
// the residual read once.  A group's rows are apart by a multiple of 8, so
// that they share one shift (8 rows of any stride are a multiple of 16
// bytes): its columns are the same in all of them, and w is fetched once.
//
// Bound by HBM on the 16-byte grid: 4096 x 4096 bf16 19.7 us, 6.8 TB/s, with
// 73 % of the issue slots used, so off the grid (half as many instructions
// again: a third generator block for a warp's two chunks, shuffles, cut packs) it
// is bound by those: 2795 x 6001 bf16 35.5 us, 56 % of the copy rate, binary32
// 81 %.  The L2 hint for the row that the next
// resident group starts with hides the ramp between rows of one SM.
// ---------------------------------------------------------------------------
template <typename T, bool WARP, int U, int MAP, int REGS>
__global__ void __maxnreg__(REGS) drop_add_rms_kernel(const DropRmsArgs a, const int64_t pf) {
    __shared__ float slot[2][32];
    const int nw = WARP ? 1 : (int)blockDim.x / 32, groups = WARP ? (int)blockDim.x / 32 : 1;
    const int warp = WARP ? 0 : (int)threadIdx.x >> 5;
    const bool lead = WARP ? (threadIdx.x & 31) == 0 : threadIdx.x == 0;
    const int N = (int)a.N;
    const T *W = static_cast<const T *>(a.w);
    int64_t row = (int64_t)blockIdx.x * groups + (WARP ? threadIdx.x >> 5 : 0);
    const Access<T, MAP, U> at(warp * U, N, row_shift<T, MAP>(static_cast<const T *>(a.x) + row * a.ldx));
    const T *X = static_cast<const T *>(a.x) + at.first(), *R = static_cast<const T *>(a.res) + at.first();
    T *H = static_cast<T *>(a.h) + at.first(), *Y = static_cast<T *>(a.y) + at.first();
    // a hint ahead of the wait, as the norm kernels give it: L2 is where the
    // previous grid's writes arrive too
    if (lead && row < a.rows) {
        prefetch_row(static_cast<const T *>(a.x) + row * a.ldx, N);
        prefetch_row(static_cast<const T *>(a.res) + row * a.ldr, N);
    }
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(a.d);
    int parity = 0;
    Frag<T> fw[U];
    if (MAP == MAP_A && W) {
#pragma unroll
        for (int u = 0; u < U; ++u) frag_param(fw[u], W, at, u);
    }
    for (; row < a.rows; row += (int64_t)gridDim.x * groups, parity ^= 1) {
        if (pf > 0 && lead && row + pf < a.rows) {
            prefetch_row(static_cast<const T *>(a.x) + (row + pf) * a.ldx, N);
            prefetch_row(static_cast<const T *>(a.res) + (row + pf) * a.ldr, N);
        }
        Frag<T> fx[U], fr[U];
        const uint32_t read = at.readable(row, a.rows);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at.load(fx[u], X + row * a.ldx, u, read);
            at.load(fr[u], R + row * a.ldr, u, read);
        }
        if (MAP != MAP_A && W) {
#pragma unroll
            for (int u = 0; u < U; ++u) frag_param(fw[u], W, at, u);
        }
        float2 acc = f2(0.f);
        Masks<T, MAP> m(a.d, o, row, at.ch0, at.shift);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 v[4], r[4];
            Keep<T, MAP> k;
            if (a.d.on) k = m.next();
            at.trim(fx[u], u);
            at.trim(fr[u], u);
            frag_unpack<T>(fx[u], v);
            if (a.d.on) drop_apply<T, MAP>(a.d, k, v);
            frag_unpack<T>(fr[u], r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r[i]);
            fr[u] = frag_pack<T>(v);  // the stream's value: the norm is of this rounding
            at.store(fr[u], H + row * a.ldh, u);
            frag_unpack<T>(fr[u], v);
            // places outside the row hold zeros and add nothing
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __ffma2_rn(v[i], v[i], acc);
        }
        float ss = acc.x + acc.y;
        ss = WARP ? warp_sum_all(ss) : warps_sum_all(ss, slot[parity], nw);
        const float rstd = rsqrtf(fmaf(ss, a.invN, a.eps));
        if (lead && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 v[4], w[4];
            frag_unpack<T>(fr[u], v);
            if (W) frag_unpack<T>(fw[u], w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __fmul2_rn(v[i], f2(rstd));
                if (W) v[i] = __fmul2_rn(v[i], w[i]);
            }
            at.store(frag_pack<T>(v), Y + row * a.ldy, u);
        }
    }
}

// Rows longer than the register plan holds, or tensors that differ in
// alignment: the sum of squares while h is written, then h read again (each
// lane re-reads what it wrote, mostly from L2) for y.
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
            const Access<T, MAP, 1> at(ch, a.N, 0);
            Frag<T> fx, fr;
            at.load(fx, X + row * a.ldx + at.first(), 0, at.whole);
            at.load(fr, R + row * a.ldr + at.first(), 0, at.whole);
            float2 v[4], r[4];
            frag_unpack<T>(fx, v);
            if (a.d.on) drop_apply<T, MAP>(a.d, Masks<T, MAP>(a.d, o, row, ch, 0).next(), v);
            frag_unpack<T>(fr, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r[i]);
            fr = frag_pack<T>(v);
            at.store(fr, H + row * a.ldh + at.first(), 0);
            frag_unpack<T>(fr, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __ffma2_rn(v[i], v[i], acc);
        }
        const float ss = cta_sum_all<NW>(acc.x + acc.y, slot[parity]);
        const float rstd = rsqrtf(fmaf(ss, a.invN, a.eps));
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int64_t ch = warp; ch < chunks; ch += NW) {
            const Access<T, MAP, 1> at(ch, a.N, 0);
            Frag<T> fh, fw;
            float2 v[4], w[4];
            at.load(fh, H + row * a.ldh + at.first(), 0, at.whole);
            if (W) frag_param(fw, W, at, 0);
            frag_unpack<T>(fh, v);
            if (W) frag_unpack<T>(fw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __fmul2_rn(v[i], f2(rstd));
                if (W) v[i] = __fmul2_rn(v[i], w[i]);
            }
            at.store(frag_pack<T>(v), Y + row * a.ldy + at.first(), 0);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  With k = -rstd^3 / N * sum_j dy_j w_j h_j (one row-wide sum):
//   dh = rstd * dy * w + k * h + dh_up
// ---------------------------------------------------------------------------
// A row's factor k from its sum; rstd^3 alone can leave binary32 where the
// product does not.
__device__ __forceinline__ float bwd_factor(float rstd, float dot, float invN) {
    return -(rstd * dot) * invN * rstd * rstd;
}
// A lane's share of the row's sum.
template <typename T>
__device__ __forceinline__ float2 bwd_dot(const Frag<T> &fd, const Frag<T> &fh, const Frag<T> &fw, bool weighted,
                                          float2 acc) {
    float2 dy[4], h[4], w[4];
    frag_unpack<T>(fd, dy);
    frag_unpack<T>(fh, h);
    if (weighted) frag_unpack<T>(fw, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (weighted) dy[i] = __fmul2_rn(dy[i], w[i]);
        acc = __ffma2_rn(dy[i], h[i], acc);
    }
    return acc;
}
// The outputs of one lane's 8 elements of chunk u of a row, and their share of
// dw.
template <typename T, int MAP, int U>
__device__ __forceinline__ void drop_bwd_chunk(const DropRmsBwdArgs &a, Masks<T, MAP> &m, const Access<T, MAP, U> &at,
                                               T *dres, T *dx, int u, const Frag<T> &fd, const Frag<T> &fh,
                                               const Frag<T> &fu, const Frag<T> &fw, float rstd, float k,
                                               float2 dw[4]) {
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
    if (a.dres) at.store(frag_pack<T>(dy), dres, u);
    if (a.dx) {
        if (a.d.on) drop_apply<T, MAP>(a.d, m.next(), dy);
        at.store(frag_pack<T>(dy), dx, u);
    }
}

// A warp's sums of one chunk into row P of the partials: through shared memory
// (the warp's own), so that the stores are of neighbouring columns.  c0: the
// column of the chunk's place 0.
template <typename T, int MAP>
__device__ __forceinline__ void store_sums(float *stage, const float2 dw[4], float *P, int64_t c0, int64_t n) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) stage[frag_col<T, MAP>(j)] = j & 1 ? dw[j >> 1].y : dw[j >> 1].x;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t c = c0 + 32 * j + lane;
        if (c >= 0 && c < n) P[c] = stage[32 * j + lane];
    }
}

// Register plan: persistent groups (as the forward's), a row at a time; a
// thread's columns are the same in every row, so dw accumulates in registers
// and each CTA leaves one row of partial sums (folded in order by
// dw_fold_kernel: no atomics, the same bits every time).  The mask is made
// again from the seed: reading one back would add 1 to 16 bits an element.
//
// 4096 x 4096 bf16 with dh_up 29.3 us (2.3 of them the fold), 5.7 TB/s, 84 % of
// the copy rate: dw, w and two rows fill 119 registers, so an SM has 16 warps,
// at 58 % of its issue slots, and their waits are not all covered.  Off the
// 16-byte grid instructions bound it: 1999 x 5001 f16 27.5 us, 43 %.
template <typename T, bool WARP, int U, int MAP, int REGS, bool AHEAD>
__global__ void __maxnreg__(REGS) drop_add_rms_bwd_kernel(const DropRmsBwdArgs a) {
    constexpr int G = WARP ? kRowWarps : 1;
    __shared__ float slot[2][32];
    __shared__ float part[WARP ? G - 1 : 1][WARP ? U * kChunk : 1];
    __shared__ float stage[WARP ? 1 : kBwdWarps][kChunk];
    const int nw = WARP ? 1 : (int)blockDim.x / 32;
    const int warp = WARP ? 0 : (int)threadIdx.x >> 5;
    const bool lead = WARP ? (threadIdx.x & 31) == 0 : threadIdx.x == 0;
    const int N = (int)a.N;
    const T *W = static_cast<const T *>(a.w);
    int64_t row = (int64_t)blockIdx.x * G + (WARP ? threadIdx.x >> 5 : 0);
    const Access<T, MAP, U> at(warp * U, N, row_shift<T, MAP>(static_cast<const T *>(a.dy) + row * a.lddy));
    const T *DY = static_cast<const T *>(a.dy) + at.first(), *H = static_cast<const T *>(a.h) + at.first();
    const T *UP = static_cast<const T *>(a.up) + at.first();
    T *DR = static_cast<T *>(a.dres) + at.first(), *DX = static_cast<T *>(a.dx) + at.first();
    const int64_t step = (int64_t)gridDim.x * G;
    auto prefetch = [&](int64_t r) {
        if (lead && r < a.rows) {
            prefetch_row(static_cast<const T *>(a.dy) + r * a.lddy, N);
            prefetch_row(static_cast<const T *>(a.h) + r * a.ldh, N);
            if (a.up) prefetch_row(static_cast<const T *>(a.up) + r * a.ldu, N);
        }
    };
    prefetch(row);
    if (AHEAD) prefetch(row + step);
    pdl_wait();
    pdl_launch_dependents();
    const DropCtr o = drop_ctr(a.d);
    Frag<T> fw[U];
    float2 dw[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (W) frag_param(fw[u], W, at, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[u][i] = f2(0.f);
    }
    Frag<T> fd[U], fh[U], fu[U];
    float rstd = 0.f;
    auto fetch = [&](int64_t r, Frag<T>(&xd)[U], Frag<T>(&xh)[U], Frag<T>(&xu)[U], float &xr) {
        const uint32_t read = at.readable(r, a.rows);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at.load(xd[u], DY + r * a.lddy, u, read);
            at.load(xh[u], H + r * a.ldh, u, read);
            if (a.up) at.load(xu[u], UP + r * a.ldu, u, read);
        }
        xr = a.rstd[r];
    };
    if (AHEAD && row < a.rows) fetch(row, fd, fh, fu, rstd);
    int parity = 0;
    for (; row < a.rows; row += step, parity ^= 1) {
        prefetch(row + (AHEAD ? 2 : 1) * step);
        if (!AHEAD) fetch(row, fd, fh, fu, rstd);
        float2 acc = f2(0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // with zeros for dy what the others hold there reaches no output
            // (0 times an infinity would: h too)
            at.trim(fd[u], u);
            at.trim(fh[u], u);
            acc = bwd_dot<T>(fd[u], fh[u], fw[u], W != nullptr, acc);
        }
        float dot = acc.x + acc.y;
        dot = WARP ? warp_sum_all(dot) : warps_sum_all(dot, slot[parity], nw);
        Frag<T> nd[AHEAD ? U : 1], nh[AHEAD ? U : 1], nu[AHEAD ? U : 1];
        float nr = 0.f;
        if constexpr (AHEAD) {
            if (row + step < a.rows) fetch(row + step, nd, nh, nu, nr);
        }
        const float k = bwd_factor(rstd, dot, a.invN);
        Masks<T, MAP> m(a.d, o, row, at.ch0, at.shift);
#pragma unroll
        for (int u = 0; u < U; ++u)
            drop_bwd_chunk(a, m, at, DR + row * a.lddr, DX + row * a.lddx, u, fd[u], fh[u], fu[u], fw[u], rstd, k,
                           dw[u]);
        if constexpr (AHEAD) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                fd[u] = nd[u];
                fh[u] = nh[u];
                fu[u] = nu[u];
            }
            rstd = nr;
        }
    }
    // (a stepped grid is rounded up: a CTA past the last row has no partial row)
    if (!a.dw || (int64_t)blockIdx.x * G >= a.rows) return;
    if constexpr (WARP) {
        // the CTA's warps meet in shared memory by column, added in order
        const int g = threadIdx.x >> 5;
        if (g > 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = u * kChunk + frag_col<T, MAP>(j) - at.shift;
                    if (c >= 0 && c < N) part[g - 1][c] = j & 1 ? dw[u][j >> 1].y : dw[u][j >> 1].x;
                }
        }
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = u * kChunk + frag_col<T, MAP>(j) - at.shift;
                float &s = j & 1 ? dw[u][j >> 1].y : dw[u][j >> 1].x;
                if (c >= 0 && c < N)
                    for (int q = 0; q < G - 1; ++q) s += part[q][c];
            }
    }
    float *P = a.part + (int64_t)blockIdx.x * a.N;
#pragma unroll
    for (int u = 0; u < U; ++u) store_sums<T, MAP>(stage[warp], dw[u], P, (at.ch0 + u) * kChunk - at.shift, a.N);
}

// Long rows (or tensors that differ in alignment): the row sums first (k per
// row into the workspace), which reads dy and h once more than the register
// plan: binary32 1638 x 10240 90.9 us, 54 % of the copy rate by the bytes that a
// single pass needs (register plan: 61.9, 80 %) ...
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
            const Access<T, MAP, 1> at(ch, a.N, 0);
            Frag<T> fd, fh, fw;
            at.load(fd, static_cast<const T *>(a.dy) + row * a.lddy + at.first(), 0, at.whole);
            at.load(fh, static_cast<const T *>(a.h) + row * a.ldh + at.first(), 0, at.whole);
            if (a.w) frag_param(fw, static_cast<const T *>(a.w), at, 0);
            acc = bwd_dot<T>(fd, fh, fw, a.w != nullptr, acc);
        }
        const float dot = cta_sum_all<NW>(acc.x + acc.y, slot[parity]);
        const float rstd = a.rstd[row];
        if (threadIdx.x == 0) a.k[row] = bwd_factor(rstd, dot, a.invN);
    }
}

// ... then columns: a warp owns one chunk of columns and walks its split of
// the rows, so dw accumulates in registers as in the register plan.
template <typename T, int MAP>
__global__ void __launch_bounds__(256) drop_bwd_cols_kernel(const DropRmsBwdArgs a, const int64_t rows_per) {
    __shared__ float stage[8][kChunk];
    pdl_wait();
    const DropCtr o = drop_ctr(a.d);
    const int64_t chunks = (a.N + kChunk - 1) / kChunk;
    const int64_t ch = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (ch >= chunks) return;
    const Access<T, MAP, 1> at(ch, a.N, 0);
    Frag<T> fw;
    if (a.w) frag_param(fw, static_cast<const T *>(a.w), at, 0);
    float2 dw[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
    const int64_t r0 = (int64_t)blockIdx.y * rows_per;
    const int64_t r1 = r0 + rows_per < a.rows ? r0 + rows_per : a.rows;
    for (int64_t row = r0; row < r1; ++row) {
        Frag<T> fd, fh, fu;
        at.load(fd, static_cast<const T *>(a.dy) + row * a.lddy + at.first(), 0, at.whole);
        at.load(fh, static_cast<const T *>(a.h) + row * a.ldh + at.first(), 0, at.whole);
        if (a.up) at.load(fu, static_cast<const T *>(a.up) + row * a.ldu + at.first(), 0, at.whole);
        Masks<T, MAP> m(a.d, o, row, ch, 0);
        drop_bwd_chunk(a, m, at, static_cast<T *>(a.dres) + row * a.lddr + at.first(),
                       static_cast<T *>(a.dx) + row * a.lddx + at.first(), 0, fd, fh, fu, fw, a.rstd[row], a.k[row], dw);
    }
    if (!a.dw) return;
    store_sums<T, MAP>(stage[threadIdx.x >> 5], dw, a.part + (int64_t)blockIdx.y * a.N, ch * kChunk, a.N);
}

// ---------------------------------------------------------------------------
// Launchers, one instance of each per storage type (drop_<type>.cu).
// ---------------------------------------------------------------------------
template <typename T, int MAP, int U>
cudaError_t launch_dropout_u(const DropoutArgs &a, int64_t per_row, int sms, cudaStream_t s) {
    int64_t ctas = (a.rows * per_row + 7) / 8;
    const int64_t most = (int64_t)sms * 256;
    if (ctas > most) ctas = most;
    return launch_row(dropout_kernel<T, MAP, U>, (unsigned)ctas, 256u, 0, s, a.d,
                      static_cast<const T *>(a.x), a.ldx, static_cast<T *>(a.y), a.ldy, a.rows, a.N,
                      (uint32_t)per_row);
}
// Chunks of a row of n elements, wherever it starts.
template <typename T> int64_t row_chunks(int64_t n, int map) {
    return (n + (map == MAP_A ? IO<T>::V - 1 : 0) + kChunk - 1) / kChunk;
}
// Chunks per item: the most whose last item of a row is not mostly empty.
template <typename T, int MAP>
cudaError_t launch_dropout_m(const DropoutArgs &a, int sms, cudaStream_t s) {
    const int64_t c = row_chunks<T>(a.N, MAP);
    const int64_t i4 = (c + 3) / 4, i2 = (c + 1) / 2;
    if (sizeof(T) == 2 && i4 * 4 * 8 <= c * 9) return launch_dropout_u<T, MAP, sizeof(T) == 2 ? 4 : 2>(a, i4, sms, s);
    if (i2 * 2 * 8 <= c * 9) return launch_dropout_u<T, MAP, 2>(a, i2, sms, s);
    return launch_dropout_u<T, MAP, 1>(a, c, sms, s);
}
template <typename T> cudaError_t launch_dropout_t(const DropoutArgs &a, int map, int sms, cudaStream_t s) {
    return map == MAP_V   ? launch_dropout_m<T, MAP_V>(a, sms, s)
           : map == MAP_A ? launch_dropout_m<T, MAP_A>(a, sms, s)
                          : launch_dropout_m<T, MAP_S>(a, sms, s);
}

// Grid of the register plans: every row its group (MAP_V, forward), or
// resident groups that step over the rows by a multiple of 8.
inline int64_t stepped_grid(int64_t ctas, int64_t resident) {
    ctas = (ctas + 7) / 8 * 8;
    resident = resident / 8 * 8;
    if (resident < 8) resident = 8;
    return ctas < resident ? ctas : resident;
}

template <typename T, bool WARP, int U, int MAP, int REGS>
cudaError_t launch_drop_fwd_k(const DropRmsArgs &a, int warps, int sms, cudaStream_t s, Plan *p) {
    auto kernel = drop_add_rms_kernel<T, WARP, U, MAP, REGS>;
    const int threads = 32 * warps, G = WARP ? warps : 1;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), threads, 0, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t ctas = (a.rows + G - 1) / G;
    int64_t pf = (int64_t)sms * per_sm * G;
    if (MAP == MAP_A) {
        ctas = stepped_grid(ctas, (int64_t)sms * per_sm);
        pf = ctas * G;
    }
    if (ctas > 0x7fffffff) ctas = 0x7ffffff8;
    p->kind = WARP ? PLAN_WARP : PLAN_CTA;
    p->threads = threads;
    p->packs = U * 2 * (int)sizeof(T) / 4;
    return launch_row(kernel, (unsigned)ctas, (unsigned)threads, 0, s, a, pf);
}

// The group and its share of the row: a warp a row where rows are short and
// many (16384 x 1024 bf16 20.8 us, by CTAs of a chunk a warp 26.6; binary32 up
// to two chunks, 16384 x 640 26.2 us by warps, 24.2 by CTAs), else a CTA of as
// many warps as the row needs.  The bounds on the registers buy rows in flight:
// 16384 x 256 bf16 8.8 us with 64, 10.0 with the 84 that the compiler took.
template <typename T, int MAP>
cudaError_t launch_drop_fwd_m(const DropRmsArgs &a, int sms, cudaStream_t s, Plan *p) {
    const int C = (int)row_chunks<T>(a.N, MAP);
    constexpr int R = MAP == MAP_V && sizeof(T) == 2 ? 64 : 96;
    const int warps = (C + 1) / 2;
    if (C <= 4 && a.rows >= 4 * (int64_t)sms) {
        constexpr int E = MAP == MAP_V ? 0 : 24;
        constexpr bool H = sizeof(T) == 2;
        if (C <= 1) return launch_drop_fwd_k<T, true, 1, MAP, 64 + E>(a, kRowWarps, sms, s, p);
        if (C <= 2) return launch_drop_fwd_k<T, true, 2, MAP, H ? 72 + E : 128>(a, kRowWarps, sms, s, p);
        if constexpr (H) return launch_drop_fwd_k<T, true, 4, MAP, 128>(a, kRowWarps, sms, s, p);
    }
    if (C <= 4) return launch_drop_fwd_k<T, false, 1, MAP, 64>(a, C, sms, s, p);
    // the registers of a CTA's warps come from four banks of 16384, whole warps each
    if (warps <= 4 * (16384 / (32 * R))) return launch_drop_fwd_k<T, false, 2, MAP, R>(a, warps, sms, s, p);
    return launch_drop_fwd_k<T, false, 2, MAP, 64>(a, warps, sms, s, p);
}
template <typename T, int MAP>
cudaError_t launch_drop_fwd_long(const DropRmsArgs &a, cudaStream_t s, Plan *p) {
    p->kind = PLAN_GENERIC;
    p->threads = 512;
    p->packs = 1;
    return launch_row(drop_add_rms_long_kernel<T, MAP>, (unsigned)(a.rows < 0x7fffffff ? a.rows : 0x7fffffff),
                      512u, 0, s, a);
}
constexpr int kDropFwdChunks = 64;
constexpr int kDropBwdChunks = 64;
template <typename T>
cudaError_t launch_drop_fwd_t(const DropRmsArgs &a, int map, bool longrow, int sms, cudaStream_t s, Plan *p) {
    longrow = longrow || row_chunks<T>(a.N, map) > kDropFwdChunks;
    if (map == MAP_V) return longrow ? launch_drop_fwd_long<T, MAP_V>(a, s, p) : launch_drop_fwd_m<T, MAP_V>(a, sms, s, p);
    if (map == MAP_A && !longrow) return launch_drop_fwd_m<T, MAP_A>(a, sms, s, p);
    return launch_drop_fwd_long<T, MAP_S>(a, s, p);
}

template <typename T, bool WARP, int U, int MAP, int REGS, bool AHEAD>
cudaError_t launch_drop_bwd_k(const DropRmsBwdArgs &a, int warps, int sms, cudaStream_t s, Plan *p,
                              int64_t *parts) {
    if (warps > kBwdWarps) return cudaErrorInvalidConfiguration;
    auto kernel = drop_add_rms_bwd_kernel<T, WARP, U, MAP, REGS, AHEAD>;
    const int threads = 32 * warps, G = WARP ? warps : 1;
    int per_sm = 0;
    const cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), threads, 0, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t ctas = (a.rows + G - 1) / G, most = (int64_t)sms * per_sm;
    if (most > kDropMaxParts) most = kDropMaxParts;
    if (MAP == MAP_A)
        ctas = stepped_grid(ctas, most);
    else if (ctas > most)
        ctas = most;
    p->kind = WARP ? PLAN_WARP : PLAN_CTA;
    p->threads = threads;
    p->packs = U * 2 * (int)sizeof(T) / 4;
    *parts = ctas < (a.rows + G - 1) / G ? ctas : (a.rows + G - 1) / G;
    return launch_row(kernel, (unsigned)ctas, (unsigned)threads, 0, s, a);
}
template <typename T, int MAP>
cudaError_t launch_drop_bwd_m(const DropRmsBwdArgs &a, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const int C = (int)row_chunks<T>(a.N, MAP);
    // The row ahead in registers while this one's outputs are made: 31.0 us
    // against 32.3 at 4096 x 4096 bf16; binary32 and shifted rows have no
    // registers left for it.
    constexpr bool AHEAD = sizeof(T) == 2 && MAP == MAP_V;
    const int warps = (C + 1) / 2;
    if (C <= 4 && a.rows >= 4 * (int64_t)sms) {
        if (C <= 1) return launch_drop_bwd_k<T, true, 1, MAP, 128, AHEAD>(a, kRowWarps, sms, s, p, parts);
        if (C <= 2) return launch_drop_bwd_k<T, true, 2, MAP, 160, AHEAD>(a, kRowWarps, sms, s, p, parts);
        return launch_drop_bwd_k<T, true, 4, MAP, 255, AHEAD>(a, kRowWarps, sms, s, p, parts);
    }
    // a chunk a warp up to 6 chunks (10922 x 1536 bf16 34.3 us against 39.8 with
    // two, 8192 x 2048 33.8 against 32.4)
    if (C <= 6) return launch_drop_bwd_k<T, false, 1, MAP, 80, false>(a, C, sms, s, p, parts);
    // two CTAs per SM matter more than the row ahead: up to 8 warps have both,
    // up to 10 the former (4096 x 5120 bf16 38.3 us against 47.1), beyond that
    // one CTA fits either way
    if (warps > 8 && warps <= 10) return launch_drop_bwd_k<T, false, 2, MAP, 96, false>(a, warps, sms, s, p, parts);
    // beyond 32 chunks: some spills, but read once (1024 x 16384 bf16 40.3 us,
    // 51.5 through the long-row plan; binary32 1398 x 12000 63.8 and 91.4)
    if (C > 48) return launch_drop_bwd_k<T, false, 4, MAP, 128, false>(a, (C + 3) / 4, sms, s, p, parts);
    if (C > 32) return launch_drop_bwd_k<T, false, 4, MAP, 168, false>(a, (C + 3) / 4, sms, s, p, parts);
    return launch_drop_bwd_k<T, false, 2, MAP, 128, AHEAD>(a, warps, sms, s, p, parts);
}
template <typename T, int MAP>
cudaError_t launch_drop_bwd_long(const DropRmsBwdArgs &a, int sms, cudaStream_t s, Plan *p, int64_t *parts) {
    const int64_t C = row_chunks<T>(a.N, MAP);
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
cudaError_t launch_drop_bwd_t(const DropRmsBwdArgs &a, int map, bool longrow, int sms, cudaStream_t s,
                              Plan *p, int64_t *parts) {
    const int64_t C = row_chunks<T>(a.N, map);
    // the most chunks of binary32 spill most: that pays while every SM has rows
    // to go on with (1024 x 16384 80.3 us, by the long-row plan 88.4; 300 rows
    // 30.6 and 27.4)
    longrow = longrow || C > kDropBwdChunks || (sizeof(T) == 4 && C > 48 && a.rows < 4 * (int64_t)sms);
    if (map == MAP_V)
        return longrow ? launch_drop_bwd_long<T, MAP_V>(a, sms, s, p, parts)
                       : launch_drop_bwd_m<T, MAP_V>(a, sms, s, p, parts);
    if (map == MAP_A && !longrow) return launch_drop_bwd_m<T, MAP_A>(a, sms, s, p, parts);
    return launch_drop_bwd_long<T, MAP_S>(a, sms, s, p, parts);
}

}  // namespace nrm
