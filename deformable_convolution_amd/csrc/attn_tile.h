// attn_tile.h -- what the attention kernels share: 32 x 32 matrix tiles of
// either storage type, tiles staged from strided rows into LDS, and the keys
// that a query sees.
//
// Every product is taken 32 x 32 with 16 terms at a time.  A lane holds row
// (or column) lane % 32 of an operand and eight of the 16 terms; the terms'
// order may be anything as long as both operands agree.  bf16 storage: one
// 32x32x16 matrix instruction.  fp32 storage: eight 32x32x2 ones on the same
// eight values, so the fp32 results keep fp32 products.  A result's lane
// holds column lane % 32 and, in element r, row 8*(r/4) + 4*(lane/32) + r%4.
// Its elements 8s .. 8s+7 are therefore the eight terms 16s + 8*(j/4) +
// 4*(lane/32) + j%4 of an operand with that column, without any exchange
// between lanes: a product's result (the probabilities) becomes the next
// product's operand where it stands.  The other operand then has to be read
// down the columns of its tile in the same order of terms (col_frag).
#pragma once

#include "seq_internal.h"

namespace dc1d {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kMaxLen = 1 << 29;  // limit of every length, and of window and |q_start|

// ---- tiles in LDS -------------------------------------------------------------
//
// A tile is rows of DP elements, row after row, in 16-byte pieces whose index
// is exchanged with the row's: piece c of row r stands at (r * PER + c) ^
// mix(r), PER = DP elements in pieces.  LDS has 64 banks of 4 bytes; without
// the exchange rows of 256 bytes all start in the same bank (a row read by
// 32 lanes then took 64 clocks for its 1 KiB, measured on a wave's reads),
// with it both ways of reading a tile run at the LDS's rate: along the rows
// 4.2 clocks for 1 KiB, down the columns 2.5 for 512 bytes.  Padding the rows
// by 16 or 32 bytes instead served one way at full rate and the other at half.
template <int PER>
__host__ __device__ constexpr int mix(int row) {
    static_assert(PER == 4 || PER == 8 || PER == 16 || PER == 32, "64 to 512 bytes a row");
    if constexpr (PER == 4) return (row >> 2) & 3;
    if constexpr (PER == 8) return ((row & 2) << 1) | ((row >> 2) & 3);
    return ((row & 3) << 2) | ((row >> 2) & 3);
}

template <typename T>
struct Tile;

template <>
struct Tile<BF16> {
    using E = uint16_t;
    using Frag = bf16x8;
    static constexpr int CH = 8;

    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // Elements c0 .. c0+7 of a tile's row (c0 a multiple of 8)
    template <int DP>
    static __device__ __forceinline__ Frag row_frag(const E *tile, int row, int c0) {
        return *(const Frag *)(tile + (((row * (DP / CH) + c0 / CH) ^ mix<DP / CH>(row)) * CH));
    }
    // Rows K0 .. K0+31 of the columns c0 + 32 d + lane%32, d < N, of the tile OFF
    // elements on, as the operands f[d][0] (the first 16 rows) and f[d][1]: eight
    // elements each, rows 8*(j/4) + 4*(lane/32) + j%4.  A transposing read takes a 4 x 16 block whose lane
    // 4*i + c addresses elements 4c .. 4c+3 of row i, and gives lane i of the 16
    // the block's column i.  The reads are written out with their own wait: as
    // builtins each would first wait for the loads into LDS that are in flight
    // for the tiles to come.
    template <int DP, int N, int OFF, int K0>
    static __device__ __forceinline__ void col_frags(const E *tile, int c0, int lane, Frag (*f)[2]) {
        static_assert(N == 1 || N == 2, "one or two slices");
        const int i = lane & 15, row = 4 * (lane >> 5) + (i >> 2), c = ((lane >> 4) & 1) * 16 + (i & 3) * 4;
        auto at = [&](int r, int d) {
            const E *const p = tile + (((r * (DP / CH) + (c0 + 32 * d + c) / CH) ^ mix<DP / CH>(r)) * CH + c % CH);
            return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const E *)p;
        };
        constexpr int here = (OFF + K0 * DP) * sizeof(E), next = here + 16 * DP * sizeof(E);  // mix() repeats after 16 rows
        static_assert(next < 1 << 16, "the offset's range");
        i16x4 v[2 * N][2];
        if constexpr (N == 1) {
            asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
                         "ds_read_b64_tr_b16 %1, %5 offset:%6\n\t"
                         "ds_read_b64_tr_b16 %2, %4 offset:%7\n\t"
                         "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1])
                         : "v"(at(row, 0)), "v"(at(row + 8, 0)), "n"(here), "n"(next)
                         : "memory");
        } else {
            asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %1, %9 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %2, %8 offset:%13\n\t"
                         "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
                         "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %5, %11 offset:%12\n\t"
                         "ds_read_b64_tr_b16 %6, %10 offset:%13\n\t"
                         "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1]), "=&v"(v[2][0]), "=&v"(v[2][1]),
                           "=&v"(v[3][0]), "=&v"(v[3][1])
                         : "v"(at(row, 0)), "v"(at(row + 8, 0)), "v"(at(row, 1)), "v"(at(row + 8, 1)), "n"(here), "n"(next)
                         : "memory");
        }
        typedef short i16x8 __attribute__((ext_vector_type(8)));
#pragma unroll
        for (int k = 0; k < 2 * N; ++k)
            f[k >> 1][k & 1] = __builtin_bit_cast(Frag, (i16x8)__builtin_shufflevector(v[k][0], v[k][1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // Elements 8s .. 8s+7 of a result as an operand, rounded to nearest even.
    template <int S>
    static __device__ __forceinline__ Frag pack(const f32x16 &c) {
        const f32x8 v = __builtin_shufflevector(c, c, 8 * S, 8 * S + 1, 8 * S + 2, 8 * S + 3, 8 * S + 4, 8 * S + 5,
                                                8 * S + 6, 8 * S + 7);
        return __builtin_convertvector(v, Frag);
    }
    static __device__ __forceinline__ void store4(E *p, f32x4 v) {
        *(bf16x4 *)p = __builtin_convertvector(v, bf16x4);
    }
};

template <>
struct Tile<F32> {
    using E = float;
    using Frag = f32x8;
    static constexpr int CH = 4;

    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    template <int DP>
    static __device__ __forceinline__ Frag row_frag(const E *tile, int row, int c0) {
        auto at = [&](int c) { return *(const f32x4 *)(tile + (((row * (DP / CH) + c / CH) ^ mix<DP / CH>(row)) * CH)); };
        const f32x4 a = at(c0), b = at(c0 + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    template <int DP, int N, int OFF, int K0>
    static __device__ __forceinline__ void col_frags(const E *tile, int c0, int lane, Frag (*f)[2]) {
#pragma unroll
        for (int k = 0; k < 2 * N; ++k) {
            const int c = c0 + 32 * (k >> 1) + (lane & 31);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = 16 * (k & 1) + 4 * (lane >> 5) + 8 * (j >> 2) + (j & 3);
                f[k >> 1][k & 1][j] = tile[OFF + K0 * DP + ((row * (DP / CH) + c / CH) ^ mix<DP / CH>(row)) * CH + c % CH];
            }
        }
    }
    template <int S>
    static __device__ __forceinline__ Frag pack(const f32x16 &c) {
        return __builtin_shufflevector(c, c, 8 * S, 8 * S + 1, 8 * S + 2, 8 * S + 3, 8 * S + 4, 8 * S + 5, 8 * S + 6,
                                       8 * S + 7);
    }
    static __device__ __forceinline__ void store4(E *p, f32x4 v) { *(f32x4 *)p = v; }
};

// One 16-byte piece of a row of D elements, from element col on; elements at
// and past D are zero.  VEC: col < D means the whole piece is inside and
// aligned.  The load itself is unconditional where VEC (at a clamped
// element), so that several of a thread's loads are in flight together.
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 load_piece(const typename T::T *row, int col, int D) {
    if constexpr (VEC) {
        return *(const u32x4 *)(row + (col < D ? col : 0));
    } else {
        constexpr int CH = Tile<T>::CH;
        typename T::T e[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) e[i] = col + i < D ? row[col + i] : (typename T::T)0;
        u32x4 r;
        __builtin_memcpy(&r, e, 16);
        return r;
    }
}

// Row n of a key head's queries: position n / G, head n % G of its G heads.
struct RowAt {
    int pos, head;
};
__device__ __forceinline__ RowAt row_at(const AttnArgs &a, int64_t n) {
    const uint32_t pos = fdiv((uint32_t)n, a.by_G);
    return {(int)pos, (int)((uint32_t)n - pos * (uint32_t)a.G)};
}

// A tile of ROWS rows of DP elements brought into LDS by NT threads (whole
// waves).  Rows ahead of `from`, rows at and past `limit` and elements at and
// past D become zero, whatever memory holds there: what no row of the other
// operand sees meets probability 0 in a product, where a NaN would not vanish.
//
// Aligned rows (VEC) go from memory to LDS without passing through registers:
// a load of the wave writes 64 consecutive pieces of LDS, each lane's from an
// address of its own, and a lane whose offset lies outside the buffer's range
// writes zeros.  Such loads are in flight until landed().  Rows that are not
// aligned, or so far apart that a tile passes 32-bit offsets (not `near`),
// are read element by element (or piece by piece) and stored at once.
//
// A thread's i-th piece stands at place t + i NT, i.e. row t / PER + i STEP,
// and mix() is linear in the row's bits: its column is the first piece's with
// a constant exchanged in.
template <typename T, int ROWS, int DP, int NT, bool VEC>
struct Stage {
    using E = typename T::T;
    static constexpr int CH = Tile<T>::CH, PER = DP / CH, N = (ROWS * PER + NT - 1) / NT;
    static constexpr int STEP = NT / PER;
    static constexpr bool PART = ROWS * PER < NT;  // fewer pieces than threads
    static_assert(NT % PER == 0, "a thread's pieces are of one column, but for the exchange");
    static_assert(PART ? ROWS * PER % 64 == 0 : ROWS * PER % NT == 0, "whole waves carry the tile");
    static constexpr int64_t kNear = 1 << 22;       // elements between rows: 64 rows of 4 bytes stay below 2^30
    static constexpr uint32_t kRange = 0x7fffffff, kOut = 0x80000000u;
    uint32_t row, col, rows_at;  // the first piece's row and first element; the row's offset in bytes
    bool near;

    // rows `stride` elements apart
    __device__ __forceinline__ void init(int64_t stride, int t) {
        row = t / PER;
        col = ((t % PER) ^ mix<PER>(row)) * CH;
        near = VEC && stride < kNear;
        rows_at = row * (uint32_t)stride * (uint32_t)sizeof(E);
    }
    // rows of a key head's queries: all of a thread's pieces are of one head
    // where G divides the rows between them.  Where it does not they are loaded
    // piece by piece: causal gradients of 4 x 2048 positions, 6 and 8 heads over
    // 1 of 128 (times two), bf16: 301 and 279 us.
    __device__ __forceinline__ void init_rows(const AttnArgs &a, const Strides3 &st, int t) {
        row = t / PER;
        col = ((t % PER) ^ mix<PER>(row)) * CH;
        near = VEC && ROWS % a.G == 0 && (N == 1 || STEP % a.G == 0) && st.l < kNear && st.h < kNear;
        const RowAt at = row_at(a, row);
        rows_at = ((uint32_t)at.pos * (uint32_t)st.l + (uint32_t)at.head * (uint32_t)st.h) * (uint32_t)sizeof(E);
    }
    static constexpr int col_flip(int i) { return mix<PER>(i * STEP) * CH; }

    // base and lds are the same for the whole wave
    static __device__ __forceinline__ void to_lds(const E *base, uint32_t off, E *lds) {
        const uint64_t p = (uint64_t)base;
        const uint64_t u = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p) |
                           (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(p >> 32)) << 32;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)u, 0, kRange, 0x00027000);
        typedef __attribute__((address_space(3))) void lds_void;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, off, 0, 0, 0);
    }
    // pieces whose rows are `step` elements apart from base on
    __device__ __forceinline__ void fetch(E *lds, const E *base, int64_t step, int from, int limit, int D, int t) const {
        E *const to = lds + __builtin_amdgcn_readfirstlane(t >> 6) * 64 * CH;
        if (from <= 0 && limit >= ROWS && D == DP) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                to_lds(base + i * step, rows_at + (col ^ col_flip(i)) * (uint32_t)sizeof(E), to + i * NT * CH);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = col ^ col_flip(i);
                const int r = (int)row + i * STEP;
                const bool in = r >= from && r < limit && c < D;
                to_lds(base + i * step, in ? rows_at + c * (uint32_t)sizeof(E) : kOut, to + i * NT * CH);
            }
        }
    }

    // base: the tile's row 0, `limit` (at least 1) rows may be read
    __device__ __forceinline__ void load(E *lds, const E *base, int64_t stride, int from, int limit, int D, int t) const {
        if (PART && t >= ROWS * PER) return;  // whole waves
        if (VEC && near) return fetch(lds, base, STEP * stride, from, limit, D, t);
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            const int r = row + i * STEP, c = col ^ (mix<PER>(i * STEP) * CH);
            u32x4 v = load_piece<T, VEC>(base + (int64_t)min(r, limit - 1) * stride, c, D);
            if (r < from || r >= limit || (VEC && c >= D)) v = u32x4{0, 0, 0, 0};
            *(u32x4 *)(lds + (t + i * NT) * CH) = v;
        }
    }
    // The rows from row0 (a multiple of ROWS) on of a key head's queries; base: its
    // first query head, position 0
    __device__ __forceinline__ void load_rows(E *lds, const E *base, const AttnArgs &a, const Strides3 &st, int64_t row0,
                                              int from, int limit, int t) const {
        if (PART && t >= ROWS * PER) return;
        if (VEC && near)
            return fetch(lds, base + (int64_t)fdiv((uint32_t)row0, a.by_G) * st.l, (int64_t)fdiv(STEP, a.by_G) * st.l, from,
                         limit, a.D, t);
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            const int r = row + i * STEP, c = col ^ (mix<PER>(i * STEP) * CH);
            const RowAt at = row_at(a, row0 + min(r, limit - 1));
            u32x4 v = load_piece<T, VEC>(base + at.pos * st.l + at.head * st.h, c, a.D);
            if (r < from || r >= limit || (VEC && c >= a.D)) v = u32x4{0, 0, 0, 0};
            *(u32x4 *)(lds + (t + i * NT) * CH) = v;
        }
    }
};

// Waits until all but the latest N of the wave's loads into LDS have landed.
template <int N>
__device__ __forceinline__ void landed() {
    static_assert(N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4 << 14));
    asm volatile("" ::: "memory");
}

// Between the reads of the next product's operands and this product: the
// scheduler otherwise puts each read of LDS right before its use, and its
// latency is waited out every time.  (fp32's matrix instructions are long
// enough to cover it, and its operands too many to hold twice.)
template <typename T>
__device__ __forceinline__ void reads_first() {
    if constexpr (sizeof(typename T::T) == 2) __builtin_amdgcn_sched_barrier(0);
}

// acc[d] += A_d P for the 32-column slices d of the tile OFF elements on, A_d its
// rows K0 .. K0+31 read down the columns, P the two operands p0, p1.
template <typename T, int DP, int OFF = 0, int K0 = 0>
__device__ __forceinline__ void add_columns(f32x16 *acc, const typename T::T *tile, typename Tile<T>::Frag p0,
                                            typename Tile<T>::Frag p1, int lane) {
    using M = Tile<T>;
    constexpr int ND = DP / 32, N = ND > 1 && sizeof(typename T::T) == 2 ? 2 : 1;
#pragma unroll
    for (int d = 0; d < ND; d += N) {
        typename M::Frag f[N][2];
        M::template col_frags<DP, N, OFF, K0>(tile, d * 32, lane, f);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            acc[d + n] = M::mma(f[n][0], p0, acc[d + n]);
            acc[d + n] = M::mma(f[n][1], p1, acc[d + n]);
        }
    }
}

// The keys [lo, hi) that position i of batch b sees: always an interval.
// hi <= lo: none.
struct KeyRange {
    int lo, hi;
};
struct KeyRule {
    int len, start, causal, window;
    __device__ __forceinline__ KeyRange at(int i) const {
        const int p = start + i;
        int lo = 0, hi = len;
        if (causal) hi = min(hi, p + 1);
        if (window) {
            lo = max(0, p - window + 1);
            hi = min(hi, p + window);
        }
        return {lo, max(hi, 0)};
    }
};
__device__ __forceinline__ KeyRule key_rule(const AttnArgs &a, int b) {
    KeyRule r;
    r.len = a.kv_lens ? min(max(a.kv_lens[b], 0), a.Lk) : a.Lk;
    r.start = a.q_start ? min(max(a.q_start[b], -kMaxLen), kMaxLen) : a.Lk - a.Lq;
    r.causal = a.causal;
    r.window = a.window;
    return r;
}

// The maximum and the sum over the lanes l and l ^ 32.
__device__ __forceinline__ float half_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Workgroups are dealt to the 8 XCDs in turn; this gives each XCD a
// contiguous run of the logical order, so that the workgroups that read the
// same keys share an L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t n) {
    const uint32_t per = n / 8, extra = n % 8, x = id % 8, k = id / 8;
    return x * per + (x < extra ? x : extra) + k;
}

}  // namespace dc1d
