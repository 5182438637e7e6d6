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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kMaxLen = 1 << 29;  // limit of every length, and of window and |q_start|

// PADR: elements added to a tile row that is read along the row in 16-byte
// pieces (rows then start 16 bytes apart modulo the banks); PADC: to one that
// is read down the columns (four rows of 32 bytes at a time).
template <typename T>
struct Tile;

template <>
struct Tile<BF16> {
    using E = uint16_t;
    using Frag = bf16x8;
    static constexpr int CH = 8, PADR = 8, PADC = 16;

    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // eight consecutive elements of a row
    static __device__ __forceinline__ Frag row_frag(const E *p) { return *(const Frag *)p; }
    // Eight elements of column c0 + lane%32, rows k0 + 8*(j/4) + 4*(lane/32) +
    // j%4 (k0: a multiple of 16): each transposing read takes a 4 x 16 block
    // whose lane 4*i + c addresses elements 4c .. 4c+3 of row i, and gives
    // lane i of the 16 the block's column i.
    static __device__ __forceinline__ Frag col_frag(const E *tile, int pitch, int k0, int c0, int lane) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        const int i = lane & 15;
        const E *p = tile + (k0 + 4 * (lane >> 5) + (i >> 2)) * pitch + c0 + ((lane >> 4) & 1) * 16 + (i & 3) * 4;
        const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p);
        const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + 8 * pitch));
        typedef short i16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(Frag, (i16x8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
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
    static __device__ __forceinline__ void widen8(const E *p, float *f) {
        const u32x4 u = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

template <>
struct Tile<F32> {
    using E = float;
    using Frag = f32x8;
    static constexpr int CH = 4, PADR = 4, PADC = 4;

    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag row_frag(const E *p) {
        const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ Frag col_frag(const E *tile, int pitch, int k0, int c0, int lane) {
        const E *p = tile + (k0 + 4 * (lane >> 5)) * pitch + c0 + (lane & 31);
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = p[(8 * (j >> 2) + (j & 3)) * pitch];
        return f;
    }
    template <int S>
    static __device__ __forceinline__ Frag pack(const f32x16 &c) {
        return __builtin_shufflevector(c, c, 8 * S, 8 * S + 1, 8 * S + 2, 8 * S + 3, 8 * S + 4, 8 * S + 5, 8 * S + 6,
                                       8 * S + 7);
    }
    static __device__ __forceinline__ void store4(E *p, f32x4 v) { *(f32x4 *)p = v; }
    static __device__ __forceinline__ void widen8(const E *p, float *f) {
        const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    }
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

// A tile of ROWS rows of DP elements carried by NT threads, from global
// memory through registers into LDS.  Rows at and past `limit` and elements
// at and past D become zero, whatever memory holds there.
//
// Whole tiles of aligned rows are read at the tile's base, which the whole
// workgroup shares, plus 32-bit offsets that each thread forms once (`near`:
// they fit); other tiles form their addresses as they go.
template <typename T, int ROWS, int DP, int NT, bool VEC>
struct Stage {
    using E = typename T::T;
    static constexpr int CH = Tile<T>::CH, PER = DP / CH, N = (ROWS * PER + NT - 1) / NT;
    static_assert(ROWS * PER % NT == 0 || ROWS * PER < NT, "the tile divides among the threads, or needs only some");
    static constexpr int64_t kNear = 1 << 23;  // elements between rows: 64 rows of 4 bytes stay below 2^31
    u32x4 r[N];
    uint32_t off[N];
    bool near;

    // rows `stride` elements apart
    __device__ __forceinline__ void init(int64_t stride, int D, int t) {
        near = VEC && stride < kNear;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = t + i * NT, row = min(c / PER, ROWS - 1), col = c % PER * CH;
                off[i] = (uint32_t)(row * (uint32_t)stride + (col < D ? col : 0)) * sizeof(E);
            }
        }
    }
    // rows of a key head's queries: whole tiles start at the same head where
    // G divides their rows
    __device__ __forceinline__ void init_rows(const AttnArgs &a, const Strides3 &s, int t) {
        near = VEC && ROWS % a.G == 0 && s.l < kNear && s.h < kNear;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = t + i * NT, col = c % PER * CH;
                const RowAt at = row_at(a, min(c / PER, ROWS - 1));
                off[i] = ((uint32_t)at.pos * (uint32_t)s.l + (uint32_t)at.head * (uint32_t)s.h + (col < a.D ? col : 0)) * (uint32_t)sizeof(E);
            }
        }
    }
    // base: the tile's row 0 (limit >= 1 rows of it may be read)
    __device__ __forceinline__ void load(const E *base, int64_t stride, int limit, int D, int t) {
        if (near && limit >= ROWS) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = *(const u32x4 *)((const char *)base + off[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = t + i * NT, row = c / PER, col = c % PER * CH;
                r[i] = load_piece<T, VEC>(base + (int64_t)min(row, limit - 1) * stride, col, D);
            }
        }
    }
    // base: the key head's first query head, position 0; row0: a multiple of ROWS
    __device__ __forceinline__ void load_rows(const E *base, const AttnArgs &a, const Strides3 &s, int64_t row0, int t) {
        if (near && row0 + ROWS <= a.rows) {
            const char *const p = (const char *)(base + (int64_t)fdiv((uint32_t)row0, a.by_G) * s.l);
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = *(const u32x4 *)(p + off[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = t + i * NT, col = c % PER * CH;
                const RowAt at = row_at(a, row0 + c / PER < a.rows ? row0 + c / PER : a.rows - 1);
                r[i] = load_piece<T, VEC>(base + at.pos * s.l + at.head * s.h, col, a.D);
            }
        }
    }
    __device__ __forceinline__ void store(E *lds, int pitch, int limit, int D, int t) {
        if (limit < ROWS || D < DP) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = t + i * NT, row = c / PER, col = c % PER * CH;
                if (row >= limit || col >= D) r[i] = u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = t + i * NT;
            if (ROWS * PER < NT && c >= ROWS * PER) continue;
            *(u32x4 *)(lds + c / PER * pitch + c % PER * CH) = r[i];
        }
    }
};

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
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t n) {
    const int64_t per = n / 8, extra = n % 8, x = id % 8, k = id / 8;
    return x * per + (x < extra ? x : extra) + k;
}

}  // namespace dc1d
