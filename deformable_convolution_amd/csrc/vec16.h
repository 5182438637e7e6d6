// vec16.h -- pieces of a row of either storage type: loads, stores, and the
// elements in 32 bits.
#pragma once

#include "attn_tile.h"

namespace dc1d {

template <typename T>
struct Vec;  // 16 bytes of elements
template <>
struct Vec<F32> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(u32x4 u, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(u[i]);
    }
    static __device__ __forceinline__ u32x4 narrow(const float *f) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};
template <>
struct Vec<BF16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(u32x4 u, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float *f) {
        f32x8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
        return __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8));  // nearest even
    }
};

// 16 bytes at an address that is a multiple of 16, or (ODD) of the element's
// size only: one load or store either way.
typedef u32x4 u32x4_odd __attribute__((aligned(2)));
template <bool ODD, typename E>
__device__ __forceinline__ u32x4 load16(const E *p) {
    if constexpr (ODD)
        return *(const u32x4_odd *)p;
    else
        return *(const u32x4 *)p;
}
// The elements from `skip` on of a piece.
template <typename T, bool ODD>
__device__ __forceinline__ void store16(typename T::T *p, const float *f, int skip) {
    if constexpr (ODD) {
        if (skip == 0) {
            *(u32x4_odd *)p = Vec<T>::narrow(f);
        } else {
#pragma unroll
            for (int e = 1; e < Vec<T>::N; ++e)
                if (e >= skip) T::st(p, e, f[e]);
        }
    } else {
        *(u32x4 *)p = Vec<T>::narrow(f);
    }
}

// Pieces of N neighbouring elements at any element's address, each one load and
// one store.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_odd __attribute__((aligned(2)));

template <typename T, int N>
struct Piece;
template <typename T>
struct Piece<T, 1> {
    using E = typename T::T;
    using Raw = uint32_t;  // the element's bits
    static __device__ __forceinline__ Raw load(const E *p) {
        if constexpr (sizeof(E) == 4)
            return __float_as_uint(*p);
        else
            return *p;
    }
    static __device__ __forceinline__ void widen(Raw r, float *f) { f[0] = __uint_as_float(sizeof(E) == 4 ? r : r << 16); }
    static __device__ __forceinline__ void store(E *p, const float *f) { T::st(p, 0, f[0]); }
};
template <>
struct Piece<F32, 4> {
    using E = float;
    using Raw = u32x4;
    static __device__ __forceinline__ Raw load(const E *p) { return load16<true>(p); }
    static __device__ __forceinline__ void widen(Raw r, float *f) { Vec<F32>::widen(r, f); }
    static __device__ __forceinline__ void store(E *p, const float *f) { *(u32x4_odd *)p = Vec<F32>::narrow(f); }
};
template <>
struct Piece<BF16, 8> {
    using E = uint16_t;
    using Raw = u32x4;
    static __device__ __forceinline__ Raw load(const E *p) { return load16<true>(p); }
    static __device__ __forceinline__ void widen(Raw r, float *f) { Vec<BF16>::widen(r, f); }
    static __device__ __forceinline__ void store(E *p, const float *f) { *(u32x4_odd *)p = Vec<BF16>::narrow(f); }
};
template <>
struct Piece<BF16, 4> {
    using E = uint16_t;
    using Raw = u32x2;
    static __device__ __forceinline__ Raw load(const E *p) { return *(const u32x2_odd *)p; }
    static __device__ __forceinline__ void widen(Raw r, float *f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[2 * i] = __uint_as_float(r[i] << 16);
            f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(E *p, const float *f) {
        *(u32x2_odd *)p = __builtin_bit_cast(u32x2, __builtin_convertvector(f32x4{f[0], f[1], f[2], f[3]}, bf16x4));
    }
};
// The elements from `skip` on of a piece: those before it are its neighbour's,
// which computes the same values from the same inputs, so that all of them may be
// stored unless the neighbour may have overwritten those inputs (in place).  One
// store of 16 bytes in place of up to seven: a row of 255 bf16 took twice as long.
template <typename T, int N>
__device__ __forceinline__ void store_own(typename T::T *p, const float *f, int skip, bool in_place = true) {
    if (skip == 0 || (!in_place && skip < N)) {
        Piece<T, N>::store(p, f);
    } else {
#pragma unroll
        for (int e = 1; e < N; ++e)
            if (e >= skip) T::st(p, e, f[e]);
    }
}

// Keeps what uses `v` behind what came before (and its packed form in registers
// till then): left to itself the compiler starts the exponentials of all of a
// thread's elements at once, or widens them once for several passes, and holds
// up to 100 registers more for them.
template <typename V>
__device__ __forceinline__ void hold(V &v) {
    asm volatile("" : "+v"(v));
}

// sigmoid(z) and 1 - sigmoid(z): the smaller one from exp(-|z|), the larger one as
// 1 minus it, so that neither cancels.  v_exp_f32 and v_rcp_f32 are off by an
// ulp, and the exponent's product with log2 e by 2^-24 |z|.
__device__ __forceinline__ void sigmoid_pair(float z, float &p, float &q) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e), s = e * __builtin_amdgcn_rcpf(1.0f + e), b = 1.0f - s;
    p = z < 0.0f ? s : b;
    q = z < 0.0f ? b : s;
}

}  // namespace dc1d
