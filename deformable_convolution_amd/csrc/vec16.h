// vec16.h -- 16-byte pieces of a row of either storage type: loads, stores, and
// the elements in 32 bits.
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

}  // namespace dc1d
