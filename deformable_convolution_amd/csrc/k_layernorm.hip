// k_layernorm.hip -- layer norm over axis 1 of x [B][C][L] and its gradients.
//
//   mu = mean_c x,  r = 1 / sqrt(mean_c (x - mu)^2 + eps)
//   y  = (x - mu) r w + b
//   gx = r (u - mean_c u - xh mean_c(u xh)),  u = g w,  xh = (x - mu) r
//   gw = sum over (b, l) of g xh,  gb = sum over (b, l) of g
//
// All of it is bound by HBM: the forward has to read x and write y, the
// backward to read x and g and write gx, and each is done in one pass with
// the channels of a position held in registers between the sums (the
// variance is that of the centred values, so a large mean costs no digits).
// Rows of less than 16 bytes or of more than 2048 pieces of them, and more
// than 2048 channels first, are read again for each sum instead.
//
// Rows (L = 1): 8 to 512 lanes hold a row; several short ones share a wave.
// Channels first (L > 1): a workgroup holds every channel of 128 bytes' worth
// (fewer from 513 channels on) of neighbouring positions, so that HBM is read
// in whole lines.
// The parameter gradients are summed per workgroup over all the positions
// that it visits, left in the workspace and added in workgroup order: no
// atomics, the same bits every time.
#include <algorithm>
#include <type_traits>

#include "attn_tile.h"

namespace dc1d {

namespace {

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

// The sum over the LPR lanes that share a row (a part of a wave, or all of a
// workgroup), the same value in every one.  `slot` alternates between two
// arrays so that one barrier per sum is enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *red, int slot) {
    constexpr int WPR = LPR / 64;
#pragma unroll
    for (int d = 1; d < (LPR < 64 ? LPR : 64); d <<= 1) v += __shfl_xor(v, d);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[slot * WPR + (threadIdx.x >> 6)] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += red[slot * WPR + i];
    }
    return v;
}

// ---- rows ----------------------------------------------------------------------
//
// LPR lanes to a row, NV 16-byte pieces to a lane (C <= LPR * NV * Vec::N);
// four waves a workgroup, or the row's.  Where C is no multiple of a piece, or
// the rows are not aligned (ODD), the last piece is moved back to end with the
// row (C >= Vec::N), and the elements that it shares with the one before it
// are left to that one: 16 bytes a load at any address take what aligned ones
// take, element by element a row of 1022 bf16 took four times as long.
// 32768 x 1024 bf16: 22 us (6.0 TB/s); x 1022: 25 us; 131072 x 101 fp32: 18 us
// (5.8 TB/s); 4096 x 16384 bf16: 68 us (3.9 TB/s).
template <typename T>
constexpr int row_bwd_waves(int nv) {  // a SIMD: four floats of registers an element, and 16 bytes loaded for each tensor
    return nv * Vec<T>::N > 16 ? 2 : nv > 2 ? 3 : 4;
}
template <typename T, int LPR, int NV, bool ODD>
struct RowShape {
    static constexpr int NT = LPR > 256 ? LPR : 256, RPB = NT / LPR;
    int at[NV], skip[NV];  // where a piece is read, and how many of its elements are others' (Vec::N: it is not there)
    __device__ __forceinline__ RowShape(int lane, int C) {
        constexpr int N = Vec<T>::N;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * LPR + lane) * N;
            if constexpr (ODD) {
                at[i] = min(c, C - N);
                skip[i] = min(c - at[i], N);
            } else {
                at[i] = c < C ? c : 0;
                skip[i] = c < C ? 0 : N;
            }
        }
    }
    __device__ __forceinline__ bool own(int i, int e) const { return ODD ? e >= skip[i] : skip[i] == 0; }
};

template <typename T, int LPR, int NV, bool ODD>
__global__ __launch_bounds__((RowShape<T, LPR, NV, ODD>::NT)) void k_ln_rows(LayerNormArgs a) {
    using V = Vec<T>;
    using E = typename T::T;
    using S = RowShape<T, LPR, NV, ODD>;
    __shared__ float red[LPR > 64 ? 2 * (LPR / 64) : 1];
    const int lane = threadIdx.x % LPR;
    const S sh(lane, a.C);
    for (int64_t n0 = (int64_t)blockIdx.x * S::RPB; n0 < a.B; n0 += (int64_t)gridDim.x * S::RPB) {
        const int64_t n = n0 + threadIdx.x / LPR;
        const bool on = n < a.B;
        const E *const x = (const E *)a.x + (on ? n : a.B - 1) * a.C;
        u32x4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = load16<ODD>(x + sh.at[i]);
        // the parameters are loaded before the sums are waited for
        u32x4 wr[NV], br[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (a.w) wr[i] = load16<ODD>((const E *)a.w + sh.at[i]);
            if (a.b) br[i] = load16<ODD>((const E *)a.b + sh.at[i]);
        }
        float f[NV][V::N], s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V::widen(raw[i], f[i]);
#pragma unroll
            for (int e = 0; e < V::N; ++e)
                if (sh.own(i, e)) s += f[i][e];
        }
        const float mean = row_sum<LPR>(s, red, 0) * a.inv_c;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                f[i][e] -= mean;
                if (sh.own(i, e)) s += f[i][e] * f[i][e];
            }
        }
        const float rstd = rsqrtf(row_sum<LPR>(s, red, 1) * a.inv_c + a.eps);
        if (!on) continue;
        E *const y = (E *)a.y + n * a.C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (sh.skip[i] == V::N) continue;
            float w[V::N], b[V::N];
            if (a.w) V::widen(wr[i], w);
            if (a.b) V::widen(br[i], b);
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                f[i][e] *= rstd;
                if (a.w) f[i][e] *= w[e];
                if (a.b) f[i][e] += b[e];
            }
            store16<T, ODD>(y + sh.at[i], f[i], sh.skip[i]);
        }
        if (lane == 0) {
            if (a.mean) a.mean[n] = mean;
            if (a.rstd) a.rstd[n] = rstd;
        }
    }
}

// Rows shorter than a piece (a wave a row) or longer than k_ln_rows holds (16
// waves): read once for each sum and once more, from cache where a row fits it.
// 4096 x 32768 fp32: 495 us (2.2 TB/s), gradients 998 us.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_ln_rows_any(LayerNormArgs a) {
    using E = typename T::T;
        __shared__ float red[2 * (NT / 64)];
    for (int64_t n = blockIdx.x; n < a.B; n += gridDim.x) {
        const E *const x = (const E *)a.x + n * a.C;
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += NT) s += T::ld(x, c);
        const float mean = row_sum<NT>(s, red, 0) * a.inv_c;
        s = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += NT) {
            const float d = T::ld(x, c) - mean;
            s += d * d;
        }
        const float rstd = rsqrtf(row_sum<NT>(s, red, 1) * a.inv_c + a.eps);
        E *const y = (E *)a.y + n * a.C;
        for (int c = threadIdx.x; c < a.C; c += NT) {
            float v = (T::ld(x, c) - mean) * rstd;
            if (a.w) v *= T::ld((const E *)a.w, c);
            if (a.b) v += T::ld((const E *)a.b, c);
            T::st(y, c, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[n] = mean;
            if (a.rstd) a.rstd[n] = rstd;
        }
    }
}

// Backward of rows.  Workgroups stride over the rows; a lane keeps its
// channels' parameter gradients in registers until the end.  32768 x 1024 bf16:
// 42 us with the parameters' sums (4.7 TB/s); x 1022: 47 us.
template <typename T, int LPR, int NV, bool ODD>
__global__ __launch_bounds__((RowShape<T, LPR, NV, ODD>::NT), row_bwd_waves<T>(NV)) void k_ln_rows_bwd(LayerNormArgs a) {
    using V = Vec<T>;
    using E = typename T::T;
    using S = RowShape<T, LPR, NV, ODD>;
    constexpr int RPB = S::RPB;
    __shared__ float red[LPR > 64 ? 4 * (LPR / 64) : 1];
    __shared__ float acc[RPB > 1 ? LPR * NV * V::N : 1];
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const bool params = a.gw || a.gb;
    const S sh(lane, a.C);
    float gw[NV][V::N] = {}, gb[NV][V::N] = {};
    u32x4 wr[NV] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (a.w) wr[i] = load16<ODD>((const E *)a.w + sh.at[i]);
    int slot = 0;
    for (int64_t n0 = (int64_t)blockIdx.x * RPB; n0 < a.B; n0 += (int64_t)gridDim.x * RPB) {
        const int64_t n = n0 + grp, m = n < a.B ? n : a.B - 1;
        const E *const x = (const E *)a.x + m * a.C, *const g = (const E *)a.g + m * a.C;
        const float mean = a.mean[m], rstd = a.rstd[m];
        u32x4 xr[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xr[i] = load16<ODD>(x + sh.at[i]);
            gr[i] = load16<ODD>(g + sh.at[i]);
        }
        float xh[NV][V::N], u[NV][V::N], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V::widen(xr[i], xh[i]);
            V::widen(gr[i], u[i]);
            float w[V::N];
            asm volatile("" : "+v"(wr[i]));  // stays packed between rows, in half the registers
            if (a.w) V::widen(wr[i], w);
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                const bool in = n < a.B && sh.own(i, e);
                xh[i][e] = (xh[i][e] - mean) * rstd;
                if (in) {
                    gw[i][e] += u[i][e] * xh[i][e];
                    gb[i][e] += u[i][e];
                }
                if (a.w) u[i][e] *= w[e];
                if (in) {
                    s1 += u[i][e];
                    s2 += u[i][e] * xh[i][e];
                }
            }
        }
        if (a.y) {
            s1 = row_sum<LPR>(s1, red, slot) * a.inv_c;
            s2 = row_sum<LPR>(s2, red, slot + 1) * a.inv_c;
            slot ^= 2;
            if (n < a.B) {
                E *const y = (E *)a.y + n * a.C;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (sh.skip[i] == V::N) continue;
#pragma unroll
                    for (int e = 0; e < V::N; ++e) u[i][e] = rstd * (u[i][e] - s1 - xh[i][e] * s2);
                    store16<T, ODD>(y + sh.at[i], u[i], sh.skip[i]);
                }
            }
        }
    }
    if (!params) return;
    // the workgroup's sums: over the row groups of a wave, then the waves in order
    constexpr int GROUPS = LPR < 64 ? 4 : RPB;
    const int turn = LPR < 64 ? threadIdx.x / 64 : grp;
    const bool first = LPR >= 64 || threadIdx.x % 64 < LPR;
    float *const pw = a.ws + (int64_t)blockIdx.x * 2 * a.C, *const pb = pw + a.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *const p = which ? pb : pw;
        float v[NV][V::N];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                v[i][e] = which ? gb[i][e] : gw[i][e];
#pragma unroll
                for (int d = LPR; d < 64; d <<= 1) v[i][e] += __shfl_xor(v[i][e], d);
            }
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
            if constexpr (GROUPS > 1) __syncthreads();
            if (turn != k || !first) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V::N; ++e) {
                    if constexpr (GROUPS > 1) {
                        float &sum = acc[(i * LPR + lane) * V::N + e];
                        if (k > 0) v[i][e] += sum;
                        if (k < GROUPS - 1) sum = v[i][e];
                    }
                    if (k == GROUPS - 1 && sh.own(i, e)) p[sh.at[i] + e] = v[i][e];
                }
        }
    }
}

// Backward of rows shorter than a piece or longer than k_ln_rows_bwd holds: a
// workgroup strides over the rows, its threads over the channels; the
// parameter sums are kept in the workgroup's part of the workspace.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_ln_rows_bwd_any(LayerNormArgs a) {
    using E = typename T::T;
        __shared__ float red[4 * (NT / 64)];
    const bool params = a.gw || a.gb;
    float *const pw = params ? a.ws + (int64_t)blockIdx.x * 2 * a.C : nullptr, *const pb = pw + a.C;
    int slot = 0;
    bool fresh = true;
    for (int64_t n = blockIdx.x; n < a.B; n += gridDim.x) {
        const E *const x = (const E *)a.x + n * a.C, *const g = (const E *)a.g + n * a.C;
        const float mean = a.mean[n], rstd = a.rstd[n];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += NT) {
            const float xh = (T::ld(x, c) - mean) * rstd, gc = T::ld(g, c);
            if (params) {
                pw[c] = (fresh ? 0.0f : pw[c]) + gc * xh;
                pb[c] = (fresh ? 0.0f : pb[c]) + gc;
            }
            const float u = a.w ? gc * T::ld((const E *)a.w, c) : gc;
            s1 += u;
            s2 += u * xh;
        }
        fresh = false;
        if (!a.y) continue;
        s1 = row_sum<NT>(s1, red, slot) * a.inv_c;
        s2 = row_sum<NT>(s2, red, slot + 1) * a.inv_c;
        slot ^= 2;
        E *const y = (E *)a.y + n * a.C;
        for (int c = threadIdx.x; c < a.C; c += NT) {
            const float xh = (T::ld(x, c) - mean) * rstd, gc = T::ld(g, c);
            const float u = a.w ? gc * T::ld((const E *)a.w, c) : gc;
            T::st(y, c, rstd * (u - s1 - xh * s2));
        }
    }
}

// ---- channels first ---------------------------------------------------------------
//
// A tile is TL neighbouring positions of one batch and all C channels.  A
// thread holds EPT neighbouring positions (16 bytes, or one element where a
// batch has fewer) of every RP-th channel: NP of them in registers, or,
// NP = 0, read again for each pass.  Where rows are not aligned, or end inside
// a piece (ODD), the last pieces are moved back to end with the row; what a
// thread then reads of positions before its own it neither adds nor stores.  TPR threads stand across a tile's row:
// 8 (whole 128-byte lines), fewer where C channels would not fit otherwise.
// Neighbouring tiles go to one XCD: where rows are not whole lines they share
// the lines at their edges.  8 x 256 x 16384 bf16: 36 us (3.7 TB/s) over
// inputs of more than the last-level cache, 31 where two alternate in it, x
// 16383: 32 us; 16 x 512 x 4092 fp32: 64 us (4.2 TB/s) either way; with NP = 0,
// 4 x 4096 x 1024 fp32: 50 us (2.7 TB/s).  A piece past C is loaded all the same
// (from the tile's first row): C = 300 issues the loads of 512, 1280 those of
// 2048 (64 x 300 x 1001 bf16: 29 us, 2.7 TB/s; 1 x 1280 x 4383 fp32: 21, 2.2).
template <int EPT, int TPR_, int NT>
struct ColShape {
    static constexpr int TPR = TPR_, TL = TPR * EPT, RP = NT / TPR;
};

// Where this thread's positions of a tile (its first: l0) are read.  Every
// address is inside the tensor, also of threads that have no position (!on).
template <int EPT, bool ODD>
struct ColPlace {
    int64_t base;  // the workgroup's first position
    int at, skip;  // the thread's, from base; how many of them are other threads'
    bool on;
    __device__ __forceinline__ ColPlace(int64_t l0, int tl, int64_t L) {
        on = l0 + tl < L;
        if constexpr (ODD) {
            base = min(l0, L - EPT);
            at = (int)(min(l0 + tl, L - EPT) - base);
            skip = (int)(l0 + tl - base) - at;
        } else {
            base = l0;
            at = on ? tl : 0;
            skip = 0;
        }
    }
    __device__ __forceinline__ bool own(int e) const { return !ODD || e >= skip; }
};

template <typename T, int EPT, bool ODD>
__device__ __forceinline__ void col_load(const typename T::T *p, float *f) {
    if constexpr (EPT > 1)
        Vec<T>::widen(load16<ODD>(p), f);
    else
        f[0] = T::ld(p, 0);
}
template <typename T, int EPT, bool ODD>
__device__ __forceinline__ void col_store(typename T::T *p, const float *f, int skip) {
    if constexpr (EPT > 1)
        store16<T, ODD>(p, f, skip);
    else
        T::st(p, 0, f[0]);
}

// Sums over the channels, per position: over a wave's threads of the same
// position, then over the waves in wave order.
template <int EPT, int TPR, int NT, int K>
__device__ __forceinline__ void col_sum(float (*s)[EPT], float *red) {
    constexpr int W = NT / 64, TL = TPR * EPT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tl = threadIdx.x % TPR;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EPT; ++e)
#pragma unroll
            for (int d = TPR; d < 64; d <<= 1) s[k][e] += __shfl_xor(s[k][e], d);
    __syncthreads();  // the array's last readers are done
    if (lane < TPR) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < EPT; ++e) red[(k * W + wave) * TL + tl * EPT + e] = s[k][e];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            float v = 0.0f;
#pragma unroll 2
            for (int w = 0; w < W; ++w) v += red[(k * W + w) * TL + tl * EPT + e];
            s[k][e] = v;
        }
}

// The pieces of a tile that a thread holds: channels c0 + i RP.  Each is read
// at a base that the whole workgroup shares plus this thread's 32-bit offset;
// a channel past C reads row i RP in its place and is left out of the sums.
template <typename T, int EPT, bool ODD>
struct ColPiece {
    using E = typename T::T;
    using Raw = typename std::conditional<(EPT > 1), u32x4, E>::type;
    static __device__ __forceinline__ Raw load(const E *base, uint32_t off) {
        const E *const p = (const E *)((const char *)base + off);
        if constexpr (EPT > 1)
            return load16<ODD>(p);
        else
            return *p;
    }
    // Between two uses of a held piece: the compiler otherwise keeps the
    // widened and centred values of the first use for the second, in more
    // registers than the pieces take.
    static __device__ __forceinline__ void again(Raw &r) {
        if constexpr (EPT > 1) {
            asm volatile("" : "+v"(r));
        } else {
            uint32_t v;
            if constexpr (sizeof(E) == 4)
                v = __float_as_uint(r);
            else
                v = r;
            asm volatile("" : "+v"(v));
            if constexpr (sizeof(E) == 4)
                r = __uint_as_float(v);
            else
                r = (E)v;
        }
    }
    static __device__ __forceinline__ void widen(Raw r, float *f) {
        if constexpr (EPT > 1)
            Vec<T>::widen(r, f);
        else
            f[0] = T::ld(&r, 0);
    }
};

template <typename T, int EPT, int TPR, int NP, int NT, bool ODD>
__global__ __launch_bounds__(NT, 1024 / NT) void k_ln_cols(LayerNormArgs a) {
    using E = typename T::T;
    using S = ColShape<EPT, TPR, NT>;
    using P = ColPiece<T, EPT, ODD>;
    __shared__ float red[NT / 64 * S::TL];
    const uint32_t tiles = (uint32_t)((a.L + S::TL - 1) / S::TL);  // of a batch; all positions are fewer than 2^31
    const int c0 = threadIdx.x / S::TPR;
    for (int64_t tile = xcd_order(blockIdx.x, gridDim.x); tile < tiles * a.B; tile += gridDim.x) {
        const int64_t b = (uint32_t)tile / tiles, l0 = (int64_t)((uint32_t)tile % tiles) * S::TL;
        const ColPlace<EPT, ODD> place(l0, threadIdx.x % S::TPR * EPT, a.L);
        const E *const x = (const E *)a.x + b * a.C * a.L + place.base;
        E *const y = (E *)a.y + b * a.C * a.L + place.base;
        const uint32_t row0 = place.at * sizeof(E), off = row0 + (uint32_t)c0 * (uint32_t)a.L * sizeof(E);
        typename P::Raw raw[NP > 0 ? NP : 1];
        float f[EPT], s[1][EPT] = {};
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int ci = i * S::RP < a.C ? i * S::RP : 0;
                raw[i] = P::load(x + (int64_t)ci * a.L, c0 + ci < a.C ? off : row0);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                P::widen(raw[i], f);
                if (c0 + i * S::RP < a.C)
#pragma unroll
                    for (int e = 0; e < EPT; ++e) s[0][e] += f[e];
            }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT, ODD>(x + (int64_t)c * a.L + place.at, f);
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[0][e] += f[e];
            }
        }
        col_sum<EPT, S::TPR, NT, 1>(s, red);
        float mean[EPT], rstd[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) mean[e] = s[0][e] * a.inv_c, s[0][e] = 0.0f;
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                P::again(raw[i]);
                P::widen(raw[i], f);
                if (c0 + i * S::RP < a.C)
#pragma unroll
                    for (int e = 0; e < EPT; ++e) s[0][e] += (f[e] - mean[e]) * (f[e] - mean[e]);
            }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT, ODD>(x + (int64_t)c * a.L + place.at, f);
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[0][e] += (f[e] - mean[e]) * (f[e] - mean[e]);
            }
        }
        col_sum<EPT, S::TPR, NT, 1>(s, red);
#pragma unroll
        for (int e = 0; e < EPT; ++e) rstd[e] = rsqrtf(s[0][e] * a.inv_c + a.eps);
        if (!place.on) continue;
        auto put = [&](int c) {
            const float w = a.w ? T::ld((const E *)a.w, c) : 1.0f, bias = a.b ? T::ld((const E *)a.b, c) : 0.0f;
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                f[e] = (f[e] - mean[e]) * rstd[e];
                if (a.w) f[e] *= w;
                if (a.b) f[e] += bias;
            }
            col_store<T, EPT, ODD>(y + (int64_t)c * a.L + place.at, f, place.skip);
        };
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                P::again(raw[i]);
                P::widen(raw[i], f);
                if (c0 + i * S::RP < a.C) put(c0 + i * S::RP);
            }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT, ODD>(x + (int64_t)c * a.L + place.at, f);
                put(c);
            }
        }
        if (c0 == 0) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                if (!place.own(e)) continue;
                if (a.mean) a.mean[b * a.L + place.base + place.at + e] = mean[e];
                if (a.rstd) a.rstd[b * a.L + place.base + place.at + e] = rstd[e];
            }
        }
    }
}

// Backward, channels first.  Workgroups, as many as fit the GPU at once,
// stride over the tiles, and a tile's pieces are on their way from HBM while
// the one before it is worked on.  With the channels in registers (NP > 0) so
// are their parameter sums; otherwise they are kept in the workgroup's part
// of the workspace, a thread row (TPR neighbouring lanes) owning its channels.
// 16 x 512 x 4092 fp32: 95 us (4.2 TB/s), x 4091: 99 us; 8 x 256 x 16384 bf16:
// 54 us (3.7 TB/s); with NP = 0, 4 x 4096 x 1024 fp32: 110 us.
template <typename T, int EPT, int TPR, int NP, int NT, bool ODD>
__global__ __launch_bounds__(NT, (NT < 512 ? 512 / NT : 1)) void k_ln_cols_bwd(LayerNormArgs a) {
    using E = typename T::T;
    using S = ColShape<EPT, TPR, NT>;
    using P = ColPiece<T, EPT, ODD>;
    constexpr int NR = NP > 0 ? NP : 1;
    __shared__ float red[2 * (NT / 64) * S::TL];
    const uint32_t tiles = (uint32_t)((a.L + S::TL - 1) / S::TL);  // of a batch; all positions are fewer than 2^31
    const int c0 = threadIdx.x / S::TPR, tr = threadIdx.x % S::TPR, tl = tr * EPT;
    const bool params = a.gw || a.gb;
    float *const pw = a.ws + (params ? (int64_t)blockIdx.x * 2 * a.C : 0), *const pb = pw + a.C;
    float gw[NR] = {}, gb[NR] = {};
    bool fresh = true;
    auto across = [](float v) {  // over the lanes of a thread row
#pragma unroll
        for (int d = 1; d < S::TPR; d <<= 1) v += __shfl_xor(v, d);
        return v;
    };
    struct Held {
        typename P::Raw x[NR], g[NR];
        float mean[EPT], rstd[EPT];
    };
    auto fetch = [&](int64_t tile, Held &h) {
        const int64_t b = (uint32_t)tile / tiles, l0 = (int64_t)((uint32_t)tile % tiles) * S::TL;
        const ColPlace<EPT, ODD> place(l0, tl, a.L);
        if constexpr (NP > 0) {
            const int64_t at = b * a.C * a.L + place.base;
            const E *const x = (const E *)a.x + at, *const g = (const E *)a.g + at;
            const uint32_t row0 = place.at * sizeof(E), off = row0 + (uint32_t)c0 * (uint32_t)a.L * sizeof(E);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int ci = i * S::RP < a.C ? i * S::RP : 0;
                const uint32_t o = c0 + ci < a.C ? off : row0;
                h.x[i] = P::load(x + (int64_t)ci * a.L, o);
                h.g[i] = P::load(g + (int64_t)ci * a.L, o);
            }
        }
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            h.mean[e] = a.mean[b * a.L + place.base + place.at + e];
            h.rstd[e] = a.rstd[b * a.L + place.base + place.at + e];
        }
    };
    const int64_t all = tiles * a.B;
    // held, not read in the loop: loads return in order, and one issued after
    // the next tile's would wait for all of it
    float wv[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) wv[i] = NP > 0 && a.w && c0 + i * S::RP < a.C ? T::ld((const E *)a.w, c0 + i * S::RP) : 1.0f;
    Held next;
    const int64_t tile0 = xcd_order(blockIdx.x, gridDim.x);
    fetch(tile0, next);  // there are at least as many tiles as workgroups
    for (int64_t tile = tile0; tile < all; tile += gridDim.x) {
        Held h = next;
        if (tile + gridDim.x < all) fetch(tile + gridDim.x, next);
        const int64_t b = (uint32_t)tile / tiles, l0 = (int64_t)((uint32_t)tile % tiles) * S::TL;
        const ColPlace<EPT, ODD> place(l0, tl, a.L);
        const int64_t at = b * a.C * a.L + place.base + place.at;
        float s[2][EPT] = {}, xh[EPT], u[EPT];
        // what a channel of weight w adds to the sums over the channels and to its parameters' gradients
        auto take = [&](float w, float &w_sum, float &b_sum) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                if (!place.own(e)) continue;
                xh[e] = (xh[e] - h.mean[e]) * h.rstd[e];
                w_sum += u[e] * xh[e];
                b_sum += u[e];
                u[e] *= w;
                s[0][e] += u[e];
                s[1][e] += u[e] * xh[e];
            }
        };
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = c0 + i * S::RP;
                P::widen(h.x[i], xh);
                P::widen(h.g[i], u);
                if (place.on && c < a.C) take(wv[i], gw[i], gb[i]);
            }
        } else {
            const E *const x = (const E *)a.x + at, *const g = (const E *)a.g + at;
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT, ODD>(x + (int64_t)c * a.L, xh);
                col_load<T, EPT, ODD>(g + (int64_t)c * a.L, u);
                float w_sum = 0.0f, b_sum = 0.0f;
                if (place.on) take(a.w ? T::ld((const E *)a.w, c) : 1.0f, w_sum, b_sum);
                if (params) {
                    w_sum = across(w_sum);
                    b_sum = across(b_sum);
                    if (tr == 0) {
                        pw[c] = (fresh ? 0.0f : pw[c]) + w_sum;
                        pb[c] = (fresh ? 0.0f : pb[c]) + b_sum;
                    }
                }
            }
        }
        fresh = false;
        if (!a.y) continue;
        col_sum<EPT, S::TPR, NT, 2>(s, red);
        if (!place.on) continue;
        E *const y = (E *)a.y + at;
#pragma unroll
        for (int e = 0; e < EPT; ++e) s[0][e] *= a.inv_c, s[1][e] *= a.inv_c;
        auto put = [&](int c, float w) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                xh[e] = (xh[e] - h.mean[e]) * h.rstd[e];
                u[e] = h.rstd[e] * (u[e] * w - s[0][e] - xh[e] * s[1][e]);
            }
            col_store<T, EPT, ODD>(y + (int64_t)c * a.L, u, place.skip);
        };
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                P::again(h.x[i]);
                P::again(h.g[i]);
                P::widen(h.x[i], xh);
                P::widen(h.g[i], u);
                if (c0 + i * S::RP < a.C) put(c0 + i * S::RP, wv[i]);
            }
        } else {
            const E *const x = (const E *)a.x + at, *const g = (const E *)a.g + at;
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT, ODD>(x + (int64_t)c * a.L, xh);
                col_load<T, EPT, ODD>(g + (int64_t)c * a.L, u);
                put(c, a.w ? T::ld((const E *)a.w, c) : 1.0f);
            }
        }
    }
    if constexpr (NP > 0) {
        if (!params) return;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = c0 + i * S::RP;
            const float w_sum = across(gw[i]), b_sum = across(gb[i]);
            if (tr == 0 && c < a.C) {
                pw[c] = w_sum;
                pb[c] = b_sum;
            }
        }
    }
}

// gw, gb: the workgroups' parts [parts][2][C] in order.  16 channels by 64
// runs of the parts a workgroup, so that few loads follow one another; the
// runs are added in order.  1024 parts of 1024 channels: 4.9 us.
template <typename T>
__global__ __launch_bounds__(1024) void k_ln_params(LayerNormArgs a, int parts) {
    using E = typename T::T;
    __shared__ float red[64][17];
    const int j = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int64_t n = (int64_t)blockIdx.x * 16 + j, all = 2 * (int64_t)a.C;
    const int per = (parts + 63) / 64, p0 = run * per, p1 = min(p0 + per, parts);
    float s = 0.0f;
    if (n < all) {
#pragma unroll 8
        for (int p = p0; p < p1; ++p) s += a.ws[p * all + n];
    }
    red[run][j] = s;
    __syncthreads();
    if (run != 0 || n >= all) return;
    s = 0.0f;
#pragma unroll
    for (int r = 0; r < 64; ++r) s += red[r][j];
    if (n < a.C) {
        if (a.gw) T::st((E *)a.gw, n, s);
    } else if (a.gb) {
        T::st((E *)a.gb, n - a.C, s);
    }
}

// Workgroups of a forward call: the kernels stride over what exceeds these.
dim3 grid_of(int64_t blocks) { return dim3((uint32_t)(blocks < 1 << 20 ? blocks : 1 << 20)); }

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Which kernel serves the rows: lanes per row and pieces per lane.  nv = 0:
// from memory for each pass, as rows of less than a piece or of more than
// eight waves hold are.  Rows of few pieces share a wave: 131072 x 101 bf16
// takes 50 us with a wave to a row and 15 with 16 lanes (gradients 69 and 25).
struct RowChoice {
    int lpr, nv;
};
RowChoice choose_rows(int C, int per) {
    if (C < per) return {64, 0};
    const int pieces = (C + per - 1) / per;
    if (pieces <= 8) return {8, 1};
    if (pieces <= 16) return {16, 1};
    if (pieces <= 32) return {32, 1};
    if (pieces <= 64) return {64, 1};
    if (pieces <= 128) return {64, 2};
    if (pieces <= 256) return {64, 4};
    if (pieces <= 512) return {256, 2};
    if (pieces <= 1024) return {256, 4};
    if (pieces <= 2048) return {512, 4};
    return {1024, 0};
}

// Which kernel serves channels first: threads across a row, channels held per
// thread (0: read again), threads.
struct ColChoice {
    int tpr, np, nt;
};
ColChoice choose_cols(int C, int64_t L, int per) {
    if (L < per) return C > 1024 ? ColChoice{8, 0, 1024} : ColChoice{8, 16, 512};
    // a thread's first channel lies past 32-bit byte offsets: as many as 256
    // thread rows of four bytes an element
    const bool far = L >= 1 << 22;
    if (far || C > 2048) return {8, 0, 1024};
    if (C <= 256) return {8, 8, 256};
    return {C <= 512 ? 8 : C <= 1024 ? 4 : 2, 8, 512};
}

// Whether every 16-byte piece is aligned and inside its row.
template <typename T>
bool whole(const LayerNormArgs &a, bool backward) {
    const int64_t run = a.L == 1 ? a.C : a.L;
    bool ok = run % Vec<T>::N == 0 && aligned16(a.x) && aligned16(a.y);
    if (backward) ok = ok && aligned16(a.g);
    if (a.L == 1) ok = ok && aligned16(a.w) && aligned16(a.b);
    return ok;
}

// Every combination that choose_rows and choose_cols give.
#define DC1D_ROWS_SWITCH(ODD)                                  \
    if (c.nv == 0 && c.lpr == 64) DC1D_ANY(64);                \
    else if (c.nv == 0) DC1D_ANY(1024);                        \
    else if (c.lpr == 8) DC1D_ROWS(8, 1, ODD);                 \
    else if (c.lpr == 16) DC1D_ROWS(16, 1, ODD);               \
    else if (c.lpr == 32) DC1D_ROWS(32, 1, ODD);               \
    else if (c.lpr == 64 && c.nv == 1) DC1D_ROWS(64, 1, ODD);  \
    else if (c.lpr == 64 && c.nv == 2) DC1D_ROWS(64, 2, ODD);  \
    else if (c.lpr == 64) DC1D_ROWS(64, 4, ODD);               \
    else if (c.lpr == 256 && c.nv == 2) DC1D_ROWS(256, 2, ODD);\
    else if (c.lpr == 256) DC1D_ROWS(256, 4, ODD);             \
    else DC1D_ROWS(512, 4, ODD);
#define DC1D_COLS_SWITCH(V, ODD)                             \
    if (c.np == 0) DC1D_COLS(V, 8, 0, 1024, ODD);            \
    else if (c.nt == 256) DC1D_COLS(V, 8, 8, 256, ODD);      \
    else if (c.tpr == 8) DC1D_COLS(V, 8, 8, 512, ODD);       \
    else if (c.tpr == 4) DC1D_COLS(V, 4, 8, 512, ODD);       \
    else DC1D_COLS(V, 2, 8, 512, ODD);

template <typename T>
hipError_t forward_typed(const LayerNormArgs &a, hipStream_t st) {
    const bool even = whole<T>(a, false);
    if (a.L == 1) {
        const RowChoice c = choose_rows(a.C, Vec<T>::N);
#define DC1D_ROWS(R, N, O)                                                                                       \
    hipLaunchKernelGGL((k_ln_rows<T, R, N, O>),                                                                    \
                       grid_of((a.B + RowShape<T, R, N, O>::RPB - 1) / RowShape<T, R, N, O>::RPB),                 \
                       dim3((RowShape<T, R, N, O>::NT)), 0, st, a)
#define DC1D_ANY(N) hipLaunchKernelGGL((k_ln_rows_any<T, N>), grid_of(a.B), dim3(N), 0, st, a)
        if (even) {
            DC1D_ROWS_SWITCH(false)
        } else {
            DC1D_ROWS_SWITCH(true)
        }
#undef DC1D_ROWS
#undef DC1D_ANY
        return hipGetLastError();
    }
    constexpr int V = Vec<T>::N;
    const ColChoice c = choose_cols(a.C, a.L, V);
#define DC1D_COLS(E, R, P, N, O)                                                                                     \
    hipLaunchKernelGGL((k_ln_cols<T, E, R, P, N, O>), grid_of(a.B * ((a.L + R * E - 1) / (R * E))), dim3(N), 0, st, a)
    if (a.L < V) {
        if (c.np == 0) DC1D_COLS(1, 8, 0, 1024, false);
        else DC1D_COLS(1, 8, 16, 512, false);
    } else if (even) {
        DC1D_COLS_SWITCH(V, false)
    } else {
        DC1D_COLS_SWITCH(V, true)
    }
#undef DC1D_COLS
    return hipGetLastError();
}

// Workgroups of a backward call, and so parts of the parameter gradients: no
// more than fit the GPU at once.
template <typename T>
uint32_t backward_blocks(int64_t B, int C, int64_t L, int num_cus) {
    int64_t need, fit;
    if (L == 1) {
        const RowChoice c = choose_rows(C, Vec<T>::N);
        const int rpb = c.nv > 0 && c.lpr < 256 ? 256 / c.lpr : 1, nt = c.nv > 0 && c.lpr < 256 ? 256 : c.lpr;
        need = (B + rpb - 1) / rpb;
        fit = (int64_t)num_cus * std::min(4, (c.nv > 0 ? row_bwd_waves<T>(c.nv) : 8) * 256 / nt);
    } else {
        constexpr int V = Vec<T>::N;
        const ColChoice c = choose_cols(C, L, V);
        const int TL = c.tpr * (L < V ? 1 : V);
        need = B * ((L + TL - 1) / TL);
        fit = (int64_t)num_cus * (c.nt < 512 ? 512 / c.nt : 1);
    }
    return (uint32_t)(need < fit ? need : fit);
}

template <typename T>
hipError_t backward_typed(const LayerNormArgs &a, int num_cus, hipStream_t st) {
    if (a.B == 0 || a.L == 0) {  // no parts: the parameter gradients are zero
        if (a.gw || a.gb)
            hipLaunchKernelGGL((k_ln_params<T>), dim3((uint32_t)((2 * (int64_t)a.C + 15) / 16)), dim3(1024), 0, st, a, 0);
        return hipGetLastError();
    }
    const bool even = whole<T>(a, true);
    const uint32_t blocks = backward_blocks<T>(a.B, a.C, a.L, num_cus);
    if (a.L == 1) {
        const RowChoice c = choose_rows(a.C, Vec<T>::N);
#define DC1D_ROWS(R, N, O) \
    hipLaunchKernelGGL((k_ln_rows_bwd<T, R, N, O>), dim3(blocks), dim3((RowShape<T, R, N, O>::NT)), 0, st, a)
#define DC1D_ANY(N) hipLaunchKernelGGL((k_ln_rows_bwd_any<T, N>), dim3(blocks), dim3(N), 0, st, a)
        if (even) {
            DC1D_ROWS_SWITCH(false)
        } else {
            DC1D_ROWS_SWITCH(true)
        }
#undef DC1D_ROWS
#undef DC1D_ANY
    } else {
        constexpr int V = Vec<T>::N;
        const ColChoice c = choose_cols(a.C, a.L, V);
#define DC1D_COLS(E, R, P, N, O) hipLaunchKernelGGL((k_ln_cols_bwd<T, E, R, P, N, O>), dim3(blocks), dim3(N), 0, st, a)
        if (a.L < V) {
            if (c.np == 0) DC1D_COLS(1, 8, 0, 1024, false);
            else DC1D_COLS(1, 8, 16, 512, false);
        } else if (even) {
            DC1D_COLS_SWITCH(V, false)
        } else {
            DC1D_COLS_SWITCH(V, true)
        }
#undef DC1D_COLS
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.gw || a.gb)) return e;
    hipLaunchKernelGGL((k_ln_params<T>), dim3((uint32_t)((2 * (int64_t)a.C + 15) / 16)), dim3(1024), 0, st, a, (int)blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs &a, int, hipStream_t stream) {
    return a.dtype == kF32 ? forward_typed<F32>(a, stream) : forward_typed<BF16>(a, stream);
}

size_t layer_norm_backward_workspace(int64_t B, int C, int64_t L, int dtype, bool want_params, int num_cus) {
    if (!want_params || B == 0 || L == 0) return 0;
    const uint32_t parts = dtype == kF32 ? backward_blocks<F32>(B, C, L, num_cus) : backward_blocks<BF16>(B, C, L, num_cus);
    return (size_t)parts * 2 * C * sizeof(float);
}

hipError_t launch_layer_norm_backward(const LayerNormArgs &a, int num_cus, hipStream_t stream) {
    return a.dtype == kF32 ? backward_typed<F32>(a, num_cus, stream) : backward_typed<BF16>(a, num_cus, stream);
}

}  // namespace dc1d
