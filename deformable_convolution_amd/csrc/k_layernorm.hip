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
//
// Rows (L = 1): a wave, or the four waves of a workgroup, hold a row.
// Channels first (L > 1): a workgroup holds every channel of 128 bytes'
// worth of neighbouring positions, so that HBM is read in whole lines.
// The parameter gradients are summed per workgroup over all the positions
// that it visits, left in the workspace and added in workgroup order: no
// atomics, the same bits every time.
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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// The sum over WPR waves that share a row (all of a workgroup's when WPR >
// 1), the same value in every lane.  `slot` alternates between two arrays so
// that one barrier per sum is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red, int slot) {
    v = wave_sum(v);
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
// Four waves a workgroup; WPR of them to a row, NV 16-byte pieces to a lane
// (C <= WPR * 64 * NV * Vec::N, C a multiple of Vec::N, 16-byte rows).
template <typename T, int WPR, int NV>
__global__ __launch_bounds__(256) void k_ln_rows(LayerNormArgs a) {
    using V = Vec<T>;
    using E = typename T::T;
    __shared__ float red[2 * 4];
    const int lane = threadIdx.x % (64 * WPR);
    for (int64_t n0 = (int64_t)blockIdx.x * (4 / WPR); n0 < a.B; n0 += (int64_t)gridDim.x * (4 / WPR)) {
        const int64_t n = n0 + threadIdx.x / (64 * WPR);
        const bool on = n < a.B;
        const E *const x = (const E *)a.x + (on ? n : a.B - 1) * a.C;
        u32x4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 64 * WPR + lane) * V::N;
            raw[i] = *(const u32x4 *)(x + (c < a.C ? c : 0));
        }
        // the parameters are loaded before the sums are waited for
        u32x4 wr[NV], br[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 64 * WPR + lane) * V::N, cc = c < a.C ? c : 0;
            if (a.w) wr[i] = *(const u32x4 *)((const E *)a.w + cc);
            if (a.b) br[i] = *(const u32x4 *)((const E *)a.b + cc);
        }
        float f[NV][V::N], s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V::widen(raw[i], f[i]);
            if ((i * 64 * WPR + lane) * V::N < a.C)
#pragma unroll
                for (int e = 0; e < V::N; ++e) s += f[i][e];
        }
        const float mean = row_sum<WPR>(s, red, 0) / a.C;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * 64 * WPR + lane) * V::N < a.C;
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                f[i][e] -= mean;
                if (in) s += f[i][e] * f[i][e];
            }
        }
        const float rstd = rsqrtf(row_sum<WPR>(s, red, 1) / a.C + a.eps);
        if (!on) continue;
        E *const y = (E *)a.y + n * a.C;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 64 * WPR + lane) * V::N;
            if (c >= a.C) continue;
            float w[V::N], b[V::N];
            if (a.w) V::widen(wr[i], w);
            if (a.b) V::widen(br[i], b);
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
                f[i][e] *= rstd;
                if (a.w) f[i][e] *= w[e];
                if (a.b) f[i][e] += b[e];
            }
            *(u32x4 *)(y + c) = V::narrow(f[i]);
        }
        if (lane == 0) {
            if (a.mean) a.mean[n] = mean;
            if (a.rstd) a.rstd[n] = rstd;
        }
    }
}

// Rows of any length and alignment: a workgroup a row, read once for each
// sum and once more (from cache, for rows that fit it).
template <typename T>
__global__ __launch_bounds__(256) void k_ln_rows_any(LayerNormArgs a) {
    using E = typename T::T;
    __shared__ float red[2 * 4];
    for (int64_t n = blockIdx.x; n < a.B; n += gridDim.x) {
        const E *const x = (const E *)a.x + n * a.C;
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += 256) s += T::ld(x, c);
        const float mean = row_sum<4>(s, red, 0) / a.C;
        s = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float d = T::ld(x, c) - mean;
            s += d * d;
        }
        const float rstd = rsqrtf(row_sum<4>(s, red, 1) / a.C + a.eps);
        E *const y = (E *)a.y + n * a.C;
        for (int c = threadIdx.x; c < a.C; c += 256) {
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
// channels' parameter gradients in registers until the end.
template <typename T, int WPR, int NV>
__global__ __launch_bounds__(256) void k_ln_rows_bwd(LayerNormArgs a) {
    using V = Vec<T>;
    using E = typename T::T;
    constexpr int RPB = 4 / WPR;
    __shared__ float red[4 * 4];
    __shared__ float acc[RPB > 1 ? 64 * NV * V::N : 1];
    const int lane = threadIdx.x % (64 * WPR), grp = threadIdx.x / (64 * WPR);
    const bool params = a.gw || a.gb;
    float gw[NV][V::N] = {}, gb[NV][V::N] = {};
    u32x4 wr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 64 * WPR + lane) * V::N;
        if (a.w) wr[i] = *(const u32x4 *)((const E *)a.w + (c < a.C ? c : 0));
    }
    int slot = 0;
    for (int64_t n0 = (int64_t)blockIdx.x * RPB; n0 < a.B; n0 += (int64_t)gridDim.x * RPB) {
        const int64_t n = n0 + grp, m = n < a.B ? n : a.B - 1;
        const E *const x = (const E *)a.x + m * a.C, *const g = (const E *)a.g + m * a.C;
        const float mean = a.mean[m], rstd = a.rstd[m];
        u32x4 xr[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * 64 * WPR + lane) * V::N, cc = c < a.C ? c : 0;
            xr[i] = *(const u32x4 *)(x + cc);
            gr[i] = *(const u32x4 *)(g + cc);
        }
        float xh[NV][V::N], u[NV][V::N], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = n < a.B && (i * 64 * WPR + lane) * V::N < a.C;
            V::widen(xr[i], xh[i]);
            V::widen(gr[i], u[i]);
            float w[V::N];
            if (a.w) V::widen(wr[i], w);
#pragma unroll
            for (int e = 0; e < V::N; ++e) {
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
            s1 = row_sum<WPR>(s1, red, slot) / a.C;
            s2 = row_sum<WPR>(s2, red, slot + 1) / a.C;
            slot ^= 2;
            if (n < a.B) {
                E *const y = (E *)a.y + n * a.C;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * 64 * WPR + lane) * V::N;
                    if (c >= a.C) continue;
#pragma unroll
                    for (int e = 0; e < V::N; ++e) u[i][e] = rstd * (u[i][e] - s1 - xh[i][e] * s2);
                    *(u32x4 *)(y + c) = V::narrow(u[i]);
                }
            }
        }
    }
    if (!params) return;
    // the workgroup's sums: its row groups in order
    float *const pw = a.ws + (int64_t)blockIdx.x * 2 * a.C, *const pb = pw + a.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *const p = which ? pb : pw;
#pragma unroll
        for (int k = 0; k < RPB; ++k) {
            if constexpr (RPB > 1) __syncthreads();
            if (grp == k) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < V::N; ++e) {
                        const int j = (i * 64 * WPR + lane) * V::N + e;
                        float v = which ? gb[i][e] : gw[i][e];
                        if constexpr (RPB > 1) {
                            if (k > 0) v += acc[j];
                            if (k < RPB - 1) acc[j] = v;
                        }
                        if (k == RPB - 1 && j < a.C) p[j] = v;
                    }
            }
        }
    }
}

// Backward of rows of any length and alignment: a workgroup strides over the
// rows, its threads over the channels; the parameter sums are kept in the
// workgroup's part of the workspace.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_rows_bwd_any(LayerNormArgs a) {
    using E = typename T::T;
    __shared__ float red[4 * 4];
    const bool params = a.gw || a.gb;
    float *const pw = params ? a.ws + (int64_t)blockIdx.x * 2 * a.C : nullptr, *const pb = pw + a.C;
    int slot = 0;
    bool fresh = true;
    for (int64_t n = blockIdx.x; n < a.B; n += gridDim.x) {
        const E *const x = (const E *)a.x + n * a.C, *const g = (const E *)a.g + n * a.C;
        const float mean = a.mean[n], rstd = a.rstd[n];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.C; c += 256) {
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
        s1 = row_sum<4>(s1, red, slot) / a.C;
        s2 = row_sum<4>(s2, red, slot + 1) / a.C;
        slot ^= 2;
        E *const y = (E *)a.y + n * a.C;
        for (int c = threadIdx.x; c < a.C; c += 256) {
            const float xh = (T::ld(x, c) - mean) * rstd, gc = T::ld(g, c);
            const float u = a.w ? gc * T::ld((const E *)a.w, c) : gc;
            T::st(y, c, rstd * (u - s1 - xh * s2));
        }
    }
}

// ---- channels first ---------------------------------------------------------------
//
// A tile is TL neighbouring positions of one batch and all C channels.  A
// thread holds EPT neighbouring positions (16 bytes, or one element where
// rows are not aligned) of every RP-th channel: NP of them in registers, or,
// NP = 0, read again for each pass.
template <typename T, int EPT, int NT>
struct ColShape {
    static constexpr int TPR = EPT > 1 ? 8 : 64;  // threads across a tile's row
    static constexpr int TL = TPR * EPT, RP = NT / TPR;
};

template <typename T, int EPT>
__device__ __forceinline__ void col_load(const typename T::T *p, bool in, float *f) {
    if constexpr (EPT > 1) {
        if (in) {
            Vec<T>::widen(*(const u32x4 *)p, f);
        } else {
#pragma unroll
            for (int e = 0; e < EPT; ++e) f[e] = 0.0f;
        }
    } else {
        f[0] = in ? T::ld(p, 0) : 0.0f;
    }
}
template <typename T, int EPT>
__device__ __forceinline__ void col_store(typename T::T *p, const float *f) {
    if constexpr (EPT > 1)
        *(u32x4 *)p = Vec<T>::narrow(f);
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
#pragma unroll
            for (int w = 0; w < W; ++w) v += red[(k * W + w) * TL + tl * EPT + e];
            s[k][e] = v;
        }
}

template <typename T, int EPT, int NP, int NT>
__global__ __launch_bounds__(NT) void k_ln_cols(LayerNormArgs a) {
    using E = typename T::T;
    using S = ColShape<T, EPT, NT>;
    __shared__ float red[NT / 64 * S::TL];
    const int64_t tiles = (a.L + S::TL - 1) / S::TL;
    const int c0 = threadIdx.x / S::TPR;
    for (int64_t tile = blockIdx.x; tile < tiles * a.B; tile += gridDim.x) {
        const int64_t b = tile / tiles, l = tile % tiles * S::TL + threadIdx.x % S::TPR * EPT;
        const bool on = l < a.L;
        const int64_t at = b * a.C * a.L + (on ? l : 0);
        const E *const x = (const E *)a.x + at;
        E *const y = (E *)a.y + at;
        float f[NP > 0 ? NP : 1][EPT], s[1][EPT] = {};
        if constexpr (NP > 0) {
            u32x4 raw[NP];
            if constexpr (EPT > 1) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int c = c0 + i * S::RP;
                    raw[i] = *(const u32x4 *)(x + (int64_t)(c < a.C ? c : 0) * a.L);
                }
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = c0 + i * S::RP;
                if constexpr (EPT > 1) {
                    Vec<T>::widen(raw[i], f[i]);
                } else {
                    f[i][0] = T::ld(x, (int64_t)(c < a.C ? c : 0) * a.L);
                }
                if (c < a.C)
#pragma unroll
                    for (int e = 0; e < EPT; ++e) s[0][e] += f[i][e];
            }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT>(x + (int64_t)c * a.L, on, f[0]);
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[0][e] += f[0][e];
            }
        }
        col_sum<EPT, S::TPR, NT, 1>(s, red);
        float mean[EPT], rstd[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) mean[e] = s[0][e] / a.C, s[0][e] = 0.0f;
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    f[i][e] -= mean[e];
                    if (c0 + i * S::RP < a.C) s[0][e] += f[i][e] * f[i][e];
                }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT>(x + (int64_t)c * a.L, on, f[0]);
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[0][e] += (f[0][e] - mean[e]) * (f[0][e] - mean[e]);
            }
        }
        col_sum<EPT, S::TPR, NT, 1>(s, red);
#pragma unroll
        for (int e = 0; e < EPT; ++e) rstd[e] = rsqrtf(s[0][e] / a.C + a.eps);
        if (!on) continue;
        auto put = [&](int c, float *v, bool centred) {
            const float w = a.w ? T::ld((const E *)a.w, c) : 1.0f, bias = a.b ? T::ld((const E *)a.b, c) : 0.0f;
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                v[e] = (centred ? v[e] : v[e] - mean[e]) * rstd[e];
                if (a.w) v[e] *= w;
                if (a.b) v[e] += bias;
            }
            col_store<T, EPT>(y + (int64_t)c * a.L, v);
        };
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (c0 + i * S::RP < a.C) put(c0 + i * S::RP, f[i], true);
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT>(x + (int64_t)c * a.L, true, f[0]);
                put(c, f[0], false);
            }
        }
        if (c0 == 0) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                if (a.mean) a.mean[b * a.L + l + e] = mean[e];
                if (a.rstd) a.rstd[b * a.L + l + e] = rstd[e];
            }
        }
    }
}

// Backward, channels first.  Workgroups stride over the tiles.  With the
// channels in registers (NP > 0) so are their parameter sums; otherwise they
// are kept in the workgroup's part of the workspace, a thread row (TPR
// neighbouring lanes) owning its channels.
template <typename T, int EPT, int NP, int NT>
__global__ __launch_bounds__(NT) void k_ln_cols_bwd(LayerNormArgs a) {
    using E = typename T::T;
    using S = ColShape<T, EPT, NT>;
    constexpr int NR = NP > 0 ? NP : 1;
    __shared__ float red[2 * (NT / 64) * S::TL];
    const int64_t tiles = (a.L + S::TL - 1) / S::TL;
    const int c0 = threadIdx.x / S::TPR, tr = threadIdx.x % S::TPR;
    const bool params = a.gw || a.gb;
    float *const pw = params ? a.ws + (int64_t)blockIdx.x * 2 * a.C : nullptr, *const pb = pw + a.C;
    float gw[NR] = {}, gb[NR] = {};
    bool fresh = true;
    auto across = [](float v) {  // over the lanes of a thread row
#pragma unroll
        for (int d = 1; d < S::TPR; d <<= 1) v += __shfl_xor(v, d);
        return v;
    };
    for (int64_t tile = blockIdx.x; tile < tiles * a.B; tile += gridDim.x) {
        const int64_t b = tile / tiles, l = tile % tiles * S::TL + tr * EPT;
        const bool on = l < a.L;
        const int64_t at = b * a.C * a.L + (on ? l : 0);
        const E *const x = (const E *)a.x + at, *const g = (const E *)a.g + at;
        E *const y = (E *)a.y + at;
        float mean[EPT], rstd[EPT], s[2][EPT] = {};
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            mean[e] = a.mean[b * a.L + (on ? l + e : 0)];
            rstd[e] = a.rstd[b * a.L + (on ? l + e : 0)];
        }
        float xh[NR][EPT], u[NR][EPT];
        // the normalised x and the weighted gradient of channel c, and what they add to the sums
        auto take = [&](int c, bool in, float *xv, float *uv, float &w_sum, float &b_sum) {
            const float w = a.w ? T::ld((const E *)a.w, c) : 1.0f;
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                xv[e] = (xv[e] - mean[e]) * rstd[e];
                if (in) {
                    w_sum += uv[e] * xv[e];
                    b_sum += uv[e];
                }
                uv[e] *= w;
                if (in) {
                    s[0][e] += uv[e];
                    s[1][e] += uv[e] * xv[e];
                }
            }
        };
        if constexpr (NP > 0) {
            if constexpr (EPT > 1) {
                u32x4 xr[NP], gr[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int64_t c = c0 + i * S::RP < a.C ? c0 + i * S::RP : 0;
                    xr[i] = *(const u32x4 *)(x + c * a.L);
                    gr[i] = *(const u32x4 *)(g + c * a.L);
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    Vec<T>::widen(xr[i], xh[i]);
                    Vec<T>::widen(gr[i], u[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int64_t c = c0 + i * S::RP < a.C ? c0 + i * S::RP : 0;
                    xh[i][0] = T::ld(x, c * a.L);
                    u[i][0] = T::ld(g, c * a.L);
                }
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = c0 + i * S::RP;
                take(c < a.C ? c : 0, on && c < a.C, xh[i], u[i], gw[i], gb[i]);
            }
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT>(x + (int64_t)c * a.L, on, xh[0]);
                col_load<T, EPT>(g + (int64_t)c * a.L, on, u[0]);
                float w_sum = 0.0f, b_sum = 0.0f;
                take(c, on, xh[0], u[0], w_sum, b_sum);
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
        if (!on) continue;
        auto put = [&](int c, const float *xv, float *uv) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) uv[e] = rstd[e] * (uv[e] - s[0][e] / a.C - xv[e] * (s[1][e] / a.C));
            col_store<T, EPT>(y + (int64_t)c * a.L, uv);
        };
        if constexpr (NP > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (c0 + i * S::RP < a.C) put(c0 + i * S::RP, xh[i], u[i]);
        } else {
            for (int c = c0; c < a.C; c += S::RP) {
                col_load<T, EPT>(x + (int64_t)c * a.L, true, xh[0]);
                col_load<T, EPT>(g + (int64_t)c * a.L, true, u[0]);
                const float w = a.w ? T::ld((const E *)a.w, c) : 1.0f;
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    xh[0][e] = (xh[0][e] - mean[e]) * rstd[e];
                    u[0][e] *= w;
                }
                put(c, xh[0], u[0]);
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

// gw, gb: the workgroups' parts [parts][2][C] in order.  16 channels by 16
// runs of the parts a workgroup; the runs are added in order.
template <typename T>
__global__ __launch_bounds__(256) void k_ln_params(LayerNormArgs a, int parts) {
    using E = typename T::T;
    __shared__ float red[16][17];
    const int j = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int64_t n = (int64_t)blockIdx.x * 16 + j;  // of 2 C
    const int per = (parts + 15) / 16, p0 = run * per, p1 = min(p0 + per, parts);
    float s = 0.0f;
    if (n < 2 * (int64_t)a.C)
        for (int p = p0; p < p1; ++p) s += a.ws[(int64_t)p * 2 * a.C + n];
    red[run][j] = s;
    __syncthreads();
    if (run != 0 || n >= 2 * (int64_t)a.C) return;
    s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += red[r][j];
    if (n < a.C) {
        if (a.gw) T::st((E *)a.gw, n, s);
    } else if (a.gb) {
        T::st((E *)a.gb, n - a.C, s);
    }
}

// Workgroups of a forward call: the kernels stride over what exceeds these.
dim3 grid_of(int64_t blocks) { return dim3((uint32_t)(blocks < 1 << 20 ? blocks : 1 << 20)); }

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Which kernel serves the rows: pieces per lane and waves per row, 0: any.
struct RowChoice {
    int wpr, nv;
};
RowChoice choose_rows(int C, int per, bool vec) {
    if (!vec) return {0, 0};
    const int lanes = (C / per + 63) / 64;  // 16-byte pieces a lane of one wave
    if (lanes <= 1) return {1, 1};
    if (lanes <= 2) return {1, 2};
    if (lanes <= 4) return {1, 4};
    if (lanes <= 8) return {4, 2};
    if (lanes <= 16) return {4, 4};
    return {0, 0};
}

// Threads and channels held per thread, channels first; np 0: read again.
struct ColChoice {
    int nt, np;
};
ColChoice choose_cols(int C, bool vec) {
    if (vec) {
        if (C <= 256) return {256, 8};
        if (C <= 512) return {512, 8};
        if (C <= 1024) return {1024, 8};
        return {1024, 0};
    }
    if (C <= 128) return {1024, 8};
    if (C <= 512) return {1024, 32};
    return {1024, 0};
}

template <typename T>
bool vec_ok(const LayerNormArgs &a, bool backward) {
    const int64_t run = a.L == 1 ? a.C : a.L;
    bool ok = run % Vec<T>::N == 0 && aligned16(a.x) && aligned16(a.y);
    if (backward) ok = ok && aligned16(a.g);
    if (a.L == 1) ok = ok && aligned16(a.w) && aligned16(a.b);
    return ok;
}

template <typename T>
hipError_t forward_typed(const LayerNormArgs &a, hipStream_t st) {
    const bool vec = vec_ok<T>(a, false);
    if (a.L == 1) {
        const RowChoice c = choose_rows(a.C, Vec<T>::N, vec);
        const dim3 blk(256);
#define DC1D_ROWS(W, N) \
    hipLaunchKernelGGL((k_ln_rows<T, W, N>), grid_of((a.B + 4 / W - 1) / (4 / W)), blk, 0, st, a)
        if (c.wpr == 1 && c.nv == 1) DC1D_ROWS(1, 1);
        else if (c.wpr == 1 && c.nv == 2) DC1D_ROWS(1, 2);
        else if (c.wpr == 1) DC1D_ROWS(1, 4);
        else if (c.wpr == 4 && c.nv == 2) DC1D_ROWS(4, 2);
        else if (c.wpr == 4) DC1D_ROWS(4, 4);
        else hipLaunchKernelGGL((k_ln_rows_any<T>), grid_of(a.B), blk, 0, st, a);
#undef DC1D_ROWS
        return hipGetLastError();
    }
    const ColChoice c = choose_cols(a.C, vec);
#define DC1D_COLS(E, P, N)                                                                                             \
    hipLaunchKernelGGL((k_ln_cols<T, E, P, N>),                                                                        \
                       grid_of(a.B * ((a.L + ColShape<T, E, N>::TL - 1) / ColShape<T, E, N>::TL)), dim3(N), 0, \
                       st, a)
    constexpr int V = Vec<T>::N;
    if (vec) {
        if (c.nt == 256) DC1D_COLS(V, 8, 256);
        else if (c.nt == 512) DC1D_COLS(V, 8, 512);
        else if (c.np) DC1D_COLS(V, 8, 1024);
        else DC1D_COLS(V, 0, 1024);
    } else {
        if (c.np == 8) DC1D_COLS(1, 8, 1024);
        else if (c.np) DC1D_COLS(1, 32, 1024);
        else DC1D_COLS(1, 0, 1024);
    }
#undef DC1D_COLS
    return hipGetLastError();
}

// Workgroups of a backward call: few enough that the parts stay small next
// to x, enough to fill the GPU.
int64_t backward_blocks(int64_t B, int64_t L, int num_cus) {
    // the smallest unit that any of the kernels takes at a time: a row, or 32 positions
    const int64_t units = L == 1 ? B : B * ((L + 31) / 32);
    const int64_t most = (int64_t)num_cus * (L == 1 ? 4 : 2);
    return units < most ? units : most;
}

template <typename T>
hipError_t backward_typed(const LayerNormArgs &a, int num_cus, hipStream_t st) {
    if (a.B == 0 || a.L == 0) {  // no parts: the parameter gradients are zero
        if (a.gw || a.gb)
            hipLaunchKernelGGL((k_ln_params<T>), dim3((uint32_t)((2 * (int64_t)a.C + 15) / 16)), dim3(256), 0, st, a, 0);
        return hipGetLastError();
    }
    const bool vec = vec_ok<T>(a, true);
    const int64_t most = backward_blocks(a.B, a.L, num_cus);
    uint32_t blocks;
    if (a.L == 1) {
        const RowChoice c = choose_rows(a.C, Vec<T>::N, vec);
        const int rpb = c.wpr == 1 ? 4 : 1;
        const int64_t need = (a.B + rpb - 1) / rpb;
        blocks = (uint32_t)(need < most ? need : most);
        const dim3 blk(256);
#define DC1D_ROWS(W, N) hipLaunchKernelGGL((k_ln_rows_bwd<T, W, N>), dim3(blocks), blk, 0, st, a)
        if (c.wpr == 1 && c.nv == 1) DC1D_ROWS(1, 1);
        else if (c.wpr == 1 && c.nv == 2) DC1D_ROWS(1, 2);
        else if (c.wpr == 1) DC1D_ROWS(1, 4);
        else if (c.wpr == 4 && c.nv == 2) DC1D_ROWS(4, 2);
        else if (c.wpr == 4) DC1D_ROWS(4, 4);
        else hipLaunchKernelGGL((k_ln_rows_bwd_any<T>), dim3(blocks), blk, 0, st, a);
#undef DC1D_ROWS
    } else {
        const ColChoice c = choose_cols(a.C, vec);
        constexpr int V = Vec<T>::N;
        const int TL = vec ? 8 * V : 64;
        const int64_t need = a.B * ((a.L + TL - 1) / TL);
        blocks = (uint32_t)(need < most ? need : most);
#define DC1D_COLS(E, P, N) hipLaunchKernelGGL((k_ln_cols_bwd<T, E, P, N>), dim3(blocks), dim3(N), 0, st, a)
        if (vec) {
            if (c.nt == 256) DC1D_COLS(V, 8, 256);
            else if (c.nt == 512) DC1D_COLS(V, 8, 512);
            else if (c.np) DC1D_COLS(V, 8, 1024);
            else DC1D_COLS(V, 0, 1024);
        } else {
            if (c.np == 8) DC1D_COLS(1, 8, 1024);
            else DC1D_COLS(1, 0, 1024);
        }
#undef DC1D_COLS
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.gw || a.gb)) return e;
    hipLaunchKernelGGL((k_ln_params<T>), dim3((uint32_t)((2 * (int64_t)a.C + 15) / 16)), dim3(256), 0, st, a, (int)blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs &a, int, hipStream_t stream) {
    return a.dtype == kF32 ? forward_typed<F32>(a, stream) : forward_typed<BF16>(a, stream);
}

size_t layer_norm_backward_workspace(int64_t B, int C, int64_t L, int, bool want_params, int num_cus) {
    if (!want_params || B == 0 || L == 0) return 0;
    return (size_t)backward_blocks(B, L, num_cus) * 2 * C * sizeof(float);
}

hipError_t launch_layer_norm_backward(const LayerNormArgs &a, int num_cus, hipStream_t stream) {
    return a.dtype == kF32 ? backward_typed<F32>(a, num_cus, stream) : backward_typed<BF16>(a, num_cus, stream);
}

}  // namespace dc1d
