// k_rotary.hip -- rotary positions with up to four axes.
//
// Pair i of a head's R pairs turns by the angle of its axis' position:
//   (a, b) -> (a c - b s, a s + b c),  c, s = cos, sin [pos[b, l, axis(i)], i]
// (s negated for the inverse, which is also the gradient's rotation).  A pair
// is elements (i, R + i), or (2i, 2i + 1) where interleaved; elements past
// 2R are carried over.  Queries and keys go in one launch.
//
// Bound by HBM: every element is read and written once.  A thread takes VP
// neighbouring pairs of one position (16-byte pieces of both halves) and
// turns them in several heads, so that the table, which the L2 holds, is
// read once for those heads.
#include "attn_tile.h"

namespace dc1d {

namespace {

template <typename T, int N>
struct Piece {  // N neighbouring elements, moved as one access where N > 1
    static __device__ __forceinline__ void load(const typename T::T *p, float *f) {
        if constexpr (N == 1) {
            f[0] = T::ld(p, 0);
        } else {
            struct alignas(N * sizeof(typename T::T)) W {
                typename T::T e[N];
            };
            const W w = *(const W *)p;
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = T::ld(w.e, i);
        }
    }
    static __device__ __forceinline__ void store(typename T::T *p, const float *f) {
        if constexpr (N == 1) {
            T::st(p, 0, f[0]);
        } else {
            struct alignas(N * sizeof(typename T::T)) W {
                typename T::T e[N];
            };
            W w;
#pragma unroll
            for (int i = 0; i < N; ++i) T::st(w.e, i, f[i]);
            *(W *)p = w;
        }
    }
};

// VP pairs and HT heads a thread.  Threads run over [units] of a position
// (units: pair pieces, then pieces of the carried elements), head runs, and
// positions.
template <typename T, int VP, int HT>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a, int units, int runs, int64_t total) {
    using E = typename T::T;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int unit = (int)(id % units);
        const int64_t rest = id / units;
        int h0 = (int)(rest % runs) * HT;
        const int64_t n = rest / runs;
        const int b = (int)(n / a.L), l = (int)(n % a.L);
        // runs cover the queries' heads, then the keys'
        const int q_runs = (a.t[0].H + HT - 1) / HT;
        const int which = h0 >= q_runs * HT;
        const RotaryTensor &t = a.t[which];
        if (which) h0 -= q_runs * HT;
        const E *const x = (const E *)t.x + b * t.xs.b + l * t.xs.l;
        E *const y = (E *)t.y + b * t.ys.b + l * t.ys.l;
        const int i = unit * VP;
        if (i >= a.R) {  // carried over
            const int d0 = 2 * a.R + (i - (a.R + VP - 1) / VP * VP) * 2;
            for (int h = h0; h < min(h0 + HT, t.H); ++h)
                for (int d = d0; d < min(d0 + 2 * VP, a.D); ++d) y[h * t.ys.h + d] = x[h * t.xs.h + d];
            continue;
        }
        const int *const pos = a.pos + b * a.pos_b + (int64_t)l * a.A;
        float c[VP], s[VP];
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            const int axis = (i + j >= a.first[1]) + (i + j >= a.first[2]) + (i + j >= a.first[3]);
            const int p = min(max(pos[axis], 0), a.P - 1);
            c[j] = a.cos[(int64_t)p * a.R + i + j];
            s[j] = a.sin[(int64_t)p * a.R + i + j] * a.sign;
        }
        float u[HT][2 * VP];
#pragma unroll
        for (int k = 0; k < HT; ++k) {
            const E *const xh = x + min(h0 + k, t.H - 1) * t.xs.h;
            if (a.interleaved) {
                Piece<T, VP>::load(xh + 2 * i, u[k]);
                Piece<T, VP>::load(xh + 2 * i + VP, u[k] + VP);
            } else {
                Piece<T, VP>::load(xh + i, u[k]);
                Piece<T, VP>::load(xh + a.R + i, u[k] + VP);
            }
        }
#pragma unroll
        for (int k = 0; k < HT; ++k) {
            if (h0 + k >= t.H) break;
            E *const yh = y + (h0 + k) * t.ys.h;
            float v[2 * VP];
            if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < VP; ++j) {
                    v[2 * j] = u[k][2 * j] * c[j] - u[k][2 * j + 1] * s[j];
                    v[2 * j + 1] = u[k][2 * j] * s[j] + u[k][2 * j + 1] * c[j];
                }
                Piece<T, VP>::store(yh + 2 * i, v);
                Piece<T, VP>::store(yh + 2 * i + VP, v + VP);
            } else {
#pragma unroll
                for (int j = 0; j < VP; ++j) {
                    v[j] = u[k][j] * c[j] - u[k][VP + j] * s[j];
                    v[VP + j] = u[k][j] * s[j] + u[k][VP + j] * c[j];
                }
                Piece<T, VP>::store(yh + i, v);
                Piece<T, VP>::store(yh + a.R + i, v + VP);
            }
        }
    }
}

// Pieces of VP pairs stay inside their halves and are aligned.
template <typename T>
bool pieces_ok(const RotaryArgs &a, int VP) {
    const int64_t es = sizeof(typename T::T), n = VP;
    if (a.R % VP) return false;
    for (const RotaryTensor &t : a.t) {
        if (t.H == 0) continue;
        const int64_t s[6] = {t.xs.b, t.xs.l, t.xs.h, t.ys.b, t.ys.l, t.ys.h};
        for (int64_t v : s)
            if (v % n) return false;
        if ((uintptr_t)t.x % (n * es) || (uintptr_t)t.y % (n * es)) return false;
    }
    return true;
}

template <typename T, int VP>
hipError_t launch(const RotaryArgs &a, hipStream_t stream) {
    const int units = (a.R + VP - 1) / VP + (a.D - 2 * a.R + 2 * VP - 1) / (2 * VP);
    const int64_t n = (int64_t)a.B * a.L;
    auto runs_of = [&](int ht) { return (a.t[0].H + ht - 1) / ht + (a.t[1].H + ht - 1) / ht; };
    // one head a thread while that leaves the GPU unfilled (latency counts), else four
    const int64_t one = n * units * runs_of(1);
    if (one <= 256 * 256) {
        hipLaunchKernelGGL((k_rotary<T, VP, 1>), dim3((uint32_t)((one + 255) / 256)), dim3(256), 0, stream, a, units,
                           runs_of(1), one);
    } else {
        const int64_t total = n * units * runs_of(4);
        const int64_t blocks = (total + 255) / 256;
        hipLaunchKernelGGL((k_rotary<T, VP, 4>), dim3((uint32_t)(blocks < 1 << 20 ? blocks : 1 << 20)), dim3(256), 0, stream, a, units,
                           runs_of(4), total);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream) {
    if (a.dtype == kF32) return pieces_ok<F32>(a, 4) ? launch<F32, 4>(a, stream) : launch<F32, 1>(a, stream);
    return pieces_ok<BF16>(a, 8) ? launch<BF16, 8>(a, stream) : launch<BF16, 1>(a, stream);
}

}  // namespace dc1d
