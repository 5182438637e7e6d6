// k_rotary.hip -- rotary positions with up to four axes.
//
// Pair i of a head's R pairs turns by the angle of its axis' position:
//   (a, b) -> (a c - b s, a s + b c),  c, s = cos, sin [pos[b, l, axis(i)], i]
// (s negated for the inverse, which is also the gradient's rotation).  A pair
// is elements (i, R + i), or (2i, 2i + 1) where interleaved; elements past
// 2R are carried over.  Queries and keys go in one launch.
//
// Bound by HBM: every element is read and written once.  A thread takes VP
// neighbouring pairs (16-byte pieces of both halves) of one head; the tables'
// rows come from the L2 for every head anew.  Turning two or four heads a
// thread, the row read once for them, left fewer loads in flight and was
// slower: 8 x 4096 positions, 16 heads of 64, fp32: 49 us (5.5 TB/s) with one
// head, 62 with four.
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

// VP pairs of a head a thread.  A position has `units` pieces (of pairs, then
// of the carried elements) in each of its `heads` heads, the queries' and then
// the keys'; a workgroup takes `ppb` positions.
struct RotaryGrid {
    int units, heads, ppb;
    int64_t positions;
    FastDiv by_units, by_heads, by_L;
    int rows16;  // the tables' rows of VP entries are 16-byte aligned
};

template <typename T, int VP>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a, RotaryGrid gr) {
    using E = typename T::T;
    const int64_t n0 = (int64_t)blockIdx.x * gr.ppb;
    const int work = (int)min((int64_t)gr.ppb, gr.positions - n0) * gr.units * gr.heads;
    for (int w = threadIdx.x; w < work; w += 256) {
        const uint32_t rest = fdiv(w, gr.by_units), local = fdiv(rest, gr.by_heads);
        const int unit = w - (int)rest * gr.units;
        int h = (int)(rest - local * gr.heads);
        const uint32_t n = (uint32_t)n0 + local;
        const int b = (int)fdiv(n, gr.by_L), l = (int)n - b * a.L;
        const int which = h >= a.t[0].H;
        const RotaryTensor &t = a.t[which];
        if (which) h -= a.t[0].H;
        const E *const x = (const E *)t.x + b * t.xs.b + l * t.xs.l + h * t.xs.h;
        E *const y = (E *)t.y + b * t.ys.b + l * t.ys.l + h * t.ys.h;
        const int i = unit * VP;
        if (i >= a.R) {  // carried over
            const int d0 = 2 * a.R + (i - (a.R + VP - 1) / VP * VP) * 2;
            for (int d = d0; d < min(d0 + 2 * VP, a.D); ++d) y[d] = x[d];
            continue;
        }
        float u[2 * VP], v[2 * VP];
        Piece<T, VP>::load(x + (a.interleaved ? 2 * i : i), u);
        Piece<T, VP>::load(x + (a.interleaved ? 2 * i + VP : a.R + i), u + VP);
        const int *const pos = a.pos + b * a.pos_b + (int64_t)l * a.A;
        auto axis_of = [&](int j) { return (j >= a.first[1]) + (j >= a.first[2]) + (j >= a.first[3]); };
        auto row_of = [&](int axis) { return (int64_t)min(max(pos[axis], 0), a.P - 1) * a.R + i; };
        float c[VP], s[VP];
        const int axis = axis_of(i);
        if (VP > 1 && gr.rows16 && axis == axis_of(i + VP - 1)) {  // the piece lies in one section
            const int64_t at = row_of(axis);
#pragma unroll
            for (int j = 0; j < VP; j += 4) {
                Piece<F32, VP < 4 ? VP : 4>::load(a.cos + at + j, c + j);
                Piece<F32, VP < 4 ? VP : 4>::load(a.sin + at + j, s + j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                const int64_t at = row_of(axis_of(i + j)) + j;
                c[j] = a.cos[at];
                s[j] = a.sin[at];
            }
        }
#pragma unroll
        for (int j = 0; j < VP; ++j) s[j] *= a.sign;
        if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                v[2 * j] = u[2 * j] * c[j] - u[2 * j + 1] * s[j];
                v[2 * j + 1] = u[2 * j] * s[j] + u[2 * j + 1] * c[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                v[j] = u[j] * c[j] - u[VP + j] * s[j];
                v[VP + j] = u[j] * s[j] + u[VP + j] * c[j];
            }
        }
        Piece<T, VP>::store(y + (a.interleaved ? 2 * i : i), v);
        Piece<T, VP>::store(y + (a.interleaved ? 2 * i + VP : a.R + i), v + VP);
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
    RotaryGrid g;
    g.units = (a.R + VP - 1) / VP + (a.D - 2 * a.R + 2 * VP - 1) / (2 * VP);
    g.heads = a.t[0].H + a.t[1].H;
    g.positions = (int64_t)a.B * a.L;
    const int64_t per = (int64_t)g.units * g.heads;
    // one piece a thread, and few enough workgroups for one launch
    int64_t ppb = per >= 256 ? 1 : 256 / per;
    const int64_t least = (g.positions + (1 << 22) - 1) >> 22;
    if (ppb < least) ppb = least;
    g.ppb = (int)ppb;
    g.by_units = make_fastdiv((uint32_t)g.units);
    g.by_heads = make_fastdiv((uint32_t)g.heads);
    g.by_L = make_fastdiv((uint32_t)a.L);
    g.rows16 = a.R % 4 == 0 && ((uintptr_t)a.cos & 15) == 0 && ((uintptr_t)a.sin & 15) == 0;
    hipLaunchKernelGGL((k_rotary<T, VP>), dim3((uint32_t)((g.positions + ppb - 1) / ppb)), dim3(256), 0, stream, a, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream) {
    if (a.dtype == kF32) return pieces_ok<F32>(a, 4) ? launch<F32, 4>(a, stream) : launch<F32, 1>(a, stream);
    return pieces_ok<BF16>(a, 8) ? launch<BF16, 8>(a, stream) : launch<BF16, 1>(a, stream);
}

}  // namespace dc1d
