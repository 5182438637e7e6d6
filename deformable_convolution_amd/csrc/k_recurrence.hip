// k_recurrence.hip -- a gated linear recurrence along the positions and its
// gradients, every channel on its own:
//
//   h_s = a_s h_{s-1} + u_s,  a = sigmoid(gate),  u = x or (1 - a) x
//   r_s = g_s + a_{s+1} r_{s+1},  gx = r or r (1 - a),
//   ggate = r (h_{s-1} or h_{s-1} - x) a (1 - a),  gstate = a_0 r_0
//
// s counts the positions in the recurrence's order.  Both are scans of affine
// maps h -> A h + H, which are joined as (A, H) then (A', H') = (A A', A' H + H').
// Bound by HBM: the forward has to read x and gate and write y, the backward to
// read x, gate and g and write two gradients.
//
// A workgroup is 16 slots of a few positions by 16 pieces of N channels, so that
// rows are read in runs of 16 pieces; a tile is the slots' positions.  A slot's
// positions stay in registers: their map is formed, the slots' maps are joined
// over the wave's lanes and the waves, and the states follow.
#include <algorithm>
#include <type_traits>

#include "vec16.h"

namespace dc1d {

namespace {

constexpr int kLanes = 16, kSlots = 16, kThreads = kLanes * kSlots;
constexpr int kWaveSlots = 64 / kLanes, kWaves = kThreads / 64;
constexpr int kPer = 8, kPerBack = 4;  // positions of a slot
constexpr int kTile = kSlots * kPer, kTileBack = kSlots * kPerBack;
static_assert(kStateEvery % kPer == 0, "a kept state stands ahead of a slot");
static_assert(kTileBack % kStateEvery == 0, "a tile of the backward pass starts at a kept state");

struct RecPlan {
    int slabs, segs, seg_tiles;
    size_t ws_bytes;
};

int rec_piece(int C) { return C >= 4 ? 4 : 1; }

// The positions in segments of whole tiles, a workgroup each, until there are
// four workgroups for every CU; with one segment a workgroup walks through all of them.
RecPlan plan_recurrence(int B, int L, int C, int tile, int num_cus) {
    RecPlan p;
    const int P = (C + rec_piece(C) - 1) / rec_piece(C);
    p.slabs = (P + kLanes - 1) / kLanes;
    const int64_t rows = (int64_t)B * p.slabs, tiles = std::max(1, (L + tile - 1) / tile);
    const int64_t want = rows > 0 ? (4ll * num_cus + rows - 1) / rows : 1;
    p.segs = (int)std::max<int64_t>(1, std::min({want, tiles, (int64_t)64}));
    p.seg_tiles = (int)((tiles + p.segs - 1) / p.segs);
    p.segs = (int)((tiles + p.seg_tiles - 1) / p.seg_tiles);
    p.ws_bytes = p.segs > 1 ? (size_t)B * p.segs * C * sizeof(float2) : 0;
    return p;
}

// A thread's channels and its sequence.
template <int N>
struct Lane {
    int b, n, slot, at, skip, seg;  // n: positions within the length
    bool on;
    __device__ __forceinline__ Lane(const RecurrenceArgs &a, const RecPlan &p, int64_t job) {
        const int slab = (int)(job % p.slabs);
        const int64_t q = job / p.slabs;
        seg = (int)(q % p.segs);
        b = (int)(q / p.segs);
        n = a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
        slot = threadIdx.x / kLanes;
        const int c = (slab * kLanes + threadIdx.x % kLanes) * N;
        on = c < a.C;
        at = on ? min(c, a.C - N) : 0;
        skip = on ? c - at : N;
    }
    __device__ __forceinline__ bool own(int e) const { return e >= skip; }
};

// A thread's channels of a tensor along the recurrence: position s at p + s * step.
template <typename T>
struct Walk {
    typename T::T *p;
    int64_t step;
    template <int N>
    __device__ __forceinline__ Walk(const void *t, Strides2 st, const RecurrenceArgs &a, const Lane<N> &l) {
        p = (typename T::T *)t + l.b * st.b + l.at + (a.reverse ? (int64_t)(l.n - 1) * st.l : 0);
        step = a.reverse ? -st.l : st.l;
    }
};

template <int N>
struct Map {  // h -> A h + H
    float A[N], H[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < N; ++e) A[e] = 1.0f, H[e] = 0.0f;
    }
    // `first`, then this one
    __device__ __forceinline__ void after(const Map &first) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            H[e] = fmaf(A[e], first.H[e], H[e]);
            A[e] *= first.A[e];
        }
    }
    __device__ __forceinline__ void apply(float *h) const {
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = fmaf(A[e], h[e], H[e]);
    }
};

// The maps of the slots ahead of a thread's in its tile (of those behind it
// where BACK), and the whole tile's.  `ends` holds a map for every wave and lane;
// the caller's barriers keep one tile's from the next.
template <int N, bool BACK>
__device__ __forceinline__ void join_slots(Map<N> own, Map<N> &ahead, Map<N> &tile, Map<N> (*ends)[kLanes]) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, slot = lane / kLanes, p = lane % kLanes;
    const int place = BACK ? kWaveSlots - 1 - slot : slot;
#pragma unroll
    for (int d = 1; d < kWaveSlots; d <<= 1) {
        const int from = (lane + (BACK ? d : -d) * kLanes) & 63;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float A = __shfl(own.A[e], from), H = __shfl(own.H[e], from);
            own.H[e] = fmaf(own.A[e], place >= d ? H : 0.0f, own.H[e]);
            own.A[e] *= place >= d ? A : 1.0f;
        }
    }
    if (place == kWaveSlots - 1) ends[w][p] = own;
    const int from = (lane + (BACK ? 1 : -1) * kLanes) & 63;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float A = __shfl(own.A[e], from), H = __shfl(own.H[e], from);
        ahead.A[e] = place > 0 ? A : 1.0f;
        ahead.H[e] = place > 0 ? H : 0.0f;
    }
    __syncthreads();
    tile.clear();
    Map<N> before = tile;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const int wave = BACK ? kWaves - 1 - i : i;
        if (wave == w) before = tile;  // the same for all of a wave
        Map<N> o = ends[wave][p];
        o.after(tile);
        tile = o;
    }
    ahead.after(before);
}

// The rows of a slot's positions, PER of them from s0 on; the last one within
// the length in place of those past it where FULL is false.
template <typename T, int N, int PER>
struct Rows {
    typename Piece<T, N>::Raw r[PER];
    template <bool FULL>
    __device__ __forceinline__ void load(const Walk<T> &w, int s0, int n) {
        const typename T::T *const p = w.p + (int64_t)s0 * w.step;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            r[k] = Piece<T, N>::load(FULL ? p + k * w.step : w.p + (int64_t)min(s0 + k, n - 1) * w.step);
    }
};

// sigmoid(gate) and 1 - it, (1, 0) past the length.
template <typename T, int N, int PER>
struct Gates {
    float a[PER][N], q[PER][N];
    __device__ __forceinline__ Gates(const Rows<T, N, PER> &g) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            float z[N];
            Piece<T, N>::widen(g.r[k], z);
#pragma unroll
            for (int e = 0; e < N; ++e) sigmoid_pair(z[e], a[k][e], q[k][e]);
        }
    }
    __device__ __forceinline__ void end(int s0, int n) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (s0 + k >= n)
#pragma unroll
                for (int e = 0; e < N; ++e) a[k][e] = 1.0f, q[k][e] = 0.0f;
    }
};

// f in 32 bits, 0 past the length.
template <typename T, int N, int PER>
__device__ __forceinline__ void widen_rows(const Rows<T, N, PER> &r, float (*f)[N]) {
#pragma unroll
    for (int k = 0; k < PER; ++k) Piece<T, N>::widen(r.r[k], f[k]);
}
template <int N, int PER>
__device__ __forceinline__ void end_rows(float (*f)[N], int s0, int n) {
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (s0 + k >= n)
#pragma unroll
            for (int e = 0; e < N; ++e) f[k][e] = 0.0f;
}

template <int N, int PER>
__device__ __forceinline__ Map<N> map_of(const float (*a)[N], const float (*u)[N]) {
    Map<N> m;
#pragma unroll
    for (int e = 0; e < N; ++e) m.A[e] = a[0][e], m.H[e] = u[0][e];
#pragma unroll
    for (int k = 1; k < PER; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            m.H[e] = fmaf(a[k][e], m.H[e], u[k][e]);
            m.A[e] *= a[k][e];
        }
    return m;
}

// Rows past the length, in a segment's part of the positions, become 0.
template <typename T, int N>
__device__ __forceinline__ void clear_rows(void *t, Strides2 st, const Lane<N> &l, int from, int to) {
    if (!t || !l.on) return;
    const float zero[N] = {};
    typename T::T *const p = (typename T::T *)t + l.b * st.b + l.at;
    for (int s = from + l.slot; s < to; s += kSlots) store_own<T, N>(p + s * st.l, zero, l.skip);
}

// Walks the tiles of a segment within the length: next(i, FULL) starts the loads
// of tile i, tile(i, FULL) uses what was loaded last.  A tile's loads are in
// flight while the one before it is worked on.
template <int TILE, bool BACK, typename Next, typename Work>
__device__ __forceinline__ void walk(int first, int past, int n, Next next, Work work) {
    past = min(past, (n + TILE - 1) / TILE);
    const int tiles = past - first;
    for (int j = 0; j < tiles; ++j) {
        const int i = BACK ? past - 1 - j : first + j;
        work(i, j, [&] {
            if (j + 1 < tiles) next(BACK ? i - 1 : i + 1);
        });
    }
}

// The map of every segment but the last: [b][seg][C].  In the last one's place
// stands the first state, which the next kernel may overwrite with the last.
template <typename T, int N, bool BLEND>
__global__ __launch_bounds__(kThreads) void k_rec_segments(RecurrenceArgs a, RecPlan p, float2 *out, int64_t jobs) {
    __shared__ Map<N> ends[2][kWaves][kLanes];
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const Walk<T> xw(a.x, a.xs, a, t), gw(a.gate, a.gates, a, t);
        Map<N> all;
        all.clear();
        if (t.seg == p.segs - 1) {
            if (a.state)
#pragma unroll
                for (int e = 0; e < N; ++e) all.H[e] = a.state[(int64_t)t.b * a.C + t.at + e];
        } else {
            const int first = t.seg * p.seg_tiles, past = first + p.seg_tiles;
            Rows<T, N, kPer> xr, gr;
            auto next = [&](int i) {
                const int s0 = i * kTile + t.slot * kPer;
                if ((i + 1) * kTile <= t.n) {
                    xr.template load<true>(xw, s0, t.n);
                    gr.template load<true>(gw, s0, t.n);
                } else {
                    xr.template load<false>(xw, s0, t.n);
                    gr.template load<false>(gw, s0, t.n);
                }
            };
            if (first * kTile < t.n) next(first);
            walk<kTile, false>(first, past, t.n, next, [&](int i, int j, auto then) {
                const int s0 = i * kTile + t.slot * kPer;
                Gates<T, N, kPer> v(gr);
                float u[kPer][N];
                widen_rows<T, N, kPer>(xr, u);
                then();
                if (BLEND)
#pragma unroll
                    for (int k = 0; k < kPer; ++k)
#pragma unroll
                        for (int e = 0; e < N; ++e) u[k][e] *= v.q[k][e];
                if ((i + 1) * kTile > t.n) {
                    v.end(s0, t.n);
                    end_rows<N, kPer>(u, s0, t.n);
                }
                Map<N> ahead, tile;
                join_slots<N, false>(map_of<N, kPer>(v.a, u), ahead, tile, ends[j & 1]);
                tile.after(all);
                all = tile;
            });
        }
        __syncthreads();
        if (t.slot == 0) {
            float2 *const o = out + ((int64_t)t.b * p.segs + t.seg) * a.C + t.at;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (t.own(e)) o[e] = make_float2(all.A[e], all.H[e]);
        }
    }
}

// The state ahead of a segment: the one that a call starts from, and the maps of
// the segments before it.
template <int N>
__device__ __forceinline__ void carry_in(const RecurrenceArgs &a, const RecPlan &p, const Lane<N> &t, const float *start,
                                         const float2 *maps, int from, int to, int step, float *h) {
    if (p.segs > 1) {  // from the place of the map that nobody needs
        const float2 *const m = maps + ((int64_t)t.b * p.segs + (step > 0 ? p.segs - 1 : 0)) * a.C + t.at;
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = m[e].y;
    } else if (start) {
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = start[(int64_t)t.b * a.C + t.at + e];
    }
    for (int i = from; i != to; i += step) {
        const float2 *const m = maps + ((int64_t)t.b * p.segs + i) * a.C + t.at;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float2 v = m[e];
            h[e] = fmaf(v.x, h[e], v.y);
        }
    }
}

template <typename T, int N, bool BLEND>
__global__ __launch_bounds__(kThreads) void k_recurrence(RecurrenceArgs a, RecPlan p, const float2 *maps, int64_t jobs) {
    using E = typename T::T;
    __shared__ Map<N> ends[2][kWaves][kLanes];
    const int kept = (a.L + kStateEvery - 1) / kStateEvery;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const Walk<T> xw(a.x, a.xs, a, t), gw(a.gate, a.gates, a, t), yw(a.y, a.ys, a, t);
        const int64_t bc = (int64_t)t.b * a.C + t.at;
        const int first = t.seg * p.seg_tiles, past = first + p.seg_tiles;
        Rows<T, N, kPer> xr, gr;
        auto next = [&](int i) {
            const int s0 = i * kTile + t.slot * kPer;
            if ((i + 1) * kTile <= t.n) {
                xr.template load<true>(xw, s0, t.n);
                gr.template load<true>(gw, s0, t.n);
            } else {
                xr.template load<false>(xw, s0, t.n);
                gr.template load<false>(gw, s0, t.n);
            }
        };
        if (first * kTile < t.n) next(first);
        float h0[N] = {};
        carry_in<N>(a, p, t, a.state, maps, 0, t.seg, 1, h0);
        auto keep = [&](int s, const float *h) {
            float *const o = a.states + ((int64_t)t.b * kept + s / kStateEvery) * a.C + t.at;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (t.own(e)) o[e] = h[e];
        };
        walk<kTile, false>(first, past, t.n, next, [&](int i, int j, auto then) {
            const int s0 = i * kTile + t.slot * kPer;
            const bool full = (i + 1) * kTile <= t.n;
            Gates<T, N, kPer> v(gr);
            float u[kPer][N];
            widen_rows<T, N, kPer>(xr, u);
            then();
            if (BLEND)
#pragma unroll
                for (int k = 0; k < kPer; ++k)
#pragma unroll
                    for (int e = 0; e < N; ++e) u[k][e] *= v.q[k][e];
            if (!full) {
                v.end(s0, t.n);
                end_rows<N, kPer>(u, s0, t.n);
            }
            Map<N> ahead, tile;
            join_slots<N, false>(map_of<N, kPer>(v.a, u), ahead, tile, ends[j & 1]);
            float h[N];
#pragma unroll
            for (int e = 0; e < N; ++e) h[e] = h0[e];
            ahead.apply(h);
            tile.apply(h0);
            if (!t.on) return;
            if (a.states && s0 % kStateEvery == 0 && s0 < a.L) keep(s0, h);
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) u[k][e] = h[e] = fmaf(v.a[k][e], h[e], u[k][e]);
            E *const y = yw.p + (int64_t)s0 * yw.step;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (full || s0 + k < t.n) store_own<T, N>(y + k * yw.step, u[k], t.skip);
        });
        // past the length: no outputs, and the last state from the next tile's start on
        const int from = max(first * kTile, t.n), to = min(past * kTile, a.L);
        clear_rows<T, N>(a.y, a.ys, t, from, to);
        if (a.states && t.on)
            for (int s = (max((t.n + kTile - 1) / kTile, first) * (kTile / kPer) + t.slot) * kPer; s < to; s += kTile)
                if (s % kStateEvery == 0) keep(s, h0);
        __syncthreads();
        if (a.last && t.on && t.seg == p.segs - 1 && t.slot == 0) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (t.own(e)) a.last[bc + e] = h0[e];
        }
    }
}

// ---- gradients -------------------------------------------------------------------
//
// m_s = a_s r_s = a_s (m_{s+1} + g_s): the gradient of the state ahead of s, a
// scan from the end whose maps have the same factors.

template <int N, int PER>
__device__ __forceinline__ Map<N> back_map(const float (*a)[N], const float (*g)[N]) {
    Map<N> m;
    m.clear();
#pragma unroll
    for (int k = PER - 1; k >= 0; --k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            m.H[e] = a[k][e] * (m.H[e] + g[k][e]);
            m.A[e] *= a[k][e];
        }
    return m;
}

// The map from the end of every segment but the first, in whose place stands
// the last state's gradient.
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_rec_back_segments(RecurrenceArgs a, RecPlan p, float2 *out, int64_t jobs) {
    __shared__ Map<N> ends[2][kWaves][kLanes];
    constexpr int TILE = kTileBack, PER = kPerBack;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const Walk<T> dw(a.g, a.gs, a, t), gw(a.gate, a.gates, a, t);
        Map<N> all;
        all.clear();
        if (t.seg == 0) {
            if (a.g_last)
#pragma unroll
                for (int e = 0; e < N; ++e) all.H[e] = a.g_last[(int64_t)t.b * a.C + t.at + e];
        } else {
            const int first = t.seg * p.seg_tiles, past = min(first + p.seg_tiles, (t.n + TILE - 1) / TILE);
            Rows<T, N, PER> dr, gr;
            auto next = [&](int i) {
                const int s0 = i * TILE + t.slot * PER;
                if ((i + 1) * TILE <= t.n) {
                    dr.template load<true>(dw, s0, t.n);
                    gr.template load<true>(gw, s0, t.n);
                } else {
                    dr.template load<false>(dw, s0, t.n);
                    gr.template load<false>(gw, s0, t.n);
                }
            };
            if (past > first) next(past - 1);
            walk<TILE, true>(first, past, t.n, next, [&](int i, int j, auto then) {
                const int s0 = i * TILE + t.slot * PER;
                Gates<T, N, PER> v(gr);
                float g[PER][N];
                widen_rows<T, N, PER>(dr, g);
                then();
                if ((i + 1) * TILE > t.n) {
                    v.end(s0, t.n);
                    end_rows<N, PER>(g, s0, t.n);
                }
                Map<N> behind, tile;
                join_slots<N, true>(back_map<N, PER>(v.a, g), behind, tile, ends[j & 1]);
                tile.after(all);
                all = tile;
            });
        }
        __syncthreads();
        if (t.slot == 0) {
            float2 *const o = out + ((int64_t)t.b * p.segs + t.seg) * a.C + t.at;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (t.own(e)) o[e] = make_float2(all.A[e], all.H[e]);
        }
    }
}

template <typename T, int N, bool BLEND>
__global__ __launch_bounds__(kThreads) void k_recurrence_back(RecurrenceArgs a, RecPlan p, const float2 *maps, int64_t jobs) {
    using E = typename T::T;
    __shared__ Map<N> ends[2][2][kWaves][kLanes];
    constexpr int TILE = kTileBack, PER = kPerBack;
    const int kept = (a.L + kStateEvery - 1) / kStateEvery;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const Walk<T> xw(a.x, a.xs, a, t), gw(a.gate, a.gates, a, t), dw(a.g, a.gs, a, t), gxw(a.gx, a.gxs, a, t), ggw(a.gg, a.ggs, a, t);
        const int64_t bc = (int64_t)t.b * a.C + t.at;
        const int first = t.seg * p.seg_tiles, whole = first + p.seg_tiles, past = min(whole, (t.n + TILE - 1) / TILE);
        Rows<T, N, PER> xr, gr, dr;
        float hn[N];  // the state that a tile starts from
        auto next = [&](int i) {
            const int s0 = i * TILE + t.slot * PER;
            if ((i + 1) * TILE <= t.n) {
                xr.template load<true>(xw, s0, t.n);
                gr.template load<true>(gw, s0, t.n);
                dr.template load<true>(dw, s0, t.n);
            } else {
                xr.template load<false>(xw, s0, t.n);
                gr.template load<false>(gw, s0, t.n);
                dr.template load<false>(dw, s0, t.n);
            }
            const float *const st = a.states + ((int64_t)t.b * kept + (int64_t)i * TILE / kStateEvery) * a.C + t.at;
#pragma unroll
            for (int e = 0; e < N; ++e) hn[e] = st[e];
        };
        if (past > first) next(past - 1);
        float m0[N] = {};
        carry_in<N>(a, p, t, a.g_last, maps, p.segs - 1, t.seg, -1, m0);
        walk<TILE, true>(first, past, t.n, next, [&](int i, int j, auto then) {
            const int s0 = i * TILE + t.slot * PER;
            const bool full = (i + 1) * TILE <= t.n;
            Gates<T, N, PER> v(gr);
            float x[PER][N], g[PER][N], h[N], m[N], u[PER][N];
            widen_rows<T, N, PER>(xr, x);
            widen_rows<T, N, PER>(dr, g);
#pragma unroll
            for (int e = 0; e < N; ++e) h[e] = hn[e];
            then();
            if (!full) {
                v.end(s0, t.n);
                end_rows<N, PER>(x, s0, t.n);
                end_rows<N, PER>(g, s0, t.n);
            }
#pragma unroll
            for (int k = 0; k < PER; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) u[k][e] = BLEND ? v.q[k][e] * x[k][e] : x[k][e];
            Map<N> ahead, behind, tile;
            join_slots<N, false>(map_of<N, PER>(v.a, u), ahead, tile, ends[j & 1][0]);
            join_slots<N, true>(back_map<N, PER>(v.a, g), behind, tile, ends[j & 1][1]);
            ahead.apply(h);
#pragma unroll
            for (int e = 0; e < N; ++e) m[e] = m0[e];
            behind.apply(m);
            tile.apply(m0);
            if (!t.on) return;
            // the state ahead of each position (less x), then the gradients from the last one on
#pragma unroll
            for (int k = 0; k < PER; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    x[k][e] = BLEND ? h[e] - x[k][e] : h[e];
                    h[e] = fmaf(v.a[k][e], h[e], u[k][e]);
                }
#pragma unroll
            for (int k = PER - 1; k >= 0; --k)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float r = m[e] + g[k][e];
                    m[e] = v.a[k][e] * r;
                    g[k][e] = BLEND ? r * v.q[k][e] : r;
                    x[k][e] = m[e] * v.q[k][e] * x[k][e];
                }
            if (a.gx) {
                E *const o = gxw.p + (int64_t)s0 * gxw.step;
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (full || s0 + k < t.n) store_own<T, N>(o + k * gxw.step, g[k], t.skip);
            }
            if (a.gg) {
                E *const o = ggw.p + (int64_t)s0 * ggw.step;
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (full || s0 + k < t.n) store_own<T, N>(o + k * ggw.step, x[k], t.skip);
            }
        });
        const int from = max(first * TILE, t.n), to = min(whole * TILE, a.L);
        clear_rows<T, N>(a.gx, a.gxs, t, from, to);
        clear_rows<T, N>(a.gg, a.ggs, t, from, to);
        __syncthreads();
        if (a.g_state && t.on && t.seg == 0 && t.slot == 0) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (t.own(e)) a.g_state[bc + e] = m0[e];
        }
    }
}

constexpr int64_t kMaxGrid = 1 << 21;  // workgroups of a launch; more jobs are looped over
unsigned grid_for(int64_t jobs) { return (unsigned)std::min(jobs, kMaxGrid); }

template <typename T, int N, bool BLEND>
hipError_t run(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, kTile, num_cus);
    const int64_t jobs = (int64_t)a.B * p.segs * p.slabs;
    if (p.segs > 1)
        hipLaunchKernelGGL((k_rec_segments<T, N, BLEND>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (float2 *)a.ws, jobs);
    hipLaunchKernelGGL((k_recurrence<T, N, BLEND>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (const float2 *)a.ws, jobs);
    return hipGetLastError();
}

template <typename T, int N, bool BLEND>
hipError_t run_back(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, kTileBack, num_cus);
    const int64_t jobs = (int64_t)a.B * p.segs * p.slabs;
    if (p.segs > 1)
        hipLaunchKernelGGL((k_rec_back_segments<T, N>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (float2 *)a.ws, jobs);
    hipLaunchKernelGGL((k_recurrence_back<T, N, BLEND>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (const float2 *)a.ws, jobs);
    return hipGetLastError();
}

template <typename F>
hipError_t by_type(const RecurrenceArgs &a, F f) {
    auto blend = [&](auto t, auto n) { return a.blend ? f(t, n, std::true_type()) : f(t, n, std::false_type()); };
    auto piece = [&](auto t) {
        return rec_piece(a.C) == 4 ? blend(t, std::integral_constant<int, 4>()) : blend(t, std::integral_constant<int, 1>());
    };
    return a.dtype == kF32 ? piece(F32()) : piece(BF16());
}

}  // namespace

size_t recurrence_workspace(int B, int L, int C, int, bool backward, int num_cus) {
    return plan_recurrence(B, L, C, backward ? kTileBack : kTile, num_cus).ws_bytes;
}

hipError_t launch_recurrence(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    return by_type(a, [&](auto t, auto n, auto blend) { return run<decltype(t), decltype(n)::value, decltype(blend)::value>(a, num_cus, stream); });
}

hipError_t launch_recurrence_backward(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    return by_type(a,
                   [&](auto t, auto n, auto blend) { return run_back<decltype(t), decltype(n)::value, decltype(blend)::value>(a, num_cus, stream); });
}

}  // namespace dc1d
