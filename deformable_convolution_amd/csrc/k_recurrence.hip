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
// A workgroup is kSlots slots of kPer positions by kLanes pieces of N channels,
// so that rows are read in runs of kLanes pieces; a tile is kTile positions.  A
// slot's positions stay in registers: their map is formed, the slots' maps are
// joined over the wave's lanes and the waves, and the states follow.
#include <algorithm>

#include "vec16.h"

namespace dc1d {

namespace {

constexpr int kLanes = 16, kSlots = 16, kPer = 4, kTile = kSlots * kPer, kThreads = kLanes * kSlots;
constexpr int kWaveSlots = 64 / kLanes, kWaves = kThreads / 64;
static_assert(kStateEvery % kTile == 0 || kTile % kStateEvery == 0, "a tile starts at a kept state or the other way round");
static_assert(kStateEvery % kPer == 0, "a kept state stands ahead of a slot");

struct RecPlan {
    int slabs, segs, seg_tiles;
    size_t ws_bytes;
};

int rec_piece(int C) { return C >= 4 ? 4 : 1; }

// The positions in segments of whole tiles, a workgroup each, until there are
// four workgroups for every CU; with one segment a workgroup walks through all of them.
RecPlan plan_recurrence(int B, int L, int C, int num_cus) {
    RecPlan p;
    const int P = (C + rec_piece(C) - 1) / rec_piece(C);
    p.slabs = (P + kLanes - 1) / kLanes;
    const int64_t rows = (int64_t)B * p.slabs, tiles = std::max(1, (L + kTile - 1) / kTile);
    const int64_t want = rows > 0 ? (4ll * num_cus + rows - 1) / rows : 1;
    p.segs = (int)std::max<int64_t>(1, std::min({want, tiles, (int64_t)64}));
    p.seg_tiles = (int)((tiles + p.segs - 1) / p.segs);
    p.segs = (int)((tiles + p.seg_tiles - 1) / p.seg_tiles);
    p.ws_bytes = p.segs > 1 ? (size_t)B * p.segs * C * sizeof(float2) : 0;
    return p;
}

// A thread's channels and the order of its sequence.
template <int N>
struct Lane {
    int b, n, slot, at, skip, seg;
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
    __device__ __forceinline__ int64_t row(const RecurrenceArgs &a, int s) const {
        return a.reverse && s < n ? n - 1 - s : s;
    }
    __device__ __forceinline__ bool own(int e) const { return e >= skip; }
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
        Map<N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int from = lane + (BACK ? d : -d) * kLanes;
            o.A[e] = __shfl(own.A[e], from & 63);
            o.H[e] = __shfl(own.H[e], from & 63);
        }
        if (place >= d) own.after(o);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int from = lane + (BACK ? 1 : -1) * kLanes;
        ahead.A[e] = __shfl(own.A[e], from & 63);
        ahead.H[e] = __shfl(own.H[e], from & 63);
    }
    if (place == 0) ahead.clear();
    if (place == kWaveSlots - 1) ends[w][p] = own;
    __syncthreads();
    tile.clear();
    Map<N> before = tile;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const int from = BACK ? kWaves - 1 - i : i;
        if (from == w) before = tile;
        Map<N> o = ends[from][p];
        o.after(tile);
        tile = o;
    }
    ahead.after(before);
}

// The factors and terms of a slot's positions, (1, 0) past the length.
template <typename T, int N>
struct Slot {
    using P = Piece<T, N>;
    using E = typename T::T;
    float a[kPer][N], q[kPer][N], x[kPer][N];  // sigmoid(gate), 1 - it
    __device__ __forceinline__ void load(const RecurrenceArgs &r, const Lane<N> &t, int s0) {
        const E *const xp = (const E *)r.x + t.b * r.xs.b + t.at, *const gp = (const E *)r.gate + t.b * r.gates.b + t.at;
        typename P::Raw xr[kPer], gr[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int s = s0 + k;
            if (!t.on || s >= t.n) continue;
            const int64_t row = t.row(r, s);
            xr[k] = P::load(xp + row * r.xs.l);
            gr[k] = P::load(gp + row * r.gates.l);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const bool in = t.on && s0 + k < t.n;
            float f[N] = {}, z[N] = {};
            if (in) {
                P::widen(xr[k], f);
                P::widen(gr[k], z);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sigmoid_pair(z[e], a[k][e], q[k][e]);
                x[k][e] = f[e];
                if (!in) a[k][e] = 1.0f, q[k][e] = 0.0f;
            }
        }
    }
    __device__ __forceinline__ float term(int k, int e, bool blend) const { return blend ? q[k][e] * x[k][e] : x[k][e]; }
    __device__ __forceinline__ Map<N> map(bool blend) const {
        Map<N> m;
        m.clear();
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                m.H[e] = fmaf(a[k][e], m.H[e], term(k, e, blend));
                m.A[e] *= a[k][e];
            }
        return m;
    }
};

// The map of every segment but the last: [b][seg][C].  In the last one's place
// stands the first state, which the next kernel may overwrite with the last.
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_rec_segments(RecurrenceArgs a, RecPlan p, float2 *out, int64_t jobs) {
    __shared__ Map<N> ends[2][kWaves][kLanes];
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        Map<N> all;
        all.clear();
        const bool none = t.seg == p.segs - 1;
        if (none && a.state) {
#pragma unroll
            for (int e = 0; e < N; ++e) all.H[e] = a.state[(int64_t)t.b * a.C + t.at + e];
        }
        for (int i = 0; i < p.seg_tiles && !none; ++i) {
            const int s0 = (t.seg * p.seg_tiles + i) * kTile;
            if (s0 >= t.n) break;
            Slot<T, N> v;
            v.load(a, t, s0 + t.slot * kPer);
            Map<N> ahead, tile;
            join_slots<N, false>(v.map(a.blend), ahead, tile, ends[i & 1]);
            tile.after(all);
            all = tile;
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
    if (!t.on) return;
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

template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_recurrence(RecurrenceArgs a, RecPlan p, const float2 *maps, int64_t jobs) {
    using E = typename T::T;
    __shared__ Map<N> ends[2][kWaves][kLanes];
    const int kept = (a.L + kStateEvery - 1) / kStateEvery, tiles = (a.L + kTile - 1) / kTile;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const int64_t bc = (int64_t)t.b * a.C + t.at;
        float h0[N] = {};
        carry_in<N>(a, p, t, a.state, maps, 0, t.seg, 1, h0);
        const int first = t.seg * p.seg_tiles, past = min(first + p.seg_tiles, tiles);
        for (int i = first; i < past; ++i) {
            const int s0 = i * kTile + t.slot * kPer;
            Slot<T, N> v;
            v.load(a, t, s0);
            Map<N> ahead, tile;
            join_slots<N, false>(v.map(a.blend), ahead, tile, ends[i & 1]);
            float h[N];
#pragma unroll
            for (int e = 0; e < N; ++e) h[e] = h0[e];
            ahead.apply(h);
            tile.apply(h0);
            if (a.states && t.on && s0 % kStateEvery == 0 && s0 < a.L) {
                float *const o = a.states + ((int64_t)t.b * kept + s0 / kStateEvery) * a.C + t.at;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (t.own(e)) o[e] = h[e];
            }
            E *const y = (E *)a.y + t.b * a.ys.b + t.at;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int s = s0 + k;
                float f[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    h[e] = fmaf(v.a[k][e], h[e], v.term(k, e, a.blend));
                    f[e] = s < t.n ? h[e] : 0.0f;
                }
                if (t.on && s < a.L) store_own<T, N>(y + t.row(a, s) * a.ys.l, f, t.skip);
            }
        }
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

template <typename T, int N>
__device__ __forceinline__ void load_grad(const RecurrenceArgs &r, const Lane<N> &t, int s0, float (*g)[N]) {
    using P = Piece<T, N>;
    const typename T::T *const p = (const typename T::T *)r.g + t.b * r.gs.b + t.at;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        float f[N] = {};
        if (t.on && s0 + k < t.n) P::widen(P::load(p + t.row(r, s0 + k) * r.gs.l), f);
#pragma unroll
        for (int e = 0; e < N; ++e) g[k][e] = f[e];
    }
}

template <typename T, int N>
__device__ __forceinline__ Map<N> back_map(const Slot<T, N> &v, float (*g)[N]) {
    Map<N> m;
    m.clear();
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            m.H[e] = v.a[k][e] * (m.H[e] + g[k][e]);
            m.A[e] *= v.a[k][e];
        }
    return m;
}

// The map from the end of every segment but the first, in whose place stands
// the last state's gradient.
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_rec_back_segments(RecurrenceArgs a, RecPlan p, float2 *out, int64_t jobs) {
    __shared__ Map<N> ends[2][kWaves][kLanes];
    const int tiles = (a.L + kTile - 1) / kTile;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        Map<N> all;
        all.clear();
        const bool none = t.seg == 0;
        if (none && a.g_last) {
#pragma unroll
            for (int e = 0; e < N; ++e) all.H[e] = a.g_last[(int64_t)t.b * a.C + t.at + e];
        }
        const int first = t.seg * p.seg_tiles, past = min(first + p.seg_tiles, tiles);
        for (int i = past - 1; i >= first && !none; --i) {
            if (i * kTile >= t.n) continue;
            const int s0 = i * kTile + t.slot * kPer;
            Slot<T, N> v;
            v.load(a, t, s0);
            float g[kPer][N];
            load_grad<T, N>(a, t, s0, g);
            Map<N> behind, tile;
            join_slots<N, true>(back_map<T, N>(v, g), behind, tile, ends[i & 1]);
            tile.after(all);
            all = tile;
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

template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_recurrence_back(RecurrenceArgs a, RecPlan p, const float2 *maps, int64_t jobs) {
    using E = typename T::T;
    __shared__ Map<N> ends[2][2][kWaves][kLanes];
    const int kept = (a.L + kStateEvery - 1) / kStateEvery, tiles = (a.L + kTile - 1) / kTile;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Lane<N> t(a, p, job);
        const int64_t bc = (int64_t)t.b * a.C + t.at;
        float m0[N] = {};
        carry_in<N>(a, p, t, a.g_last, maps, p.segs - 1, t.seg, -1, m0);
        const int first = t.seg * p.seg_tiles, past = min(first + p.seg_tiles, tiles);
        for (int i = past - 1; i >= first; --i) {
            const int s0 = i * kTile + t.slot * kPer;
            Slot<T, N> v;
            v.load(a, t, s0);
            float g[kPer][N], h[N] = {}, m[N];
            load_grad<T, N>(a, t, s0, g);
            if (t.on) {
                const float *const st = a.states + ((int64_t)t.b * kept + (int64_t)i * kTile / kStateEvery) * a.C + t.at;
#pragma unroll
                for (int e = 0; e < N; ++e) h[e] = st[e];
            }
            Map<N> ahead, behind, tile;
            join_slots<N, false>(v.map(a.blend), ahead, tile, ends[i & 1][0]);
            join_slots<N, true>(back_map<T, N>(v, g), behind, tile, ends[i & 1][1]);
            ahead.apply(h);
#pragma unroll
            for (int e = 0; e < N; ++e) m[e] = m0[e];
            behind.apply(m);
            tile.apply(m0);
            // the state ahead of each position (less x), then the gradients from the last one on
            float d[kPer][N];
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    d[k][e] = a.blend ? h[e] - v.x[k][e] : h[e];
                    h[e] = fmaf(v.a[k][e], h[e], v.term(k, e, a.blend));
                }
            E *const gx = (E *)a.gx + t.b * a.gxs.b + t.at, *const gg = (E *)a.gg + t.b * a.ggs.b + t.at;
#pragma unroll
            for (int k = kPer - 1; k >= 0; --k) {
                const int s = s0 + k;
                float fx[N], fg[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float r = m[e] + g[k][e];
                    m[e] = v.a[k][e] * r;
                    fx[e] = s < t.n ? (a.blend ? r * v.q[k][e] : r) : 0.0f;
                    fg[e] = s < t.n ? m[e] * v.q[k][e] * d[k][e] : 0.0f;
                }
                if (!t.on || s >= a.L) continue;
                const int64_t row = t.row(a, s);
                if (a.gx) store_own<T, N>(gx + row * a.gxs.l, fx, t.skip);
                if (a.gg) store_own<T, N>(gg + row * a.ggs.l, fg, t.skip);
            }
        }
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

template <typename T, int N>
hipError_t run(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, num_cus);
    const int64_t jobs = (int64_t)a.B * p.segs * p.slabs;
    if (p.segs > 1) hipLaunchKernelGGL((k_rec_segments<T, N>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (float2 *)a.ws, jobs);
    hipLaunchKernelGGL((k_recurrence<T, N>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (const float2 *)a.ws, jobs);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t run_back(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, num_cus);
    const int64_t jobs = (int64_t)a.B * p.segs * p.slabs;
    if (p.segs > 1)
        hipLaunchKernelGGL((k_rec_back_segments<T, N>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (float2 *)a.ws, jobs);
    hipLaunchKernelGGL((k_recurrence_back<T, N>), dim3(grid_for(jobs)), dim3(kThreads), 0, stream, a, p, (const float2 *)a.ws, jobs);
    return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace(int B, int L, int C, int, bool, int num_cus) { return plan_recurrence(B, L, C, num_cus).ws_bytes; }

hipError_t launch_recurrence(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    if (a.dtype == kF32) return a.C >= 4 ? run<F32, 4>(a, num_cus, stream) : run<F32, 1>(a, num_cus, stream);
    return a.C >= 4 ? run<BF16, 4>(a, num_cus, stream) : run<BF16, 1>(a, num_cus, stream);
}

hipError_t launch_recurrence_backward(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    if (a.dtype == kF32) return a.C >= 4 ? run_back<F32, 4>(a, num_cus, stream) : run_back<F32, 1>(a, num_cus, stream);
    return a.C >= 4 ? run_back<BF16, 4>(a, num_cus, stream) : run_back<BF16, 1>(a, num_cus, stream);
}

}  // namespace dc1d
