// k_recurrence.hip -- a gated linear recurrence along the positions and its
// gradients, every channel on its own:
//
//   h_s = a_s h_{s-1} + u_s,  a = sigmoid(gate),  u = x or (1 - a) x
//   r_s = g_s + a_{s+1} r_{s+1},  gx = r or r (1 - a),
//   ggate = r (h_{s-1} or h_{s-1} - x) a (1 - a),  gstate = a_0 r_0
//
// s counts the positions in the recurrence's order.  Both are scans of affine
// maps h -> A h + H, joined as (A, H) then (A', H') = (A A', A' H + H').  Bound
// by HBM: the forward has to read x and gate and write y, the backward to read x,
// gate and g and write two gradients; at some 30 and 45 instructions an element
// the arithmetic takes more than half of that time and has to run beside it.
//
// A workgroup is 16 or 32 slots of a few positions by 16 pieces of N channels, so that
// rows are read in runs of 16 pieces; a tile is the slots' positions.  A slot's
// positions stay in registers: their map is formed, the slots' maps are joined
// over the wave's rows of lanes and the waves, and the states follow.  Four
// positions: the join is some 6 instructions an element then, and more would leave
// fewer waves a SIMD to hide the loads.
#include <algorithm>
#include <type_traits>

#include "vec16.h"

namespace dc1d {

namespace {

constexpr int kLanes = 16, kSlots = 16;  // a workgroup has SL slots: kSlots or twice that
constexpr int kPer = 4, kPerBack = 4;  // positions of a slot
static_assert(kStateEvery % kPer == 0, "a kept state stands ahead of a slot");
static_assert(kSlots * kPerBack % kStateEvery == 0, "a tile of the backward pass starts at a kept state");

// Offsets inside a tile: 32 bits for pieces of four channels, 64 for single ones,
// which also serve rows too far apart for that.
template <int N>
using Offset = std::conditional_t<N == 1, int64_t, uint32_t>;

// A thread's channels and its sequence.
template <int N>
struct Lane {
    int b, n, slot, at, skip;  // n: positions within the length
    bool on;
    __device__ __forceinline__ Lane(const RecurrenceArgs &a, uint32_t chain, const FastDiv &by_slabs) {
        b = (int)fdiv(chain, by_slabs);
        const int slab = (int)(chain - (uint32_t)b * by_slabs.d);
        n = a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
        slot = threadIdx.x / kLanes;
        const int c = (slab * kLanes + threadIdx.x % kLanes) * N;
        on = c < a.C;
        at = on ? min(c, a.C - N) : 0;
        skip = on ? c - at : N;
    }
    __device__ __forceinline__ bool own(int e) const { return e >= skip; }
    __device__ __forceinline__ int64_t state(const RecurrenceArgs &a) const { return (int64_t)b * a.C + at; }
    // the kept state ahead of position s
    __device__ __forceinline__ int64_t kept(const RecurrenceArgs &a, int s) const {
        return ((int64_t)b * ((a.L + kStateEvery - 1) / kStateEvery) + s / kStateEvery) * a.C + at;
    }
};

// A piece's store; only where C is no multiple of a piece (ODD) may elements of it
// be its neighbour's.  Both threads then store the same values, unless the call
// writes over what they are formed from (`in_place`): the neighbour's workgroup
// may have done so already.
template <typename T, int N, bool ODD>
__device__ __forceinline__ void put(typename T::T *p, const float *f, int skip, bool in_place) {
    if constexpr (ODD)
        store_own<T, N>(p, f, skip, in_place);
    else
        Piece<T, N>::store(p, f);
}

// A slot's rows of a tensor in one tile: a base that all threads share (of each
// row, on scalar registers), and the slot's offset from it.  Reversed, the base is
// the tile's last position.
template <typename T, int N, int PER, int SL>
struct Walk {
    static constexpr int TILE = SL * PER;
    using E = typename T::T;
    char *base;
    int64_t step;
    Offset<N> off;
    bool reverse;
    __device__ __forceinline__ Walk(const void *t, Strides2 st, const RecurrenceArgs &a, const Lane<N> &l, int tile) {
        reverse = a.reverse;
        const int64_t row = reverse ? (int64_t)max(l.n, 1) - (int64_t)(tile + 1) * TILE : (int64_t)tile * TILE;
        base = (char *)t + (l.b * st.b + row * st.l) * (int64_t)sizeof(E);
        step = st.l * (int64_t)sizeof(E);
        off = (Offset<N>)(l.at * sizeof(E)) + (Offset<N>)((reverse ? SL - 1 - l.slot : l.slot) * PER) * (Offset<N>)step;
    }
    // Row k of the slot, the same k for all threads; or any of the tile's rows, counted from the slot's first.
    __device__ __forceinline__ E *at(int k) const { return (E *)((base + (reverse ? PER - 1 - k : k) * step) + off); }
    __device__ __forceinline__ E *any(int k) const {
        return (E *)(base + (Offset<N>)(off + (Offset<N>)(reverse ? PER - 1 - k : k) * (Offset<N>)step));
    }
};

// Ends a branch whose loads or stores the compiler would join with the other
// branch's, at addresses of 64 bits a lane.
__device__ __forceinline__ void apart() { asm volatile("; whole tile" ::: "memory"); }

// A tile past the length reads the last one within it (and uses none of it): the
// rows that are read lie in the tile that they are read from, so that no offset
// is negative.
template <int TILE>
__device__ __forceinline__ int last_tile(int n, int i) {
    return min(i, (max(n, 1) - 1) / TILE);
}

// A piece of a value's bits.
template <typename T, int N>
__device__ __forceinline__ typename Piece<T, N>::Raw every(uint32_t f32) {
    const uint32_t w = std::is_same<T, F32>::value ? f32 : N == 1 ? f32 >> 16 : (f32 >> 16) * 0x10001u;
    typename Piece<T, N>::Raw r;
    if constexpr (N == 1)
        r = w;
    else
        for (int i = 0; i < (int)(sizeof(r) / 4); ++i) r[i] = w;
    return r;
}

template <typename T, int N, int PER>
struct Rows {
    typename Piece<T, N>::Raw r[PER];
    // From the slot's position `left` on, a value: a gate of infinity holds the state (a = 1, 1 - a = 0) and zeros add nothing.
    __device__ __forceinline__ void end(int left, uint32_t f32) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k >= left) r[k] = every<T, N>(f32);
    }
    // `last`: the sequence's last position within the length (the first, for none),
    // counted from the slot's first, in place of those past it
    template <bool FULL, int SL>
    __device__ __forceinline__ void load(const Walk<T, N, PER, SL> &w, int last) {
#pragma unroll
        for (int k = 0; k < PER; ++k) r[k] = Piece<T, N>::load(FULL ? w.at(k) : w.any(min(k, last)));
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
    // this one, then h -> a h + u
    __device__ __forceinline__ void then(const float *a, const float *u) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            H[e] = fmaf(a[e], H[e], u[e]);
            A[e] *= a[e];
        }
    }
    __device__ __forceinline__ void hold_all() {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            hold(A[e]);
            hold(H[e]);
        }
    }
    // this one, then h -> a (h + g)
    __device__ __forceinline__ void then_back(const float *a, const float *g) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            H[e] = a[e] * (H[e] + g[e]);
            A[e] *= a[e];
        }
    }
};

// A wave has four slots.  The map of those ahead of a thread's goes to `ahead` (of
// those behind it where BACK), the wave's to `ends`.  The slots are rows of 16 lanes:
// v_permlane16_swap gives both rows of a pair their even and odd row's values,
// v_permlane32_swap both halves' to both.  The caller's barriers keep `ends` from
// the next use; two of them in turn need one barrier each.
template <int N, int SL>
using Ends = Map<N>[SL / 4][kLanes];

template <int N, bool BACK, int SL>
__device__ __forceinline__ void join_slots(const Map<N> &own, Map<N> &ahead, Ends<N, SL> &ends) {
    const int lane = threadIdx.x & 63;
    const bool second = ((lane >> 4) & 1) != BACK, later = (lane >> 5) != BACK;
    Map<N> all;
    auto both = [](float v, bool wide, float &first, float &next) {
        const auto r = wide ? __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false)
                            : __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        first = __uint_as_float(r[BACK ? 1 : 0]);
        next = __uint_as_float(r[BACK ? 0 : 1]);
    };
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float A1, A2, H1, H2;
        both(own.A[e], false, A1, A2);
        both(own.H[e], false, H1, H2);
        const float A = second ? A1 : 1.0f, H = second ? H1 : 0.0f;
        H2 = fmaf(A2, H1, H2);
        A2 *= A1;
        both(A2, true, A1, A2);
        both(H2, true, H1, H2);
        ahead.A[e] = A * (later ? A1 : 1.0f);
        ahead.H[e] = fmaf(A, later ? H1 : 0.0f, H);
        all.A[e] = A2 * A1;
        all.H[e] = fmaf(A2, H1, H2);
    }
    if (lane < kLanes) ends[threadIdx.x >> 6][lane] = all;
}

// After a barrier: h goes from the tile's start to its end, and `here` is the state ahead of the thread's wave.
template <int N, bool BACK, int SL>
__device__ __forceinline__ void pass_waves(const Ends<N, SL> &ends, float *h, float *here) {
    const int w = threadIdx.x >> 6, p = threadIdx.x % kLanes;
#pragma unroll
    for (int i = 0; i < SL / 4; ++i) {
        const int wave = BACK ? SL / 4 - 1 - i : i;
        if (wave == w)  // the same for all of a wave
#pragma unroll
            for (int e = 0; e < N; ++e) here[e] = h[e];
        ends[wave][p].apply(h);
    }
}

// After a barrier: the map of all of the waves' slots, behind `m`.
template <int N, bool BACK, int SL>
__device__ __forceinline__ void join_waves(const Ends<N, SL> &ends, Map<N> &m) {
#pragma unroll
    for (int i = 0; i < SL / 4; ++i) {
        Map<N> o = ends[BACK ? SL / 4 - 1 - i : i][threadIdx.x % kLanes];
        o.after(m);
        m = o;
    }
}

// Rows past the length become 0: positions from ... to - 1, slot by slot.
template <typename T, int N, int SL>
__device__ __forceinline__ void clear_rows(void *t, Strides2 st, const Lane<N> &l, int from, int to) {
    if (!t || !l.on) return;
    const float zero[N] = {};
    typename T::T *const p = (typename T::T *)t + l.b * st.b + l.at;
    for (int s = from + l.slot; s < to; s += SL) store_own<T, N>(p + s * st.l, zero, l.skip);
}

template <int N>
__device__ __forceinline__ void store_state(float *o, const Lane<N> &t, const float *h) {
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (t.own(e)) o[e] = h[e];
}

// ---- the forward's tile -------------------------------------------------------------

template <typename T, int N, int PER, int SL, bool ODD, bool BLEND>
struct Tile {
    static constexpr int TILE = SL * PER;
    Rows<T, N, PER> xr, gr;
    float a[PER][N], u[PER][N];
    __device__ __forceinline__ void load(const RecurrenceArgs &r, const Lane<N> &t, int i) {
        const int from = last_tile<TILE>(t.n, i), last = max(t.n, 1) - 1 - from * TILE - t.slot * PER;
        const Walk<T, N, PER, SL> gw(r.gate, r.gates, r, t, from), xw(r.x, r.xs, r, t, from);
        if ((i + 1) * TILE <= t.n) {
            gr.template load<true>(gw, last);
            xr.template load<true>(xw, last);
            apart();
        } else {
            gr.template load<false>(gw, last);
            xr.template load<false>(xw, last);
        }
    }
    // The slot's map, from its last position on where BACK.
    template <bool BACK = false>
    __device__ __forceinline__ Map<N> form(const Lane<N> &t, int i) {
        if ((i + 1) * TILE > t.n) {
            const int left = t.n - i * TILE - t.slot * PER;
            gr.end(left, 0x7f800000u);
            xr.end(left, 0u);
        }
        Map<N> m;
        m.clear();
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int k = BACK ? PER - 1 - j : j;
            float z[N], q[N];
            hold(gr.r[k]);
            hold(xr.r[k]);
            Piece<T, N>::widen(gr.r[k], z);
            Piece<T, N>::widen(xr.r[k], u[k]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sigmoid_pair(z[e], a[k][e], q[e]);
                if (BLEND) u[k][e] *= q[e];
            }
            if (BACK)
                m.then_back(a[k], u[k]);
            else
                m.then(a[k], u[k]);
            m.hold_all();
        }
        return m;
    }
    // the states from h on, to y
    __device__ __forceinline__ void store(const RecurrenceArgs &r, const Lane<N> &t, int i, float *h) {
        if (!t.on) return;
        const int s0 = i * TILE + t.slot * PER, left = t.n - s0;
        if (r.states && s0 % kStateEvery == 0 && s0 < r.L) store_state<N>(r.states + t.kept(r, s0), t, h);
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) u[k][e] = h[e] = fmaf(a[k][e], h[e], u[k][e]);
        const Walk<T, N, PER, SL> yw(r.y, r.ys, r, t, i);
        if ((i + 1) * TILE <= t.n) {
#pragma unroll
            for (int k = 0; k < PER; ++k) put<T, N, ODD>(yw.at(k), u[k], t.skip, r.in_place);
            apart();
        } else {
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (k < left) put<T, N, ODD>(yw.at(k), u[k], t.skip, r.in_place);
        }
    }
};

// ---- segments -----------------------------------------------------------------------
//
// A chain (a sequence's 16 pieces of channels) is cut into segments of whole
// tiles, a workgroup each.  Where there is more than one, a kernel ahead forms
// every segment's map; a workgroup joins those of the segments ahead of its own,
// a slot some of them, and walks through its tiles.  So gate and x are
// read twice: 8 x 16384 x 256 bf16 moves 335 MB in 32 + 43 us, gradients 470 in 35 +
// 76.  (Joined as they come from workgroup to workgroup in one pass, the result
// depends on the order of arrival; in a fixed order it waited longer: 95 us and
// 159.  A run of neighbouring positions for every slot, whose maps need no joins
// inside a tile: 72 to 77.)
struct Segments {
    int segs, tiles;          // segments of a chain, tiles of a segment (the last one may have fewer)
    FastDiv by_segs, by_slabs;
    uint32_t jobs, first;     // workgroups in all, and where a launch begins
    float2 *maps;             // [chain][seg][kLanes * N]: the maps; in place of the one that nobody needs, the first state
    template <int N>
    __device__ __forceinline__ float2 *at(uint32_t chain, int seg, int lane) const {
        return maps + (((int64_t)chain * segs + seg) * kLanes + lane) * N;
    }
};

// The state ahead of segment `to` in the order of the scan (BACK: from the last segment on).
template <int N, bool BACK, int SL>
__device__ __forceinline__ void carry_in(const Segments &g, uint32_t chain, int seg, const float *start, float *h, Ends<N, SL> &ends) {
    const int slot = threadIdx.x / kLanes, p = threadIdx.x % kLanes;
    if (g.segs == 1) {
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = start ? start[e] : 0.0f;
        return;
    }
    const int before = BACK ? g.segs - 1 - seg : seg, each = (before + SL - 1) / SL;  // of every slot
    const float2 *const s = g.at<N>(chain, BACK ? 0 : g.segs - 1, p);
    Map<N> m, rest;
    m.clear();
    const int from = (BACK ? SL - 1 - slot : slot) * each;
    for (int i = from; i < min(from + each, before); ++i) {
        const float2 *const o = g.at<N>(chain, BACK ? g.segs - 1 - i : i, p);
        Map<N> n;
#pragma unroll
        for (int e = 0; e < N; ++e) n.A[e] = o[e].x, n.H[e] = o[e].y;
        n.after(m);
        m = n;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = s[e].y;
    join_slots<N, BACK, SL>(m, rest, ends);
    __syncthreads();
    float here[N];
    pass_waves<N, BACK, SL>(ends, h, here);
}

template <int N>
__device__ __forceinline__ void store_map(float2 *o, const Map<N> &m) {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = make_float2(m.A[e], m.H[e]);
}

template <typename T, int N, bool BLEND>
__global__ __launch_bounds__(kLanes * kSlots) void k_rec_maps(RecurrenceArgs a, Segments g) {
    __shared__ Ends<N, kSlots> ends[2];
    using W = Tile<T, N, kPer, kSlots, false, BLEND>;
    const uint32_t job = g.first + blockIdx.x, chain = fdiv(job, g.by_segs);
    const int seg = (int)(job - chain * g.by_segs.d);
    const Lane<N> t(a, chain, g.by_slabs);
    Map<N> all;
    all.clear();
    const int first = seg * g.tiles, past = min(first + g.tiles, (t.n + W::TILE - 1) / W::TILE);
    if (seg == g.segs - 1) {
        if (a.state)
#pragma unroll
            for (int e = 0; e < N; ++e) all.H[e] = a.state[t.state(a) + e];
    } else if (first < past) {
        W v;
        v.load(a, t, first);
        for (int i = first;;) {
            const Map<N> own = v.form(t, i);
            if (i + 1 < past) v.load(a, t, i + 1);
            Map<N> ahead;
            join_slots<N, false, kSlots>(own, ahead, ends[i & 1]);
            __syncthreads();
            join_waves<N, false, kSlots>(ends[i & 1], all);
            if (++i == past) break;
        }
    }
    if (t.slot == 0) store_map<N>(g.at<N>(chain, seg, threadIdx.x), all);
}

// A tile's loads are in flight while the one before it is worked on.  32 x 1024 x
// 1024 fp32 in one pass: 82 us, 4.9 TB/s, at the rate of a copy; one position of 16
// x 512: 4 us.
template <typename T, int N, int SL, bool ODD, bool BLEND>
__global__ __launch_bounds__(kLanes * SL) void k_rec_walk(RecurrenceArgs a, Segments g) {
    __shared__ Ends<N, SL> ends[2];
    using W = Tile<T, N, kPer, SL, ODD, BLEND>;
    const int tiles = (a.L + W::TILE - 1) / W::TILE;
    const uint32_t job = g.first + blockIdx.x, chain = fdiv(job, g.by_segs);
    const int seg = (int)(job - chain * g.by_segs.d);
    const Lane<N> t(a, chain, g.by_slabs);
    const int first = seg * g.tiles, past = min(first + g.tiles, tiles);
    W v;
    v.load(a, t, first);
    float h0[N];
    carry_in<N, false, SL>(g, chain, seg, a.state ? a.state + t.state(a) : nullptr, h0, ends[(first & 1) ^ 1]);
    for (int i = first;;) {
        const Map<N> own = v.form(t, i);
        if (i + 1 < past) v.load(a, t, i + 1);
        Map<N> ahead;
        join_slots<N, false, SL>(own, ahead, ends[i & 1]);
        __syncthreads();
        float h[N];
        pass_waves<N, false, SL>(ends[i & 1], h0, h);
        ahead.apply(h);
        v.store(a, t, i, h);
        if (++i == past) break;
    }
    clear_rows<T, N, SL>(a.y, a.ys, t, max(first * W::TILE, t.n), min(past * W::TILE, a.L));
    __syncthreads();  // every thread has read the state, which `last` may be
    if (a.last && t.on && seg == g.segs - 1 && t.slot == 0) store_state<N>(a.last + t.state(a), t, h0);
}

// ---- gradients -------------------------------------------------------------------
//
// m_s = a_s r_s = a_s (m_{s+1} + g_s): the gradient of the state ahead of s, a
// scan from the end whose maps have the same factors.

template <typename T, int N, int PER, int SL, bool ODD, bool BLEND>
struct TileBack {
    static constexpr int TILE = SL * PER;
    Rows<T, N, PER> xr, gr, dr;
    float kept[N];  // the state that the tile starts from
    float a[PER][N], q[PER][N], x[PER][N], g[PER][N];
    __device__ __forceinline__ void load(const RecurrenceArgs &r, const Lane<N> &t, int i) {
        const int from = last_tile<TILE>(t.n, i), last = max(t.n, 1) - 1 - from * TILE - t.slot * PER;
        const Walk<T, N, PER, SL> gw(r.gate, r.gates, r, t, from), xw(r.x, r.xs, r, t, from), dw(r.g, r.gs, r, t, from);
        if ((i + 1) * TILE <= t.n) {
            gr.template load<true>(gw, last);
            xr.template load<true>(xw, last);
            dr.template load<true>(dw, last);
            apart();
        } else {
            gr.template load<false>(gw, last);
            xr.template load<false>(xw, last);
            dr.template load<false>(dw, last);
        }
        const float *const st = r.states + t.kept(r, i * TILE);
#pragma unroll
        for (int e = 0; e < N; ++e) kept[e] = st[e];
    }
    __device__ __forceinline__ float term(int k, int e) const { return BLEND ? q[k][e] * x[k][e] : x[k][e]; }
    // the slot's map of the states, and h = the state that the tile starts from
    __device__ __forceinline__ Map<N> form(const Lane<N> &t, int i, float *h) {
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = kept[e];
        if ((i + 1) * TILE > t.n) {
            const int left = t.n - i * TILE - t.slot * PER;
            gr.end(left, 0x7f800000u);
            xr.end(left, 0u);
            dr.end(left, 0u);
        }
        Map<N> m;
        m.clear();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            float z[N], u[N];
            hold(gr.r[k]);
            hold(xr.r[k]);
            hold(dr.r[k]);
            Piece<T, N>::widen(gr.r[k], z);
            Piece<T, N>::widen(xr.r[k], x[k]);
            Piece<T, N>::widen(dr.r[k], g[k]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sigmoid_pair(z[e], a[k][e], q[k][e]);
                u[e] = term(k, e);
                hold(q[k][e]);
            }
            m.then(a[k], u);
            m.hold_all();
        }
        return m;
    }
    __device__ __forceinline__ Map<N> map_back() const {
        Map<N> m;
        m.clear();
#pragma unroll
        for (int k = PER - 1; k >= 0; --k) m.then_back(a[k], g[k]);
        return m;
    }
    // the gradients from the state h ahead of the slot and m behind it
    __device__ __forceinline__ void store(const RecurrenceArgs &r, const Lane<N> &t, int i, float *h, float *m) {
        if (!t.on) return;
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float u = term(k, e);
                x[k][e] = BLEND ? h[e] - x[k][e] : h[e];
                h[e] = fmaf(a[k][e], h[e], u);
            }
#pragma unroll
        for (int k = PER - 1; k >= 0; --k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = m[e] + g[k][e];
                m[e] = a[k][e] * d;
                g[k][e] = BLEND ? d * q[k][e] : d;
                x[k][e] = m[e] * q[k][e] * x[k][e];
            }
        const bool full = (i + 1) * TILE <= t.n;
        const int left = t.n - i * TILE - t.slot * PER;
        if (r.gx) {
            const Walk<T, N, PER, SL> w(r.gx, r.gxs, r, t, i);
            if (full) {
#pragma unroll
                for (int k = 0; k < PER; ++k) put<T, N, ODD>(w.at(k), g[k], t.skip, r.in_place);
                apart();
            } else {
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (k < left) put<T, N, ODD>(w.at(k), g[k], t.skip, r.in_place);
            }
        }
        if (r.gg) {
            const Walk<T, N, PER, SL> w(r.gg, r.ggs, r, t, i);
            if (full) {
#pragma unroll
                for (int k = 0; k < PER; ++k) put<T, N, ODD>(w.at(k), x[k], t.skip, r.in_place);
                apart();
            } else {
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (k < left) put<T, N, ODD>(w.at(k), x[k], t.skip, r.in_place);
            }
        }
    }
};

// Of every segment, from its end: its own kernel reads gate and g only.
template <typename T, int N>
__global__ __launch_bounds__(kLanes * kSlots) void k_rec_maps_back(RecurrenceArgs a, Segments g) {
    __shared__ Ends<N, kSlots> ends[2];
    a.x = a.g, a.xs = a.gs;
    using W = Tile<T, N, kPerBack, kSlots, false, false>;
    const uint32_t job = g.first + blockIdx.x, chain = fdiv(job, g.by_segs);
    const int seg = (int)(job - chain * g.by_segs.d);
    const Lane<N> t(a, chain, g.by_slabs);
    Map<N> all;
    all.clear();
    const int first = seg * g.tiles, past = min(first + g.tiles, (t.n + W::TILE - 1) / W::TILE);
    if (seg == 0) {
        if (a.g_last)
#pragma unroll
            for (int e = 0; e < N; ++e) all.H[e] = a.g_last[t.state(a) + e];
    } else if (first < past) {
        W v;
        v.load(a, t, past - 1);
        for (int i = past - 1;;) {
            const Map<N> own = v.template form<true>(t, i);
            if (i > first) v.load(a, t, i - 1);
            Map<N> behind;
            join_slots<N, true, kSlots>(own, behind, ends[i & 1]);
            __syncthreads();
            join_waves<N, true, kSlots>(ends[i & 1], all);
            if (i-- == first) break;
        }
    }
    if (t.slot == 0) store_map<N>(g.at<N>(chain, seg, threadIdx.x), all);
}

// Both scans of a tile side by side: the states from the kept one ahead of the
// tile, the gradients from its end.  Two waves a SIMD of 200 registers (fp32 228):
// 8 x 16384 x 256 bf16 76 us, 4.4 TB/s, the vector unit busy for 60 % of it; 13 x
// 4092 x 511 fp32, ragged, 109 us (of both passes, 152; 133 with 512 channels, whose
// rows stand at even addresses).
template <typename T, int N, int SL, bool ODD, bool BLEND>
__global__ __launch_bounds__(kLanes * SL) void k_rec_walk_back(RecurrenceArgs a, Segments g) {
    __shared__ Ends<N, SL> ends[2][2];
    using W = TileBack<T, N, kPerBack, SL, ODD, BLEND>;
    const int tiles = (a.L + W::TILE - 1) / W::TILE;
    const uint32_t job = g.first + blockIdx.x, chain = fdiv(job, g.by_segs);
    const int seg = (int)(job - chain * g.by_segs.d);
    const Lane<N> t(a, chain, g.by_slabs);
    const int first = seg * g.tiles, past = min(first + g.tiles, tiles);
    W v;
    v.load(a, t, past - 1);
    float m0[N];
    carry_in<N, true, SL>(g, chain, seg, a.g_last ? a.g_last + t.state(a) : nullptr, m0, ends[past & 1][0]);
    for (int i = past - 1;;) {
        float start[N], h[N], m[N];
        const Map<N> own = v.form(t, i, start);
        if (i > first) v.load(a, t, i - 1);
        Map<N> ahead, behind;
        join_slots<N, false, SL>(own, ahead, ends[i & 1][0]);
        join_slots<N, true, SL>(v.map_back(), behind, ends[i & 1][1]);
        __syncthreads();
        pass_waves<N, false, SL>(ends[i & 1][0], start, h);
        ahead.apply(h);
        pass_waves<N, true, SL>(ends[i & 1][1], m0, m);
        behind.apply(m);
        v.store(a, t, i, h, m);
        if (i-- == first) break;
    }
    const int from = max(first * W::TILE, t.n), to = min(past * W::TILE, a.L);
    clear_rows<T, N, SL>(a.gx, a.gxs, t, from, to);
    clear_rows<T, N, SL>(a.gg, a.ggs, t, from, to);
    __syncthreads();
    if (a.g_state && t.on && seg == 0 && t.slot == 0) store_state<N>(a.g_state + t.state(a), t, m0);
}

// ---- launches ------------------------------------------------------------------------

struct RecPlan {
    Segments g;
    int slots;
    size_t ws_bytes;
};

// One pass (a segment a chain) where the chains alone keep the memory busy, with
// twice the slots where a CU has no more than one or two of them.  8 x 4096 x 1024,
// 128 chains: fp32 105 us, in two passes 134, gradients 184, 191; bf16 78, 80 and
// (three quarters of a chain a CU are needed) 145, 121; 12 x 4096 x 1024 bf16,
// 192 chains: 80, 106 and 155, 161; 6 x 4096 x 1024, 96 chains: fp32 96, 100 and
// 176, 141, bf16 75, 54 and 135, 87.  Twice the slots: 16 x 4092 x 1024 bf16, 256
// chains: 108 -> 88 us, gradients 185 -> 166; 28 x 1024 x 1024 bf16, 448 chains:
// 42.2 -> 40.8, gradients 75.7 -> 81.9; four times: 104 and 52.7; 16 x 1 x 512: 4.4 ->
// 5.3.  One pass too where another launch costs more than the tiles one after another: 2 x 512 x 256, 8 tiles of 64: 11.4,
// 15.4; 2 x 900 x 512, 15 of them: 20.4, 14.2; gradients 4 x 384 x 256, 6 tiles: 13.7,
// 16.7; 2 x 512 x 256, 8 tiles: 16.7, 16.4.  Otherwise eight workgroups a CU (16: 8 x
// 16384 x 256 bf16 77.4 -> 77.5, gradients 111 -> 120; 4: 76.2, 111), in at most 256
// segments.
RecPlan plan_recurrence(int B, int L, int C, int N, int dtype, bool backward, int num_cus) {
    RecPlan p = {};
    const int slabs = (C + N * kLanes - 1) / (N * kLanes), per = backward ? kPerBack : kPer;
    const int64_t chains = (int64_t)B * slabs;
    const auto of = [&](int slots) { return std::max<int64_t>(1, (L + (int64_t)slots * per - 1) / (slots * per)); };
    const bool one = 4 * chains >= (backward && dtype != kF32 ? 3 : 2) * num_cus || of(kSlots) <= (backward ? 6 : 10);
    p.slots = one && of(kSlots) > 1 && (backward ? chains <= num_cus : chains < 2 * num_cus) ? 2 * kSlots : kSlots;
    const int64_t tiles = of(p.slots);
    const int64_t want = chains > 0 ? (8ll * num_cus + chains - 1) / chains : 1;
    p.g.segs = (int)(one ? 1 : std::min({want, tiles, (int64_t)256}));
    p.g.tiles = (int)((tiles + p.g.segs - 1) / p.g.segs);
    p.g.segs = (int)((tiles + p.g.tiles - 1) / p.g.tiles);
    p.g.by_segs = make_fastdiv((uint32_t)p.g.segs);
    p.g.by_slabs = make_fastdiv((uint32_t)slabs);
    p.g.jobs = (uint32_t)(chains * p.g.segs);
    p.ws_bytes = p.g.segs > 1 ? (size_t)chains * p.g.segs * kLanes * N * sizeof(float2) : 0;
    return p;
}

// Pieces of four channels, where a tile's rows lie within 2^31 bytes of each other.
int rec_piece(const RecurrenceArgs &a, int tile) {
    if (a.C < 4) return 1;
    const int64_t far = ((int64_t)1 << 31) / 4 - a.C;
    for (const Strides2 &s : {a.xs, a.gates, a.gs, a.ys, a.gxs, a.ggs})
        if (s.l > far / tile) return 1;
    return 4;
}

// No positions: the state stays.
__global__ __launch_bounds__(256) void k_rec_empty(const float *from, float *to, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) to[i] = from ? from[i] : 0.0f;
}
hipError_t run_empty(const RecurrenceArgs &a, const float *from, float *to, hipStream_t stream) {
    const int64_t n = (int64_t)a.B * a.C;
    if (to && to != from)
        hipLaunchKernelGGL(k_rec_empty, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16)), dim3(256), 0, stream, from, to, n);
    return hipGetLastError();
}

constexpr uint32_t kMaxGrid = 1 << 23;  // workgroups of a launch

// f(workgroups), for all of the jobs
template <typename F>
hipError_t in_launches(Segments &g, F f) {
    for (g.first = 0; g.first < g.jobs; g.first += std::min(g.jobs - g.first, kMaxGrid)) f(dim3(std::min(g.jobs - g.first, kMaxGrid)));
    return hipGetLastError();
}

template <typename T, int N, bool ODD, bool BLEND>
hipError_t run(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, N, a.dtype, false, num_cus);
    Segments g = p.g;
    g.maps = (float2 *)a.ws;
    const dim3 block(kLanes * p.slots);
    if (g.segs > 1) {
        const hipError_t e = in_launches(g, [&](dim3 grid) { hipLaunchKernelGGL((k_rec_maps<T, N, BLEND>), grid, block, 0, stream, a, g); });
        if (e != hipSuccess) return e;
    }
    return in_launches(g, [&](dim3 grid) {
        if (p.slots == kSlots)
            hipLaunchKernelGGL((k_rec_walk<T, N, kSlots, ODD, BLEND>), grid, block, 0, stream, a, g);
        else
            hipLaunchKernelGGL((k_rec_walk<T, N, 2 * kSlots, ODD, BLEND>), grid, block, 0, stream, a, g);
    });
}

template <typename T, int N, bool ODD, bool BLEND>
hipError_t run_back(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    const RecPlan p = plan_recurrence(a.B, a.L, a.C, N, a.dtype, true, num_cus);
    Segments g = p.g;
    g.maps = (float2 *)a.ws;
    const dim3 block(kLanes * p.slots);
    if (g.segs > 1) {
        const hipError_t e = in_launches(g, [&](dim3 grid) { hipLaunchKernelGGL((k_rec_maps_back<T, N>), grid, block, 0, stream, a, g); });
        if (e != hipSuccess) return e;
    }
    return in_launches(g, [&](dim3 grid) {
        if (p.slots == kSlots)
            hipLaunchKernelGGL((k_rec_walk_back<T, N, kSlots, ODD, BLEND>), grid, block, 0, stream, a, g);
        else
            hipLaunchKernelGGL((k_rec_walk_back<T, N, 2 * kSlots, ODD, BLEND>), grid, block, 0, stream, a, g);
    });
}

// f(storage type, elements of a piece, whether C is no multiple of it, blend)
template <typename F>
hipError_t by_type(const RecurrenceArgs &a, int tile, F f) {
    auto blend = [&](auto t, auto n, auto odd) { return a.blend ? f(t, n, odd, std::true_type()) : f(t, n, odd, std::false_type()); };
    auto piece = [&](auto t) {
        if (rec_piece(a, tile) == 1) return blend(t, std::integral_constant<int, 1>(), std::false_type());
        return a.C % 4 ? blend(t, std::integral_constant<int, 4>(), std::true_type())
                       : blend(t, std::integral_constant<int, 4>(), std::false_type());
    };
    return a.dtype == kF32 ? piece(F32()) : piece(BF16());
}

}  // namespace

// The strides decide between pieces of four channels and single ones: room for either.
size_t recurrence_workspace(int B, int L, int C, int dtype, bool backward, int num_cus) {
    const size_t one = plan_recurrence(B, L, C, 1, dtype, backward, num_cus).ws_bytes;
    return C < 4 ? one : std::max(one, plan_recurrence(B, L, C, 4, dtype, backward, num_cus).ws_bytes);
}

hipError_t launch_recurrence(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    if (a.L == 0) return run_empty(a, a.state, a.last, stream);
    return by_type(a, 2 * kSlots * kPer, [&](auto t, auto n, auto odd, auto blend) {
        return run<decltype(t), decltype(n)::value, decltype(odd)::value, decltype(blend)::value>(a, num_cus, stream);
    });
}

hipError_t launch_recurrence_backward(const RecurrenceArgs &a, int num_cus, hipStream_t stream) {
    if (a.L == 0) return run_empty(a, a.g_last, a.g_state, stream);
    return by_type(a, 2 * kSlots * kPerBack, [&](auto t, auto n, auto odd, auto blend) {
        return run_back<decltype(t), decltype(n)::value, decltype(odd)::value, decltype(blend)::value>(a, num_cus, stream);
    });
}

}  // namespace dc1d
