// k_attention.hip -- attention's forward pass in one sweep over the keys,
// with the running maximum and sum of the softmax.
//
// A workgroup takes rows of one key head (the query rows of all the query
// heads that share it) and walks the keys that they see in tiles staged
// through LDS.  Scores are formed transposed, S^T = K Q^T, so that a lane's
// 16 scores of a tile belong to one row: its maximum and sum need one
// exchange with lane ^ 32, and the probabilities stand where the next
// product, O^T = V^T P^T, wants its operand.
//
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j     (s in units of log 2)
//
// out = o / l, lse = m + log l.  A row that sees no key keeps l = 0: out 0,
// lse -infinity.
//
// The probabilities of a bf16 call are rounded to bf16 for the second product,
// as operands of its matrix instructions have to be (fp32 calls keep fp32
// ones); m, l, o and the parts' sums are in 32 bits.  8 x 4096 positions, 8 heads
// of 64: 0.0023 off 64-bit values, where one rounding of the exact result is
// 0.0017.
#include <type_traits>

#include "attn_tile.h"

namespace dc1d {

namespace {

constexpr int kMaxParts = 128;  // of the keys: lanes of k_attn_join times two

// Rows of the softmax that a lane carries (row lane % 32 of its wave; the
// two halves hold the same maximum and each its own part of the sum).
struct Softmax {
    float m, l;  // maximum in units of log 2 (-inf: nothing seen), part of the sum
};

// The scores S^T = K Q^T of 32 * NT keys (first key k0), in place of those
// that a lane's row does not see -infinity.  masked: some lane's range cuts
// the tile.
template <typename T, int DP, int NT>
__device__ __forceinline__ void scores(f32x16 *s, const typename T::T *kt, const typename Tile<T>::Frag *q, bool masked, int k0,
                                       KeyRange kr, int lane) {
    using M = Tile<T>;
    constexpr int NS = DP / 16;
    const int half = lane >> 5;
    typename M::Frag ka = M::template row_frag<DP>(kt, lane & 31, half * 8);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        s[t] = f32x16{};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            typename M::Frag kn = ka;
            if (i + 1 < NS)
                kn = M::template row_frag<DP>(kt, t * 32 + (lane & 31), (i + 1) * 16 + half * 8);
            else if (t + 1 < NT)
                kn = M::template row_frag<DP>(kt, (t + 1) * 32 + (lane & 31), half * 8);
            reads_first<T>();
            s[t] = M::mma(ka, q[i], s[t]);
            ka = kn;
        }
    }
    if (masked) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int j = k0 + t * 32 + 8 * (r >> 2) + 4 * half + (r & 3);
                s[t][r] = j >= kr.lo && j < kr.hi ? s[t][r] : -INFINITY;
            }
    }
}

// Scores into probabilities against the running maximum, which they may move.
template <int DP, int NT>
__device__ __forceinline__ void soften(f32x16 *s, f32x16 *o, Softmax &sm, float c) {
    constexpr int ND = DP / 32;
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
    top = half_max(top) * c;
    // The reference that the exponents are taken from moves only when the
    // maximum has outgrown it by a factor of 2^8: sums of that size lose
    // nothing in 32 bits, and rescaling o is rare.
    if (__any(top > sm.m + 8.0f)) {
        const float m = fmaxf(sm.m, top);
        const float alpha = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm.m - m);
        sm.m = m;
        sm.l *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= alpha;
    }
    const float m = sm.m == -INFINITY ? 0.0f : sm.m;
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -m));
            sum += s[t][r];
        }
    sm.l += sum;
}

// o^T += V^T P^T, V the tile OFF elements on
template <typename T, int DP, int NT, int OFF>
__device__ __forceinline__ void add_values(f32x16 *o, const typename T::T *vt, const f32x16 *s, int lane) {
    using M = Tile<T>;
    static_assert(NT <= 2, "up to 64 keys");
    add_columns<T, DP, OFF, 0>(o, vt, M::template pack<0>(s[0]), M::template pack<1>(s[0]), lane);
    if constexpr (NT > 1) add_columns<T, DP, OFF, 32>(o, vt, M::template pack<0>(s[1]), M::template pack<1>(s[1]), lane);
}

// 16 elements of a row's 32 d's in a result's order, times f.
template <typename T, bool VEC>
__device__ __forceinline__ void store_row(typename T::T *row, const f32x16 &o, float f, int d0, int half, int D) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int d = d0 + 8 * g + 4 * half;
        const f32x4 v = {o[4 * g] * f, o[4 * g + 1] * f, o[4 * g + 2] * f, o[4 * g + 3] * f};
        if constexpr (VEC) {
            if (d < D) Tile<T>::store4(row + d, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D) T::st(row, d + e, v[e]);
        }
    }
}

template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_q(const AttnArgs &a, typename Tile<T>::Frag *q, int b, int hk, int64_t row, int half) {
    constexpr int CH = Tile<T>::CH;
    const int pos = row_at(a, row).pos, h = hk * a.G + row_at(a, row).head;
    const typename T::T *p = (const typename T::T *)a.q + b * a.qs.b + pos * a.qs.l + h * a.qs.h;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
        u32x4 w[8 / CH];
#pragma unroll
        for (int j = 0; j < 8 / CH; ++j) {
            const int col = i * 16 + half * 8 + j * CH;
            w[j] = load_piece<T, VEC>(p, col, a.D);
            if (VEC && col >= a.D) w[j] = u32x4{0, 0, 0, 0};
        }
        __builtin_memcpy(&q[i], w, sizeof(w));
    }
}

// ---- rows split among the waves ---------------------------------------------
//
// 128 rows a workgroup, 32 a wave; tiles of KT keys, double-buffered, the
// next one on its way while this one is used.  8 x 4096 positions, 8 heads of
// 64, bf16: 300 to 326 us (0.84 to 0.9 PFLOP/s, by the card), bound by the vector
// instructions of the softmax (matrix unit 48% busy); 4 x 4096, 8 heads of 128:
// 263 us (1.05), causal over 2 key heads 144 us (0.96).
template <typename T, int DP>
struct RowsShape {
    static constexpr int KT = sizeof(typename T::T) == 2 ? 64 : 32;
    static constexpr int tile = KT * DP;
    static constexpr size_t lds = (size_t)4 * tile * sizeof(typename T::T);
    static constexpr int blocks = sizeof(typename T::T) * DP == 128 ? 4 : 2;  // a CU; bf16, D 64: 312 -> 307 us for four
};

template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(256, (RowsShape<T, DP>::blocks)) void k_attn_rows(AttnArgs a) {
    using E = typename T::T;
    using S = RowsShape<T, DP>;
    constexpr int KT = S::KT, ND = DP / 32;
    extern __shared__ __align__(512) char smem[];
    E *const kbuf = (E *)smem, *const vbuf = kbuf + 2 * S::tile;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;

    const uint32_t tiles = (uint32_t)((a.rows + 127) / 128), id = xcd_order(blockIdx.x, gridDim.x), bh = id / tiles;
    const uint32_t tile = tiles - 1 - (id - bh * tiles);  // causal: the longest first
    const int b = (int)(bh / (uint32_t)a.Hkv), hk = (int)(bh % (uint32_t)a.Hkv);
    const int64_t row0 = (int64_t)tile * 128;
    const int64_t last = min(row0 + 127, a.rows - 1);
    const int64_t row = row0 + wave * 32 + (lane & 31), rc = min(row, a.rows - 1);

    const KeyRule rule = key_rule(a, b);
    const KeyRange kr = rule.at(row_at(a, rc).pos);
    // the ranges' ends grow with the position, so the first and last row bound them
    const int lo = rule.at(row_at(a, row0).pos).lo;
    const int hi = rule.at(row_at(a, last).pos).hi;
    const KeyRange first = {__builtin_amdgcn_readfirstlane(kr.lo), __builtin_amdgcn_readfirstlane(kr.hi)};
    const KeyRange final = {__builtin_amdgcn_readlane(kr.lo, 31), __builtin_amdgcn_readlane(kr.hi, 31)};

    typename Tile<T>::Frag q[DP / 16];
    load_q<T, DP, VEC>(a, q, b, hk, rc, half);
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
    Softmax sm = {-INFINITY, 0.0f};
    const float c = a.scale * kLog2e;

    const E *const kp = (const E *)a.k + b * a.ks.b + hk * a.ks.h, *const vp = (const E *)a.v + b * a.vs.b + hk * a.vs.h;
    Stage<T, KT, DP, 256, VEC> ks, vs;
    ks.init(a.ks.l, t);
    vs.init(a.vs.l, t);
    ks.near = vs.near = ks.near && vs.near;
    auto load = [&](int at, int k0) {
        ks.load(kbuf + at * S::tile, kp + k0 * a.ks.l, a.ks.l, lo - k0, hi - k0, a.D, t);
        vs.load(vbuf + at * S::tile, vp + k0 * a.vs.l, a.vs.l, lo - k0, hi - k0, a.D, t);
    };
    int k0 = lo / KT * KT;
    // one tile: the buffer it stands in is a constant, so that every read's
    // address is one that the lane keeps plus a constant
    auto step = [&](auto at) {
        constexpr int AT = decltype(at)::value;
        landed<0>();
        __syncthreads();
        if (k0 + KT < hi) load(AT ^ 1, k0 + KT);
        if (k0 < final.hi && k0 + KT > first.lo) {
            f32x16 s[KT / 32];
            scores<T, DP, KT / 32>(s, kbuf + AT * S::tile, q, final.lo > k0 || first.hi < k0 + KT, k0, kr, lane);
            soften<DP, KT / 32>(s, o, sm, c);
            // this wave's products before another's exponentials: the matrix unit
            // is the one to keep busy (D 128: 274 -> 263 us)
            __builtin_amdgcn_s_setprio(1);
            add_values<T, DP, KT / 32, AT * S::tile>(o, vbuf, s, lane);
            __builtin_amdgcn_s_setprio(0);
        }
        k0 += KT;
    };
    if (k0 < hi) load(0, k0);
    while (k0 < hi) {
        step(std::integral_constant<int, 0>{});
        if (k0 >= hi) break;
        step(std::integral_constant<int, 1>{});
    }

    const float l = half_sum(sm.l);
    if (row >= a.rows) return;
    const int pos = row_at(a, row).pos, h = hk * a.G + row_at(a, row).head;
    E *const op = (E *)a.out + b * a.os.b + pos * a.os.l + h * a.os.h;
    const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // a NaN stays one
#pragma unroll
    for (int d = 0; d < ND; ++d) store_row<T, VEC>(op, o[d], f, d * 32, half, a.D);
    if (a.lse && half == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.Lq + pos] = l == 0.0f ? -INFINITY : sm.m * kLn2 + __logf(l);
}

// ---- keys split among the waves -----------------------------------------------
//
// 32 rows a workgroup (one or a few positions of every query head of the key
// head); each wave stages and uses its own tiles of 32 keys, every fourth one
// of the workgroup's part of the keys, with no barrier between them, so the
// keys and values stream.  The waves' results are joined through LDS; where
// the keys are also split among workgroups (`splits`) each part leaves its
// maximum, sum and unscaled o, and k_attn_join adds the parts in order.  Single
// positions are bound by HBM: 16 sequences of up to 16384 keys, 2 key heads of
// 128, bf16: 39 us (4.5 TB/s).
template <typename T, int DP>
struct KeysShape {
    static constexpr int KT = 32;
    static constexpr int tile = KT * DP, PO = DP + 4;
    static constexpr size_t wave_lds = (size_t)2 * tile * sizeof(typename T::T);
    static constexpr size_t join_lds = (size_t)4 * 32 * (PO + 2) * sizeof(float);
    static constexpr size_t lds = 4 * wave_lds > join_lds ? 4 * wave_lds : join_lds;
};

template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(256, (KeysShape<T, DP>::lds > 80 << 10 ? 1 : 2)) void k_attn_keys(AttnArgs a) {
    using E = typename T::T;
    using S = KeysShape<T, DP>;
    constexpr int KT = S::KT, ND = DP / 32;
    extern __shared__ __align__(512) char smem[];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;
    E *const kbuf = (E *)(smem + wave * S::wave_lds), *const vbuf = kbuf + S::tile;

    const uint32_t tiles = (uint32_t)((a.rows + 31) / 32);
    // several tiles of rows read the same keys, and share an L2; with one the
    // workgroups are spread, so that no XCD gets only long sequences
    const uint32_t at_grid = tiles > 1 ? xcd_order(blockIdx.x, gridDim.x) : blockIdx.x;
    const uint32_t id = at_grid / (uint32_t)a.splits, bh = id / tiles;
    const int split = (int)(at_grid - id * (uint32_t)a.splits);
    const int64_t row0 = (int64_t)(id - bh * tiles) * 32;
    const int b = (int)(bh / (uint32_t)a.Hkv), hk = (int)(bh % (uint32_t)a.Hkv);
    const int64_t last = min(row0 + 31, a.rows - 1);
    const int64_t row = row0 + (lane & 31), rc = min(row, a.rows - 1);

    const KeyRule rule = key_rule(a, b);
    const KeyRange kr = rule.at(row_at(a, rc).pos);
    const KeyRange first = rule.at(row_at(a, row0).pos);
    const KeyRange final = rule.at(row_at(a, last).pos);

    typename Tile<T>::Frag q[DP / 16];
    load_q<T, DP, VEC>(a, q, b, hk, rc, half);
    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = f32x16{};
    Softmax sm = {-INFINITY, 0.0f};
    const float c = a.scale * kLog2e;

    // this part's run of the tiles [t0, t1) that the rows see: parts are of one
    // length, so that a short sequence's later parts end at once
    const int t0 = first.lo / KT, t1 = final.hi > first.lo ? (final.hi + KT - 1) / KT : t0;
    const int s0 = (int)min(t0 + (int64_t)a.part_tiles * split, (int64_t)t1), s1 = (int)min(s0 + (int64_t)a.part_tiles, (int64_t)t1);

    const E *const kp = (const E *)a.k + b * a.ks.b + hk * a.ks.h, *const vp = (const E *)a.v + b * a.vs.b + hk * a.vs.h;
    Stage<T, KT, DP, 64, VEC> ks, vs;
    ks.init(a.ks.l, lane);
    vs.init(a.vs.l, lane);
    ks.near = vs.near = ks.near && vs.near;
    auto load_k = [&](int n) {
        ks.load(kbuf, kp + (int64_t)n * KT * a.ks.l, a.ks.l, first.lo - n * KT, final.hi - n * KT, a.D, lane);
    };
    auto load_v = [&](int n) {
        vs.load(vbuf, vp + (int64_t)n * KT * a.vs.l, a.vs.l, first.lo - n * KT, final.hi - n * KT, a.D, lane);
    };
    constexpr int LOADS = decltype(ks)::N;  // of one tile, in flight where the rows are near
    int n = s0 + wave;
    if (n < s1) {
        load_k(n);
        load_v(n);
    }
    for (; n < s1; n += 4) {
        const int k0 = n * KT;
        const bool more = n + 4 < s1;
        f32x16 s[1];
        landed<LOADS>();  // the keys; the values follow
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        scores<T, DP, 1>(s, kbuf, q, final.lo > k0 || first.hi < k0 + KT, k0, kr, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (more) load_k(n + 4);  // over the keys just used
        soften<DP, 1>(s, o, sm, c);
        if (more)
            landed<LOADS>();  // the values; the next keys follow
        else
            landed<0>();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        add_values<T, DP, 1, 0>(o, vbuf, s, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (more) load_v(n + 4);
    }

    // join the four waves: each leaves o, m, l; thread (row, slice) adds them in wave order
    __syncthreads();
    float *const of = (float *)smem, *const ml = of + 4 * 32 * S::PO;
    const float l = half_sum(sm.l);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *(f32x4 *)(of + (wave * 32 + (lane & 31)) * S::PO + d * 32 + 8 * g + 4 * half) =
                f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    if (half == 0) {
        ml[(wave * 32 + lane) * 2] = sm.m;
        ml[(wave * 32 + lane) * 2 + 1] = l;
    }
    __syncthreads();
    const int r = t >> 3, slice = t & 7;  // eight threads a row
    const int64_t n_row = row0 + r;
    if (n_row >= a.rows) return;
    float m = -INFINITY, w[4], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, ml[(i * 32 + r) * 2]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float mi = ml[(i * 32 + r) * 2];
        w[i] = mi == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mi - m);
        sum += w[i] * ml[(i * 32 + r) * 2 + 1];
    }
    const int pos = row_at(a, n_row).pos, h = hk * a.G + row_at(a, n_row).head;
    const float f = a.splits > 1 ? 1.0f : sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    E *const op = (E *)a.out + b * a.os.b + pos * a.os.l + h * a.os.h;
    const int64_t at = ((int64_t)b * a.Hkv + hk) * a.rows + n_row, all = (int64_t)a.B * a.Hkv * a.rows;
    float *const pp = a.splits > 1 ? a.part + ((int64_t)split * all + at) * (DP + 2) : nullptr;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
        const int d = j * 32 + slice * 4;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) v += w[i] * *(const f32x4 *)(of + (i * 32 + r) * S::PO + d);
        v *= f;
        if (pp) {
#pragma unroll
            for (int e = 0; e < 4; ++e) pp[2 + d + e] = v[e];
        } else if constexpr (VEC) {
            if (d < a.D) Tile<T>::store4(op + d, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < a.D) T::st(op, d + e, v[e]);
        }
    }
    if (slice == 0) {
        if (pp) {
            pp[0] = m;
            pp[1] = sum;
        } else if (a.lse) {
            a.lse[((int64_t)b * a.Hq + h) * a.Lq + pos] = sum == 0.0f ? -INFINITY : m * kLn2 + __logf(sum);
        }
    }
}

// The parts of a row joined, a workgroup a row: every wave forms the parts'
// weights (a lane a part), adds up every fourth part, and the waves' sums are
// added in wave order.  The same 16 sequences: 5 us, mostly latency.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    using E = typename T::T;
    constexpr int NV = (DP + 63) / 64, PL = kMaxParts / 64;
    __shared__ float sums[4][DP], weight[kMaxParts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t all = (int64_t)a.B * a.Hkv * a.rows, at = blockIdx.x, step = all * (DP + 2);
    const float *const p = a.part + at * (DP + 2);
    float w[PL], l[PL], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int s = i * 64 + lane;
        w[i] = s < a.splits ? p[s * step] : -INFINITY;
        l[i] = s < a.splits ? p[s * step + 1] : 0.0f;
        m = fmaxf(m, w[i]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        w[i] = w[i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(w[i] - m);
        sum += w[i] * l[i];
        if (wave == 0) weight[i * 64 + lane] = w[i];
    }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    float v[NV] = {};
#pragma unroll 4
    for (int s = wave; s < a.splits; s += 4) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * 64 + lane < DP) v[j] += weight[s] * p[s * step + 2 + j * 64 + lane];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (j * 64 + lane < DP) sums[wave][j * 64 + lane] = v[j];
    __syncthreads();
    const uint32_t bh = (uint32_t)at / (uint32_t)a.rows;
    const RowAt r = row_at(a, (uint32_t)at - bh * (uint32_t)a.rows);
    const int b = (int)(bh / (uint32_t)a.Hkv), h = (int)(bh % (uint32_t)a.Hkv) * a.G + r.head;
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    if ((int)threadIdx.x < a.D) {
        const int d = threadIdx.x;
        const float o = sums[0][d] + sums[1][d] + sums[2][d] + sums[3][d];
        T::st((E *)a.out + b * a.os.b + r.pos * a.os.l + h * a.os.h, d, o * f);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.Lq + r.pos] = sum == 0.0f ? -INFINITY : m * kLn2 + __logf(sum);
}

// A tile's row and the products' length.  D between two of them pays for the
// larger: causal 8 x 2048 positions, 8 heads of 80, 96 and 128, bf16: 101, 102 and
// 97 us (64: 75).
int padded(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }

template <typename T, int DP, bool VEC>
hipError_t launch(const AttnArgs &a, const AttnPlan &pl, hipStream_t stream) {
    if (!pl.by_keys) {
        constexpr size_t lds = RowsShape<T, DP>::lds;
        hipLaunchKernelGGL((k_attn_rows<T, DP, VEC>), dim3((uint32_t)pl.blocks), dim3(256), lds, stream, a);
        return hipGetLastError();
    }
    constexpr size_t lds = KeysShape<T, DP>::lds;
    hipLaunchKernelGGL((k_attn_keys<T, DP, VEC>), dim3((uint32_t)pl.blocks), dim3(256), lds, stream, a);
    if (a.splits > 1)
        hipLaunchKernelGGL((k_attn_join<T, DP>), dim3((uint32_t)((int64_t)a.B * a.Hkv * a.rows)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(const AttnArgs &a, const AttnPlan &pl, hipStream_t stream) {
    const int DP = padded(a.D);
    if (DP == 32) return a.vec ? launch<T, 32, true>(a, pl, stream) : launch<T, 32, false>(a, pl, stream);
    if (DP == 64) return a.vec ? launch<T, 64, true>(a, pl, stream) : launch<T, 64, false>(a, pl, stream);
    return a.vec ? launch<T, 128, true>(a, pl, stream) : launch<T, 128, false>(a, pl, stream);
}

}  // namespace

AttnPlan plan_attention(const AttnArgs &a, int num_cus) {
    AttnPlan pl = {};
    const int64_t heads = (int64_t)a.B * a.Hkv, row_blocks = heads * ((a.rows + 127) / 128);
    // While workgroups of 128 rows leave CUs empty, four times as many of 32
    // rows finish sooner though each reads all the keys: 8 heads of 64 over 2048
    // positions, bf16, 128 and 512 workgroups: 36 and 25 us (fp32, 1024
    // positions: 87 and 28).  From one workgroup a CU on the wider ones win:
    // two such sequences, 256 and 1024 workgroups: 38 and 42 us.
    pl.by_keys = a.rows <= 32 || row_blocks < num_cus;
    pl.splits = 1;
    if (!pl.by_keys) {
        pl.name = "attention_rows";
        pl.blocks = row_blocks;
        return pl;
    }
    pl.name = "attention_keys";
    const int64_t blocks = heads * ((a.rows + 31) / 32);
    if (blocks == 0) return pl;
    // the most tiles of 32 keys that a tile of rows can see: its rows are of at
    // most 31 / G + 2 neighbouring positions
    int64_t tiles = a.Lk > 0 ? ((int64_t)a.Lk + 31) / 32 : 1;
    if (a.window) {
        const int64_t seen = a.window + (a.causal ? 0 : a.window) + 31 / a.G + 2, few = (seen + 31) / 32 + 1;
        tiles = tiles < few ? tiles : few;
    }
    // where there are fewer than CUs, enough for two on each, none with fewer
    // than 8 tiles
    const int64_t most = tiles / 8 > 1 ? tiles / 8 : 1;
    int64_t splits = blocks >= num_cus ? 1 : (2 * (int64_t)num_cus + blocks - 1) / blocks;
    splits = splits > most ? most : splits;
    splits = splits < 1 ? 1 : splits > kMaxParts ? kMaxParts : splits;
    // the workspace is sized before the parts are made a multiple of the four
    // waves' tiles: it then never grows where a window leaves fewer tiles, and
    // can be asked for without one
    if (splits > 1) pl.ws_bytes = (size_t)splits * heads * a.rows * (padded(a.D) + 2) * sizeof(float);
    pl.part_tiles = (int)(((tiles + splits - 1) / splits + 3) / 4 * 4);
    pl.splits = (int)((tiles + pl.part_tiles - 1) / pl.part_tiles);
    pl.blocks = blocks * pl.splits;
    return pl;
}

hipError_t launch_attention(AttnArgs a, const AttnPlan &pl, void *ws, hipStream_t stream) {
    a.splits = pl.splits;
    a.part_tiles = pl.part_tiles;
    a.part = (float *)ws;
    if (pl.blocks == 0) return hipSuccess;
    return a.dtype == kF32 ? launch_typed<F32>(a, pl, stream) : launch_typed<BF16>(a, pl, stream);
}

}  // namespace dc1d
