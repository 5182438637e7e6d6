// k_attention_bwd.hip -- attention's gradients with the probabilities formed
// again from the forward's log-sum-exp.
//
//   P = exp(scale q k^T - lse),  dV = P^T g,  dP = g v^T,
//   dS = P (dP - delta),  delta = sum_d g out,
//   dQ = scale dS k,  dK = scale dS^T q
//
// Two kinds of workgroups, each with its result's rows to itself, so that nothing is
// added atomically and every call gives the same bits: one kind walks the query
// rows for a tile of keys (dK, dV; the rows are those of every query head
// that shares the key head, so their gradients add up in registers), one the
// keys for a tile of rows (dQ).  That forms S and dP twice, seven products
// for five; the alternative, dQ parts through memory for every tile of keys,
// moves more than it saves.  A first kernel forms delta.
//
// P and dS are rounded to the storage type for the next product, as operands
// of the matrix instructions have to be; everything that is added up stays
// in 32 bits.
#include "attn_tile.h"

namespace dc1d {

namespace {

// delta[b][hk][row], eight threads a row.  Bound by HBM: 4 x 4096 positions, 8
// heads of 128, bf16: 12.6 us (5.3 TB/s).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_attn_delta(AttnArgs a, uint32_t first) {
    using E = typename T::T;
    constexpr int CH = Tile<T>::CH;
    const int64_t n = (int64_t)(first + blockIdx.x) * 32 + (threadIdx.x >> 3);
    const int part = threadIdx.x & 7;
    const int64_t all = (int64_t)a.B * a.Hkv * a.rows, m = n < all ? n : all - 1;
    const uint32_t bh = (uint32_t)m / (uint32_t)a.rows, r = (uint32_t)m - bh * (uint32_t)a.rows;
    const int b = (int)(bh / (uint32_t)a.Hkv), pos = row_at(a, r).pos, h = (int)(bh % (uint32_t)a.Hkv) * a.G + row_at(a, r).head;
    const E *const g = (const E *)a.g + b * a.gs.b + pos * a.gs.l + h * a.gs.h;
    const E *const o = (const E *)a.o + b * a.os.b + pos * a.os.l + h * a.os.h;
    float s = 0.0f;
    if constexpr (VEC) {
        for (int d = part * CH; d < a.D; d += 8 * CH) {
            E ge[CH], oe[CH];
            const u32x4 gu = *(const u32x4 *)(g + d), ou = *(const u32x4 *)(o + d);
            __builtin_memcpy(ge, &gu, 16);
            __builtin_memcpy(oe, &ou, 16);
#pragma unroll
            for (int e = 0; e < CH; ++e) s += T::ld(ge, e) * T::ld(oe, e);
        }
    } else {
        for (int d = part; d < a.D; d += 8) s += T::ld(g, d) * T::ld(o, d);
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) s += __shfl_xor(s, d);
    if (part == 0 && n < all) a.delta[n] = s;
}

// A result's 16 elements as four 4-element pieces of 32 columns' rows: the
// tile (rows x DP) is passed through LDS so that rows leave in whole pieces.
// ws: this wave's 32 x (DP + 4) floats.  put(row, col, values): one piece.
template <int DP, typename Put>
__device__ __forceinline__ void drain(float *ws, const f32x16 *c, float f, int lane, Put put) {
    constexpr int P = DP + 4;
    const int half = lane >> 5;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *(f32x4 *)(ws + (lane & 31) * P + d * 32 + 8 * g + 4 * half) =
                f32x4{c[d][4 * g] * f, c[d][4 * g + 1] * f, c[d][4 * g + 2] * f, c[d][4 * g + 3] * f};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 32 * DP / 4 / 64; ++i) {
        const int p = i * 64 + lane, row = p / (DP / 4), col = p % (DP / 4) * 4;
        put(row, col, *(const f32x4 *)(ws + row * P + col));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(typename T::T *row, int col, f32x4 v, int D) {
    if constexpr (VEC) {
        if (col < D) Tile<T>::store4(row + col, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < D) T::st(row, col + e, v[e]);
    }
}

// A wave's 32 rows of an operand, held in registers: row `row`, 8 elements
// from 16 i + 8 half on.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_frags(typename Tile<T>::Frag *f, const typename T::T *row, int D, int half, bool on) {
    constexpr int CH = Tile<T>::CH;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
        u32x4 w[8 / CH];
#pragma unroll
        for (int j = 0; j < 8 / CH; ++j) {
            const int col = i * 16 + half * 8 + j * CH;
            w[j] = load_piece<T, VEC>(row, col, D);
            if (!on || (VEC && col >= D)) w[j] = u32x4{0, 0, 0, 0};
        }
        __builtin_memcpy(&f[i], w, sizeof(w));
    }
}

// ---- dK, dV ----------------------------------------------------------------------
//
// 128 keys a workgroup, 32 a wave with k in registers and v there too, or in
// LDS where two waves a SIMD would not find the registers; tiles of 32 rows
// (q, g, lse, delta) through LDS, double-buffered.  S and dP are formed with
// a lane's elements along the rows and its column a key, so that P and dS are
// operands of dV^T = g^T P and dK^T = q^T dS where they stand.
template <typename T, int DP>
struct KvShape {
    static constexpr int RT = 32;
    static constexpr size_t tile = (size_t)RT * DP;
    static constexpr bool v_lds = sizeof(typename T::T) * DP >= 256;
    static constexpr int PV = DP + Tile<T>::CH;  // rows 16 bytes apart modulo the banks
    static constexpr size_t loop_lds = 2 * (2 * tile * sizeof(typename T::T) + 4 * RT * sizeof(float)) +
                                       (v_lds ? (size_t)128 * PV * sizeof(typename T::T) : 0);
    static constexpr size_t drain_lds = (size_t)4 * 32 * (DP + 4) * sizeof(float);
    static constexpr size_t lds = loop_lds > drain_lds ? loop_lds : drain_lds;
    static constexpr int blocks = sizeof(typename T::T) * DP > 256 ? 1 : 2;
};

template <typename T, int DP, bool VEC>
__device__ __forceinline__ void key_gradients(const AttnArgs &a, char *smem, uint32_t block, uint32_t blocks) {
    using E = typename T::T;
    using M = Tile<T>;
    using S = KvShape<T, DP>;
    constexpr int RT = S::RT, NS = DP / 16, ND = DP / 32;
    E *const qbuf = (E *)smem, *const gbuf = qbuf + 2 * S::tile;
    float *const lbuf = (float *)(gbuf + 2 * S::tile), *const dbuf = lbuf + 2 * RT;
    int *const from = (int *)(dbuf + 2 * RT), *const upto = from + 2 * RT;  // the keys that each row sees
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;
    E *const vrow = (E *)(upto + 2 * RT) + (wave * 32 + (lane & 31)) * S::PV + half * 8;  // this lane's key in LDS

    const uint32_t tiles = (uint32_t)(a.Lk + 127) / 128, at_grid = xcd_order(block, blocks);
    const uint32_t id = at_grid / (uint32_t)a.splits, bh = id / tiles;
    const int split = (int)(at_grid - id * (uint32_t)a.splits);
    const int key0 = (int)(id - bh * tiles) * 128;  // causal: the longest first
    const int b = (int)(bh / (uint32_t)a.Hkv), hk = (int)(bh % (uint32_t)a.Hkv);
    const int key = key0 + wave * 32 + (lane & 31);
    const KeyRule rule = key_rule(a, b);

    // the positions [i0, i1) that see any of the workgroup's keys: those whose
    // range's ends pass key0 and the last key (both ends grow with the position)
    int i0 = 0, i1 = a.Lq;
    const int last = min(key0 + 127, rule.len - 1);
    if (last < key0) i1 = 0;
    if (rule.causal) i0 = max(i0, key0 - rule.start);
    if (rule.window) {
        i1 = min(i1, last + rule.window - rule.start);
        i0 = max(i0, key0 - rule.window + 1 - rule.start);
    }
    int64_t r0 = (int64_t)i0 * a.G / RT * RT, r1 = i1 > i0 ? (int64_t)i1 * a.G : r0;
    // this part of them
    const uint32_t n_tiles = (uint32_t)((r1 - r0 + RT - 1) / RT), per = (n_tiles + a.splits - 1) / (uint32_t)a.splits;
    r0 += min((int64_t)per * split, (int64_t)n_tiles) * RT;
    r1 = min(r1, r0 + (int64_t)per * RT);

    typename M::Frag kf[NS], vf[S::v_lds ? 1 : NS];
    {
        const int kc = min(key, a.Lk - 1);
        const E *const vp = (const E *)a.v + b * a.vs.b + hk * a.vs.h + kc * a.vs.l;
        if constexpr (S::v_lds) {  // each lane leaves what it will read itself
            load_frags<T, DP, VEC>(kf, vp, a.D, half, key < rule.len);
#pragma unroll
            for (int i = 0; i < NS; ++i) *(typename M::Frag *)(vrow + i * 16) = kf[i];
        } else {
            load_frags<T, DP, VEC>(vf, vp, a.D, half, key < rule.len);
        }
        load_frags<T, DP, VEC>(kf, (const E *)a.k + b * a.ks.b + hk * a.ks.h + kc * a.ks.l, a.D, half, key < rule.len);
    }
    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dk[d] = f32x16{}, dv[d] = f32x16{};
    const float c = a.scale * kLog2e;

    const E *const qp = (const E *)a.q + b * a.qs.b + hk * a.G * a.qs.h, *const gp = (const E *)a.g + b * a.gs.b + hk * a.G * a.gs.h;
    const float *const dp = a.delta + ((int64_t)b * a.Hkv + hk) * a.rows, *const lp = a.lse + ((int64_t)b * a.Hq + hk * a.G) * a.Lq;
    Stage<T, RT, DP, 256, VEC> qs, gs;
    qs.init_rows(a, a.qs, t);
    gs.init_rows(a, a.gs, t);
    float lse = 0.0f, del = 0.0f;
    auto load = [&](int64_t r, int at) {
        if (t < RT) {
            const int64_t n = min(r + t, a.rows - 1);
            lse = lp[(int64_t)row_at(a, n).head * a.Lq + row_at(a, n).pos];
            del = dp[n];
        }
        // rows ahead of i0 see none of the keys (some see none at all, and hold anything)
        const int skip = (int)((int64_t)i0 * a.G - r), limit = (int)min(r1 - r, (int64_t)RT);
        qs.load_rows(qbuf + at * S::tile, qp, a, a.qs, r, skip, limit, t);
        gs.load_rows(gbuf + at * S::tile, gp, a, a.gs, r, skip, limit, t);
    };
    auto store = [&](int64_t r, int at) {
        const int limit = (int)min(r1 - r, (int64_t)RT);
        if (t < RT) {
            // rows that saw nothing, or are not there, get probability 0
            lbuf[at * RT + t] = t < limit && lse != -INFINITY ? lse * kLog2e : INFINITY;
            dbuf[at * RT + t] = t < limit ? del : 0.0f;
            const KeyRange kr = rule.at(row_at(a, min(r + t, a.rows - 1)).pos);
            from[at * RT + t] = kr.lo;
            upto[at * RT + t] = kr.hi;
        }
    };
    if (r0 < r1) {
        load(r0, 0);
        store(r0, 0);
    }
    int at = 0;
    for (int64_t r = r0; r < r1; r += RT, at ^= 1) {
        landed<0>();
        __syncthreads();
        if (r + RT < r1) load(r + RT, at ^ 1);
        const E *const qt = qbuf + at * S::tile, *const gt = gbuf + at * S::tile;
        const float *const lt = lbuf + at * RT, *const dt = dbuf + at * RT;
        f32x16 s = {}, p = {};
        auto v_frag = [&](int i) {
            if constexpr (S::v_lds)
                return *(const typename M::Frag *)(vrow + i * 16);
            else
                return vf[i];
        };
        typename M::Frag qa = M::template row_frag<DP>(qt, lane & 31, half * 8), ga = M::template row_frag<DP>(gt, lane & 31, half * 8);
        typename M::Frag va = v_frag(0);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            typename M::Frag qn = qa, gn = ga, vn = va;
            if (i + 1 < NS) {
                qn = M::template row_frag<DP>(qt, lane & 31, (i + 1) * 16 + half * 8);
                gn = M::template row_frag<DP>(gt, lane & 31, (i + 1) * 16 + half * 8);
                vn = v_frag(i + 1);
            }
            reads_first<T>();
            s = M::mma(qa, kf[i], s);
            p = M::mma(ga, va, p);
            qa = qn, ga = gn, va = vn;
        }
        // does every row of the tile see every key of the wave?
        const int w0 = key0 + wave * 32;
        const bool masked = __builtin_amdgcn_readfirstlane(from[at * RT + RT - 1]) > w0 ||
                            __builtin_amdgcn_readfirstlane(upto[at * RT]) < w0 + 32;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 l4 = *(const f32x4 *)(lt + 8 * g + 4 * half), d4 = *(const f32x4 *)(dt + 8 * g + 4 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 4 * g + e;
                s[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k], c, -l4[e]));
                p[k] = s[k] * (p[k] - d4[e]);
            }
        }
        if (masked) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const i32x4 lo = *(const i32x4 *)(from + at * RT + 8 * g + 4 * half);
                const i32x4 hi = *(const i32x4 *)(upto + at * RT + 8 * g + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool sees = key >= lo[e] && key < hi[e];
                    s[4 * g + e] = sees ? s[4 * g + e] : 0.0f;
                    p[4 * g + e] = sees ? p[4 * g + e] : 0.0f;
                }
            }
        }
        const typename M::Frag p0 = M::template pack<0>(s), p1 = M::template pack<1>(s);
        const typename M::Frag s0 = M::template pack<0>(p), s1 = M::template pack<1>(p);
        add_columns<T, DP>(dv, gt, p0, p1, lane);
        add_columns<T, DP>(dk, qt, s0, s1, lane);
        if (r + RT < r1) store(r + RT, at ^ 1);
    }
    __syncthreads();
    float *const ws = (float *)smem + wave * 32 * (DP + 4);
    if (a.splits > 1) {
        const int64_t keys = (int64_t)a.B * a.Hkv * a.Lk;
        float *const pk = a.part + (((int64_t)split * 2) * keys + ((int64_t)b * a.Hkv + hk) * a.Lk + key0 + wave * 32) * DP;
        auto put = [&](float *base) {
            return [=](int row, int col, f32x4 v) {
                if (key0 + wave * 32 + row < a.Lk) *(f32x4 *)(base + (int64_t)row * DP + col) = v;
            };
        };
        drain<DP>(ws, dk, a.scale, lane, put(pk));
        drain<DP>(ws, dv, 1.0f, lane, put(pk + keys * DP));
        return;
    }
    auto put = [&](void *out, const Strides3 &st) {
        E *const base = (E *)out + b * st.b + hk * st.h + (int64_t)(key0 + wave * 32) * st.l;
        return [=](int row, int col, f32x4 v) {
            if (key0 + wave * 32 + row < a.Lk) store_piece<T, VEC>(base + row * st.l, col, v, a.D);
        };
    };
    if (a.gk) drain<DP>(ws, dk, a.scale, lane, put(a.gk, a.gks));
    if (a.gv) drain<DP>(ws, dv, 1.0f, lane, put(a.gv, a.gvs));
}

// The parts of dK and dV added in order: a thread four elements.  Bound by HBM:
// two parts of 4 x 4096 positions, 2 key heads of 128: 14.5 us (5.8 TB/s).
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(256) void k_attn_bwd_sum(AttnArgs a) {
    using E = typename T::T;
    const int64_t keys = (int64_t)a.B * a.Hkv * a.Lk, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = id / (DP / 4);
    const int col = (int)(id % (DP / 4)) * 4;
    if (n >= 2 * keys) return;
    const int which = n >= keys;
    const uint32_t m = (uint32_t)(n - (which ? keys : 0)), bh = m / (uint32_t)a.Lk, b = bh / (uint32_t)a.Hkv;
    void *const out = which ? a.gv : a.gk;
    if (!out || col >= a.D) return;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; ++s) v += *(const f32x4 *)(a.part + ((int64_t)s * 2 * keys + n) * DP + col);
    const Strides3 st = which ? a.gvs : a.gks;
    store_piece<T, VEC>((E *)out + b * st.b + (bh - b * a.Hkv) * st.h + (int64_t)(m - bh * (uint32_t)a.Lk) * st.l, col, v, a.D);
}

// ---- dQ --------------------------------------------------------------------------
//
// 128 rows a workgroup, 32 a wave with q and g in registers; tiles of KT keys
// (k, v) through LDS, double-buffered.  S^T and dP^T have a lane's elements
// along the keys and its column a row, so that dS^T is an operand of dQ^T =
// k^T dS^T where it stands, and lse and delta are one number a lane.
template <typename T, int DP>
struct QShape {
    static constexpr int KT = 32;
    static constexpr size_t tile = (size_t)KT * DP;
    static constexpr size_t loop_lds = 4 * tile * sizeof(typename T::T);
    static constexpr size_t drain_lds = (size_t)4 * 32 * (DP + 4) * sizeof(float);
    static constexpr size_t lds = loop_lds > drain_lds ? loop_lds : drain_lds;
    static constexpr int blocks = sizeof(typename T::T) * DP > 256 ? 1 : 2;
};

template <typename T, int DP, bool VEC>
__device__ __forceinline__ void query_gradients(const AttnArgs &a, char *smem, uint32_t block, uint32_t blocks) {
    using E = typename T::T;
    using M = Tile<T>;
    using S = QShape<T, DP>;
    constexpr int KT = S::KT, NS = DP / 16, ND = DP / 32;
    E *const kbuf = (E *)smem, *const vbuf = kbuf + 2 * S::tile;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, half = lane >> 5;

    const uint32_t tiles = (uint32_t)((a.rows + 127) / 128), id = xcd_order(block, blocks), bh = id / tiles;
    const uint32_t tile = tiles - 1 - (id - bh * tiles);  // causal: the longest first
    const int b = (int)(bh / (uint32_t)a.Hkv), hk = (int)(bh % (uint32_t)a.Hkv);
    const int64_t row0 = (int64_t)tile * 128, last = min(row0 + 127, a.rows - 1);
    const int64_t row = row0 + wave * 32 + (lane & 31), rc = min(row, a.rows - 1);
    const int pos = row_at(a, rc).pos, h = hk * a.G + row_at(a, rc).head;

    const KeyRule rule = key_rule(a, b);
    const KeyRange kr = rule.at(pos);
    const int lo = rule.at(row_at(a, row0).pos).lo;
    const int hi = rule.at(row_at(a, last).pos).hi;
    const KeyRange first = {__builtin_amdgcn_readfirstlane(kr.lo), __builtin_amdgcn_readfirstlane(kr.hi)};
    const KeyRange final = {__builtin_amdgcn_readlane(kr.lo, 31), __builtin_amdgcn_readlane(kr.hi, 31)};

    typename M::Frag qf[NS], gf[NS];
    load_frags<T, DP, VEC>(qf, (const E *)a.q + b * a.qs.b + pos * a.qs.l + h * a.qs.h, a.D, half, true);
    load_frags<T, DP, VEC>(gf, (const E *)a.g + b * a.gs.b + pos * a.gs.l + h * a.gs.h, a.D, half, true);
    const float raw = a.lse[((int64_t)b * a.Hq + h) * a.Lq + pos];
    const float lse = raw != -INFINITY ? raw * kLog2e : INFINITY;  // a row that saw nothing: probability 0
    const float delta = a.delta[((int64_t)b * a.Hkv + hk) * a.rows + rc];
    f32x16 dq[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = f32x16{};
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
    if (k0 < hi) load(0, k0);
    for (int at = 0; k0 < hi; k0 += KT, at ^= 1) {
        landed<0>();
        __syncthreads();
        if (k0 + KT < hi) load(at ^ 1, k0 + KT);
        if (k0 < final.hi && k0 + KT > first.lo) {
            const E *const kt = kbuf + at * S::tile, *const vt = vbuf + at * S::tile;
            f32x16 s = {}, p = {};
            typename M::Frag ka = M::template row_frag<DP>(kt, lane & 31, half * 8), va = M::template row_frag<DP>(vt, lane & 31, half * 8);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                typename M::Frag kn = ka, vn = va;
                if (i + 1 < NS) {
                    kn = M::template row_frag<DP>(kt, lane & 31, (i + 1) * 16 + half * 8);
                    vn = M::template row_frag<DP>(vt, lane & 31, (i + 1) * 16 + half * 8);
                }
                reads_first<T>();
                s = M::mma(ka, qf[i], s);
                p = M::mma(va, gf[i], p);
                ka = kn, va = vn;
            }
            const bool masked = final.lo > k0 || first.hi < k0 + KT;
#pragma unroll
            for (int r = 0; r < 16; ++r) p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -lse)) * (p[r] - delta);
            if (masked) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = k0 + 8 * (r >> 2) + 4 * half + (r & 3);
                    p[r] = j >= kr.lo && j < kr.hi ? p[r] : 0.0f;
                }
            }
            const typename M::Frag s0 = M::template pack<0>(p), s1 = M::template pack<1>(p);
            add_columns<T, DP>(dq, kt, s0, s1, lane);
        }
    }
    __syncthreads();
    E *const out = (E *)a.gq + b * a.gqs.b;
    drain<DP>((float *)smem + wave * 32 * (DP + 4), dq, a.scale, lane, [&](int r, int col, f32x4 v) {
        const int64_t n = row0 + wave * 32 + r;
        if (n >= a.rows) return;
        const int i = row_at(a, n).pos, hq = hk * a.G + row_at(a, n).head;
        store_piece<T, VEC>(out + i * a.gqs.l + hq * a.gqs.h, col, v, a.D);
    });
}

// Both in one launch: neither needs the other's result, together they fill the
// GPU where each alone would leave part of it idle (16 x 128 positions, 8
// heads of 64, fp32: 128 workgroups each on 256 CUs, 49 us one after the
// other and 28 at once), and the shorter one fills the longer one's end.
// Causal, 4 x 4096 positions, 8 heads over 2 of 128, bf16: 497 to 539 us with
// the two kernels beside it, the matrix unit 50% busy: two waves a SIMD, each
// waiting for its own chain from the scores to the gradients.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(256, (KvShape<T, DP>::blocks < QShape<T, DP>::blocks ? KvShape<T, DP>::blocks : QShape<T, DP>::blocks))
void k_attn_bwd(AttnArgs a, uint32_t kv_blocks, uint32_t q_blocks, uint32_t first, int keys_first) {
    extern __shared__ __align__(512) char smem[];
    const uint32_t id = first + blockIdx.x, kv0 = keys_first ? 0 : q_blocks, q0 = keys_first ? kv_blocks : 0;
    if (id - kv0 < kv_blocks)
        key_gradients<T, DP, VEC>(a, smem, id - kv0, kv_blocks);
    else
        query_gradients<T, DP, VEC>(a, smem, id - q0, q_blocks);
}

// As in the forward: causal 8 x 2048 positions, 8 heads of 64, 80, 96 and 128,
// bf16: 234, 310, 315 and 314 us.
int padded(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }

// A launch holds fewer than 2^32 threads; within the documented sizes the
// key and query workgroups are up to three times that.
template <typename Launch>
void in_parts(int64_t blocks, Launch launch) {
    constexpr int64_t most = 1 << 23;  // a multiple of the XCDs, which xcd_order() counts on
    for (int64_t first = 0; first < blocks; first += most)
        launch((uint32_t)first, dim3((uint32_t)(blocks - first < most ? blocks - first : most)));
}

template <typename T, int DP, bool VEC>
hipError_t launch(const AttnArgs &a, hipStream_t stream) {
    constexpr size_t q_lds = QShape<T, DP>::lds, kv_lds = KvShape<T, DP>::lds;
    const int64_t heads = (int64_t)a.B * a.Hkv;
    const int64_t kv_blocks = a.gk || a.gv ? heads * ((a.Lk + 127) / 128) * a.splits : 0;
    const int64_t q_blocks = a.gq ? heads * ((a.rows + 127) / 128) : 0;
    if (kv_blocks + q_blocks == 0) return hipSuccess;
    in_parts((heads * a.rows + 31) / 32, [&](uint32_t first, dim3 grid) {
        hipLaunchKernelGGL((k_attn_delta<T, VEC>), grid, dim3(256), 0, stream, a, first);
    });
    const int keys_first = 4 * (a.rows / a.splits) >= 3 * (int64_t)a.Lk;  // the longer workgroups: 4 and 3 products a tile
    in_parts(kv_blocks + q_blocks, [&](uint32_t first, dim3 grid) {
        hipLaunchKernelGGL((k_attn_bwd<T, DP, VEC>), grid, dim3(256), q_lds > kv_lds ? q_lds : kv_lds, stream, a, (uint32_t)kv_blocks,
                           (uint32_t)q_blocks, first, keys_first);
    });
    if (kv_blocks > 0 && a.splits > 1)
        hipLaunchKernelGGL((k_attn_bwd_sum<T, DP, VEC>), dim3((uint32_t)((2 * heads * a.Lk * (DP / 4) + 255) / 256)),
                           dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(const AttnArgs &a, hipStream_t stream) {
    const int DP = padded(a.D);
    if (DP == 32) return a.vec ? launch<T, 32, true>(a, stream) : launch<T, 32, false>(a, stream);
    if (DP == 64) return a.vec ? launch<T, 64, true>(a, stream) : launch<T, 64, false>(a, stream);
    return a.vec ? launch<T, 128, true>(a, stream) : launch<T, 128, false>(a, stream);
}

}  // namespace

AttnBwdPlan plan_attention_backward(const AttnArgs &a, int num_cus) {
    AttnBwdPlan pl = {};
    const int64_t heads = (int64_t)a.B * a.Hkv, blocks = heads * ((a.Lk + 127) / 128);
    // Parts of the rows: enough workgroups that a causal call's uneven ones even
    // out (two to a CU; 4 x 4096 positions, 2 key heads: 1012 us unsplit, 498 in
    // two parts, 510 in four), none with fewer than 512 rows: the parts' sums cost
    // more than they save where the query workgroups already share the GPU (4 x
    // 512 positions, 8 heads of 64, fp32: 86 us whole, 97 in four parts).  Parts
    // of 256 or 128 rows only while every workgroup, those of the queries too,
    // still has a CU to itself (8 heads over 2 of 128: 2 x 256 positions, bf16,
    // 37 and 26 us; 13 x 136, 4 over 1, fp32, 99 and 57 us).
    int64_t splits = blocks > 0 ? (2 * (int64_t)num_cus + blocks - 1) / blocks : 1;
    const int64_t q_blocks = heads * ((a.rows + 127) / 128);
    int64_t least = 512;
    for (int64_t rows = 256; rows >= 128; rows /= 2)
        if (blocks * ((a.rows + rows - 1) / rows) + q_blocks <= num_cus) least = rows;
    const int64_t most = (a.rows + least - 1) / least;
    splits = splits > most ? most : splits;
    pl.splits = (int)(splits < 1 ? 1 : splits > 16 ? 16 : splits);
    pl.delta_bytes = ((size_t)heads * a.rows * sizeof(float) + 255) / 256 * 256;
    pl.ws_bytes = pl.delta_bytes;
    if (pl.splits > 1) pl.ws_bytes += (size_t)pl.splits * 2 * heads * a.Lk * padded(a.D) * sizeof(float);
    return pl;
}

hipError_t launch_attention_backward(AttnArgs a, const AttnBwdPlan &pl, void *ws, hipStream_t stream) {
    a.splits = pl.splits;
    a.delta = (float *)ws;
    a.part = (float *)((char *)ws + pl.delta_bytes);
    return a.dtype == kF32 ? launch_typed<F32>(a, stream) : launch_typed<BF16>(a, stream);
}

}  // namespace dc1d
