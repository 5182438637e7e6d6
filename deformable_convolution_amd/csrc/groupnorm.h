// groupnorm.h -- what group norm's kernels and those of its gradients share: the
// activations, samples held by a workgroup, samples in parts.
#pragma once

#include <algorithm>
#include <type_traits>

#include "vec16.h"

namespace dc1d {

enum Act { kNone = 0, kRelu = 1, kSilu = 2 };

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kRelu) return z < 0.0f ? 0.0f : z;  // a NaN stays
    if constexpr (ACT == kSilu) return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
    return z;
}
// The gradient g of act(z) taken to z.  silu: p (1 + z (1 - p)), p = 1 / (1 + exp(-z));
// 1 - p is off by 2^-24, which counts z times beside 1.
template <int ACT>
__device__ __forceinline__ float activate_back(float z, float g) {
    if constexpr (ACT == kRelu) return z > 0.0f ? g : 0.0f;
    if constexpr (ACT == kSilu) {
        const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
        return g * (p * fmaf(z, 1.0f - p, 1.0f));
    }
    return g;
}

// A sample's positions that count.
__device__ __forceinline__ int64_t positions(const GroupNormArgs &a, int64_t b) {
    if (!a.lens) return a.S;
    const int n = a.lens[b];
    return n < 0 ? 0 : n < a.S ? n : a.S;
}

// ---- held samples ------------------------------------------------------------------
//
// A workgroup holds the positions of nb samples times a slab of gs groups in
// registers: x (and g) are read once.  Its threads are nb samples x rt rows x P
// pieces of the slab's channels, R rows each (row t, t + rt, ...).  The mean is
// taken first, then the squares about it and what it leaves (a sum of differences,
// which corrects both), all from registers.
//
// Samples that fit are held (odd groups with exceptions, see plan_held): against
// parts, which read twice, 32 x 784 x 512 fp32 takes 22 us (34), 4 x 4096 x 512 bf16
// 21 (29), 32768 rows of 1024 bf16 33 (325), gradients 43 (55) and 48 to 52 (456).
struct HeldPlan {
    int P, gs, slabs, rt, nb, nt, R;
    int64_t batches;       // of nb samples
    int grid_rows;         // backward: workgroups of a slab
    int per, team;         // a group's partial sums in LDS a row of threads; lanes that add them
    int mode;
    FastDiv by_P, by_rt, by_per, by_gs, by_D;
    size_t lds;
};
// A group's lanes share a wave; a piece lies in one group; the slab is one group,
// whose last piece repeats some of it (as if it were several, 11031 rows of 890
// bf16 took 42 us, not 19; gradients 60, not 28); a piece may lie in several.
enum Mode { kShuffle, kWhole, kOne, kMixed };

// The sums of v over every group of a workgroup: [K] values for each of a
// thread's NV groups, K up to 2.
template <int N, int MODE>
struct GroupSums {
    static constexpr int NV = MODE == kMixed ? N : 1;
    float *sums, *red;
    int np;
    __device__ __forceinline__ GroupSums(const HeldPlan &p, float *lds) : sums(lds), red(lds + 2 * p.nb * p.gs), np(p.nb * p.gs) {}
    // channels: of the slab; slot: where the first of a thread's groups is among np (its sample's, for kMixed)
    template <int K>
    __device__ __forceinline__ void operator()(const HeldPlan &p, float (&v)[K][NV], int channels, int D, int slot, const int *of) {
        if constexpr (MODE == kShuffle) {
            for (int d = 1; d < p.per; d <<= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k][0] += __shfl_xor(v[k][0], d);
        } else {
            using Sums = float __attribute__((ext_vector_type(K)));  // of one group, side by side: one access for both
            Sums *const own = (Sums *)red, *const all_of = (Sums *)sums;
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                Sums s;
#pragma unroll
                for (int k = 0; k < K; ++k) s[k] = v[k][e];
                own[threadIdx.x * NV + e] = s;
            }
            __syncthreads();
            const int lane = threadIdx.x & (p.team - 1), all = p.rt * p.per, last = (channels + N - 1) / N - 1;
            for (int g = threadIdx.x / p.team; g < np; g += p.nt / p.team) {
                const int sm = (int)fdiv(g, p.by_gs), first = (g - sm * p.gs) * p.per;
                Sums s = {};
                for (int i = lane; i < all; i += p.team) {
                    const int r = (int)fdiv(i, p.by_per), j = first + i - r * p.per;
                    int at;
                    if constexpr (MODE != kMixed) {
                        at = j;
                    } else {
                        if (j >= channels) break;  // the last slab's groups are fewer
                        at = j >= last * N ? last * N + j - (channels - N) : j;
                    }
                    at += (sm * p.rt + r) * p.P * NV;
                    s += own[at];
                }
                for (int d = 1; d < p.team; d <<= 1)
#pragma unroll
                    for (int k = 0; k < K; ++k) s[k] += __shfl_xor(s[k], d);
                if (lane == 0) all_of[g] = s;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const Sums s = all_of[slot + (MODE == kMixed ? of[e] : 0)];
#pragma unroll
                for (int k = 0; k < K; ++k) v[k][e] = s[k];
            }
        }
    }
};

// Workgroup i runs on XCD i % 8, which has an L2 of its own: neighbouring numbers
// (slabs whose rows share lines) to one XCD.
__device__ __forceinline__ uint32_t by_xcd(uint32_t i, uint32_t n) {
    const uint32_t x = i & 7, q = n >> 3, r = n & 7;
    return x * q + min(x, r) + (i >> 3);
}

// A thread's place among the samples and channels of a workgroup.
template <int N, int MODE>
struct HeldPlace {
    static constexpr int NV = MODE == kMixed ? N : 1;
    int rt, sm, at, skip, channels, group, slot, of[NV];  // group: of the piece's first element, or the slab's; of: its elements', from there
    bool in;                                               // a piece of the slab
    __device__ __forceinline__ HeldPlace(const GroupNormArgs &a, const HeldPlan &p, int slab) {
        const int q = (int)fdiv(threadIdx.x, p.by_P), j = threadIdx.x - q * p.P;
        sm = (int)fdiv(q, p.by_rt);
        rt = q - sm * p.rt;
        const int g0 = slab * p.gs, c0 = g0 * a.D, end = min(c0 + p.gs * a.D, a.C), c = c0 + j * N;
        channels = end - c0;
        in = c < end && sm < p.nb;
        at = in ? min(c, end - N) : c0 + N <= a.C ? c0 : a.C - N;
        skip = in ? c - at : N;
        sm = min(sm, p.nb - 1);
        if constexpr (MODE == kMixed) {
            group = g0;
            slot = sm * p.gs;
#pragma unroll
            for (int e = 0; e < N; ++e) of[e] = max((int)fdiv(at + e, p.by_D) - g0, 0);
        } else {
            group = (int)fdiv(at, p.by_D);
            slot = sm * p.gs + group - g0;
            of[0] = 0;
        }
    }
    __device__ __forceinline__ int v(int e) const { return MODE == kMixed ? e : 0; }
    // Bytes from the batch's first element to row i of the thread's in sample `s` of
    // the batch; the sample's first row in place of those that are not read.
    __device__ __forceinline__ uint32_t offset(const GroupNormArgs &a, const HeldPlan &p, int es, int s, int i, bool there) const {
        const uint32_t row = (uint32_t)(s * (int)a.S) + (there ? (uint32_t)(rt + i * p.rt) : 0u);
        return (row * (uint32_t)a.C + (uint32_t)at) * (uint32_t)es;
    }
};
template <typename T, int N, int MODE>
__device__ __forceinline__ void put(char *p, const float *f, int skip, bool in_place) {
    if constexpr (MODE == kMixed)
        store_own<T, N>((typename T::T *)p, f, skip, in_place);
    else
        Piece<T, N>::store((typename T::T *)p, f);
}

// How a workgroup can hold samples, if it can: R == 0 if not.  `tensors` that are
// held: 16 pieces a thread in all (64 registers of the 128 that 1024 threads
// leave each, or two tensors' with 512).  A slab has as many groups as make rows
// of 64 bytes and 32 KB in all (16 or 64 KB, rows of 32 or 128 bytes: within 3 %),
// fewer where workgroups are; a few short samples share a workgroup.
inline HeldPlan plan_held(int64_t B, int64_t S, int C, int G, int N, int esize, int tensors, int num_cus) {
    HeldPlan p = {};
    const int D = C / G, most = tensors == 1 ? 16 : 8, threads = tensors == 1 ? 1024 : 512;
    const bool inside = D % N == 0;
    const int64_t whole = S * D * esize;  // bytes of a sample's group
    const int least = (N + D - 1) / D;    // groups of a piece
    if (N == 1 || S < 1 || S > threads * most || S * ((least * (int64_t)D + N - 1) / N) > threads * most) return p;
    int64_t gs = std::max<int64_t>(1, (32768 / tensors) / whole);
    while (gs < G && gs * D * esize < 64 && S * ((gs + 1) * D + N - 1) / N <= 512 * most) ++gs;
    gs = std::min<int64_t>(std::max<int64_t>(gs, least), G);
    while (gs > least && (gs * D + N - 1) / N > 256) --gs;  // at most 256 pieces a row
    // few samples: workgroups for all CUs, of 64 bytes a row at least
    const int64_t line = std::max<int64_t>(least, (64 + D * esize - 1) / (D * esize));
    while (gs > line && B * ((G + gs - 1) / gs) < 2 * num_cus) gs = std::max(gs / 2, line);
    p.slabs = (int)((G + gs - 1) / gs);
    p.gs = (int)std::max<int64_t>((G + p.slabs - 1) / p.slabs, least);
    p.slabs = (G + p.gs - 1) / p.gs;
    p.P = (int)(((int64_t)p.gs * D + N - 1) / N);
    for (p.nt = 256; p.nt <= threads; p.nt *= 2) {
        p.rt = (int)std::min<int64_t>(p.nt / p.P, S);
        if (p.rt < 1) continue;
        const int64_t rows = (S + p.rt - 1) / p.rt;
        if (rows <= (p.nt == 256 ? most / 2 : most)) {
            for (p.R = 1; p.R < rows;) p.R *= 2;
            break;
        }
    }
    const bool mixed = !inside && p.gs > 1;
    if (p.R > 8 && mixed) p.R = 0;  // registers
    if (!p.R) return p;
    p.rt = (int)((S + p.R - 1) / p.R);
    p.nb = (int)std::max<int64_t>(1, std::min<int64_t>(p.nt / (p.P * p.rt), B));
    // offsets inside a batch have 32 bits
    const int64_t bytes = S * C * esize;
    if (bytes >= (int64_t)1 << 31) p.R = 0;
    if (!p.R) return p;
    p.nb = (int)std::min<int64_t>(p.nb, ((int64_t)1 << 31) / bytes);
    // few samples: as many workgroups as there are CUs
    while (p.nb > 1 && (B + p.nb - 1) / p.nb * p.slabs < num_cus) --p.nb;
    p.batches = (B + p.nb - 1) / p.nb;
    // Gradients, eight rows a thread of pieces of eight elements or of several groups: 150 to 220 registers, one
    // workgroup a CU at a time.  With more of them than CUs parts are faster (32 x 784 x 768 bf16 in 32 groups 68 ->
    // 59 us; 64 x 1500 x 90 bf16 in 9: 72 -> 34; 16 x 600 x 510 fp32 in 34: 36 -> 30; 256 x 400 x 60 fp32 in 4: 29 ->
    // 31), with fewer not (16 x 600 x 510 bf16, 192 of them: 23, 26).
    if (tensors == 2 && p.R == 8 && (mixed || N == 8) && p.batches * p.slabs > num_cus) {
        p.R = 0;
        return p;
    }
    p.nt = (p.nb * p.rt * p.P + 63) / 64 * 64;
    // One odd group a slab whose rows are short runs of a line that other workgroups read too: forward (16 rows a thread)
    // 3 x 7215 x 192 bf16 in 16 (24 bytes) 38 us, in parts 18, 64 x 4096 x 320 bf16 in 32 (20) 134, 110, 7 x 4741 x 80
    // fp32 in 8 (40) 23, 17; of few threads not (40 x 2392 x 48 fp32 in 8: 19, 21).  Gradients 142 x 749 x 160 fp32 in 16
    // (40) 122, 72, 472 x 1212 x 18 in 3 (24) 53, 43; of 44 bytes 32, 34.
    const int64_t groups = p.batches * p.slabs;  // workgroups
    const bool odd = !inside && p.gs == 1;
    if (odd && D * esize < 44 && (tensors == 1 ? p.R == 16 && p.nt > 384 : p.R == 8 && groups > num_cus)) p.R = 0;
    // And those of bf16, one workgroup a CU at a time, where most CUs would have none, or a few a second one: 14 x 1641 x
    // 67 in 1 (14) 25 us, in parts 16; 70 x 194 x 516 in 1 24, 22; 150 of it 25.5, 35; 16 x 4092 x 510 in 17 (272) 57, 45;
    // 36 x 554 x 1197 in 9 (324) 41, 50.
    if (odd && tensors == 1 && N == 8 && p.R == 16 && p.nt > 512 && (5 * groups < 2 * num_cus || (groups > num_cus && 5 * groups < 6 * num_cus))) p.R = 0;
    if (!p.R) return p;
    const int dn = inside ? D / N : D;
    p.mode = mixed ? kMixed : !inside ? kOne : p.rt == 1 && dn <= 64 && !(dn & (dn - 1)) ? kShuffle : kWhole;
    p.per = p.mode == kOne ? p.P : dn;
    p.team = 64;
    while (p.team > 1 && (p.team > p.nt / (p.nb * p.gs) || p.team / 2 >= p.rt * p.per)) p.team /= 2;
    p.by_P = make_fastdiv(p.P), p.by_rt = make_fastdiv(p.rt), p.by_per = make_fastdiv(p.per), p.by_gs = make_fastdiv(p.gs);
    p.by_D = make_fastdiv(D);
    const size_t sums = (size_t)2 * (p.nt * (p.mode == kMixed ? N : 1) + p.nb * p.gs) * sizeof(float);
    p.lds = tensors == 1 ? sums : std::max(sums, (size_t)p.nt * N * sizeof(float2));
    const int64_t rows = std::max<int64_t>(1, (8ll * num_cus + p.slabs - 1) / p.slabs);
    p.grid_rows = (int)std::min<int64_t>(p.batches, rows);
    if (p.lds > 64 * 1024) p.R = 0;
    return p;
}

// ---- in parts --------------------------------------------------------------------
//
// A sample's positions are cut into parts, the channels into tiles of at most 256
// pieces: a workgroup's threads are rt rows of tp pieces, and a thread keeps its
// channels over the part's positions.  The parts' statistics (of each group; where
// no tile holds all of them of each channel first, which a kernel folds into
// groups', a workgroup a part) go to the workspace and are joined in order, by a kernel of its own or, where they are few, by every
// workgroup that needs them (8 x 16384 x 256 fp32 74 us, by a kernel 78; 2 x 65536 x
// 128 bf16 31, 33); x is read again, the last part first.  Two workgroups a CU
// in the first pass (four: 76, 34), up to four times as many in the second.
struct GnParts {
    int P, tp, tiles, rt, nt, parts;
    int64_t rows;     // positions of a part
    int split;        // workgroups of the second pass to a part
    bool by_group;    // a tile holds every group; else channels' statistics are folded into groups' first
    bool joined;      // the workgroups that need a sample's statistics join them themselves
    int team;         // lanes that add a group's values
    FastDiv by_tiles, by_parts, by_split, by_tp, by_rt, by_D;
    size_t channel_bytes, part_bytes, stat_bytes;  // the channels' statistics of all parts (folded), the groups', the joined ones
};

constexpr int64_t kMaxGrid = 1 << 21;  // workgroups of a launch (of at most 1024 threads)
constexpr int kJoinHere = 4096;  // statistics of a sample (32 KB) that every workgroup joins itself

inline GnParts plan_parts(int64_t B, int64_t S, int C, int G, int N, int esize, int num_cus) {
    GnParts p;
    p.P = (C + N - 1) / N;
    p.tiles = (p.P + 255) / 256;
    p.tp = (p.P + p.tiles - 1) / p.tiles;
    // threads in whole waves, 256 to 512 of them, with as few idle as possible
    double best = 0.0;
    for (int rt = 1; rt * p.tp <= 512; ++rt) {
        const int nt = (rt * p.tp + 63) / 64 * 64;
        const double used = (double)(rt * p.tp) / nt;
        if ((nt >= 256 || (rt + 1) * p.tp > 512) && used > best + 0.02) best = used, p.rt = rt, p.nt = nt;
    }
    // workgroups of 8 rows a thread at least; offsets in a part have 32 bits
    const int64_t jobs = std::max<int64_t>(1, B * p.tiles);
    const int64_t want = (2ll * num_cus + jobs - 1) / jobs;
    const int64_t most = (S + 8ll * p.rt - 1) / (8ll * p.rt);
    const int64_t parts = std::max<int64_t>(1, std::min({want, most, (int64_t)1024}));
    p.rows = std::max<int64_t>(1, std::min((S + parts - 1) / parts, ((int64_t)1 << 31) / ((int64_t)C * esize)));
    p.parts = (int)std::max<int64_t>(1, (S + p.rows - 1) / p.rows);
    p.by_group = p.tiles == 1;
    p.joined = (int64_t)p.parts * G <= kJoinHere;
    p.team = 64;
    while (p.team > 1 && p.team > p.nt / G) p.team /= 2;
    p.split = (int)std::max<int64_t>(1, std::min({(int64_t)4, p.rows / (8 * p.rt), kMaxGrid / ((int64_t)p.parts * p.tiles)}));
    p.by_split = make_fastdiv(p.split);
    p.by_tiles = make_fastdiv(p.tiles), p.by_parts = make_fastdiv(p.parts), p.by_tp = make_fastdiv(p.tp);
    p.by_rt = make_fastdiv(p.rt), p.by_D = make_fastdiv(C / G);
    p.channel_bytes = p.by_group ? 0 : ((size_t)B * p.parts * C * sizeof(float2) + 255) & ~(size_t)255;
    p.part_bytes = ((size_t)B * p.parts * G * sizeof(float2) + 255) & ~(size_t)255;
    p.stat_bytes = ((size_t)B * G * sizeof(float2) + 255) & ~(size_t)255;
    return p;
}

// A thread's place in a job of a part and a tile.
template <typename T, int N>
struct Place {
    int64_t b, base;  // sample; bytes to the part's first row
    int n, rows;      // positions of the part within the length, and all of them
    int part, tile, rt, j, at, skip;
    uint32_t off, step;  // bytes from there to the thread's first row, and from one to the next
    bool on, lead;       // lead: the sample's first workgroup
    // SPLIT: of one of the `split` pieces of the part
    template <bool SPLIT>
    static __device__ __forceinline__ Place of(const GroupNormArgs &a, const GnParts &p, int64_t first, uint32_t job) {
        const uint32_t r = fdiv(job, p.by_tiles), q = SPLIT ? fdiv(r, p.by_split) : r;
        return Place(a, p, first, q, (int)(job - r * p.tiles), SPLIT ? (int)(r - q * p.split) : 0, SPLIT ? p.split : 1);
    }
    __device__ __forceinline__ Place(const GroupNormArgs &a, const GnParts &p, int64_t first, uint32_t q, int of_tile, int sub, int split) {
        const uint32_t s = fdiv(q, p.by_parts);
        tile = of_tile;
        b = first + s;
        part = (int)(q - s * p.parts);
        lead = part == 0 && sub == 0 && tile == 0;
        const int each = ((int)p.rows + split - 1) / split;
        const int64_t begin = (int64_t)part * p.rows, until = min(begin + p.rows, a.S);
        const int64_t start = min(begin + (int64_t)sub * each, until), past = min(start + each, until);
        rows = (int)(past - start);
        n = (int)max(min(past, positions(a, b)) - start, (int64_t)0);
        rt = (int)fdiv(threadIdx.x, p.by_tp);
        j = threadIdx.x - rt * p.tp;
        const int piece = tile * p.tp + j, c = piece * N;
        on = rt < p.rt && piece < p.P;
        at = on ? min(c, a.C - N) : 0;
        skip = on ? c - at : N;
        constexpr int es = sizeof(typename T::T);
        base = (b * a.S + start) * a.C * es;
        off = ((uint32_t)(on ? rt : 0) * (uint32_t)a.C + (uint32_t)at) * es;
        step = (uint32_t)p.rt * (uint32_t)a.C * es;
    }
    // how many of the first `of` rows of the part are row-thread i's
    __device__ __forceinline__ static int rows_of(const GnParts &p, int i, int of) { return of > i ? (int)fdiv(of - i + p.rt - 1, p.by_rt) : 0; }
};

constexpr int kBatch = 8;  // rows whose loads are in flight together

// The sum over a workgroup of NT threads, the same value in every one.
template <int NT>
__device__ __forceinline__ float all_sum(float v, float *red) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if constexpr (NT > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) v += red[i];
    }
    return v;
}

// f(statistics, rows of the part) for every part of a group at v, thread by
// thread, some loads at a time.
template <int NT, typename F>
__device__ __forceinline__ void each_part(const GnParts &p, int G, const float2 *v, int64_t n, F f) {
    const int parts = (int)min((int64_t)p.parts, (n + p.rows - 1) / p.rows);  // that have rows
    constexpr int U = 4;
    for (int i = threadIdx.x; i < parts; i += U * NT) {
        float2 e[U];
#pragma unroll
        for (int k = 0; k < U; ++k) e[k] = v[(int64_t)min(i + k * NT, parts - 1) * G];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * NT < parts) f(e[k], (float)min(n - (int64_t)(i + k * NT) * p.rows, p.rows));
    }
}

// f(first sample, workgroups) for launches of whole samples, the last samples first where `back`.
template <typename F>
void by_samples(int64_t B, const GnParts &p, int split, bool back, F f) {
    const int64_t per = (int64_t)p.parts * p.tiles * split, some = std::max<int64_t>(1, kMaxGrid / per), n = (B + some - 1) / some;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t b = (back ? n - 1 - i : i) * some;
        f(b, dim3((unsigned)(std::min(some, B - b) * per)));
    }
}

inline unsigned grid_for(int64_t jobs) { return (unsigned)std::min(jobs, kMaxGrid); }

inline int piece_size(int C, int dtype) {
    const int v = dtype == kF32 ? 4 : 8;
    return C >= v ? v : 1;
}

// A sample's statistics of all parts, [part][G], to LDS.
__device__ __forceinline__ void fetch_parts(const GroupNormArgs &a, const GnParts &p, const float2 *from, int64_t b, float2 *to) {
    const int n = p.parts * a.G;
    const float2 *const v = from + b * n;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = v[i];
    __syncthreads();
}

// f(statistics, channel) for those of a group's D channels that are a lane's, some loads at a time.
template <typename F>
__device__ __forceinline__ void each_channel(const GnParts &p, const float2 *v, int D, int lane, F f) {
    constexpr int U = 8;
    for (int i = lane; i < D; i += U * p.team) {
        float2 e[U];
#pragma unroll
        for (int k = 0; k < U; ++k) e[k] = v[min(i + k * p.team, D - 1)];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * p.team < D) f(e[k], i + k * p.team);
    }
}

// f(group, lane of its team) for every group of a sample; a team's lanes share a wave.
template <typename F>
__device__ __forceinline__ void each_group(const GroupNormArgs &a, const GnParts &p, F f) {
    for (int g = threadIdx.x / p.team; g < a.G; g += blockDim.x / p.team) f(g, (int)threadIdx.x & (p.team - 1));
}
__device__ __forceinline__ float team_sum(const GnParts &p, float v) {
    for (int d = 1; d < p.team; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// f(the activation as a type)
template <typename F>
hipError_t by_activation(int act, F f) {
    if (act == kSilu) return f(std::integral_constant<int, kSilu>());
    if (act == kRelu) return f(std::integral_constant<int, kRelu>());
    return f(std::integral_constant<int, kNone>());
}

}  // namespace dc1d
