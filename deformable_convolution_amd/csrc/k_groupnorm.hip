// k_groupnorm.hip -- group norm over positions in channels-last order with an
// activation, x [B][S][C], G groups of D channels, and its gradients.
//
//   mu, r  of a sample's n positions times a group's D channels
//   z  = (x - mu) r w + b,  y = act(z)
//   g' = g act'(z),  u = g' w,  xh = (x - mu) r
//   gx = r (u - mean u - xh mean(u xh)),  gw = sum g' xh,  gb = sum g'
//
// Bound by HBM: the forward has to read x and write y, the backward to read x
// and g and write gx.
#include <algorithm>

#include "vec16.h"

namespace dc1d {

namespace {

enum Act { kNone = 0, kRelu = 1, kSilu = 2 };

__device__ __forceinline__ float activate(float z, int act) {
    if (act == kRelu) return z < 0.0f ? 0.0f : z;  // a NaN stays
    if (act == kSilu) {
        float p, q;
        sigmoid_pair(z, p, q);
        return z * p;
    }
    return z;
}
// The gradient g of act(z) taken to z.
__device__ __forceinline__ float activate_back(float z, float g, int act) {
    if (act == kRelu) return z > 0.0f ? g : 0.0f;
    if (act == kSilu) {
        float p, q;
        sigmoid_pair(z, p, q);
        return g * (p + z * p * q);
    }
    return g;
}

__device__ __forceinline__ int64_t positions(const GroupNormArgs &a, int64_t b) {
    if (!a.lens) return a.S;
    const int n = a.lens[b];
    return n < 0 ? 0 : n < a.S ? n : a.S;
}

// ---- in parts --------------------------------------------------------------------
//
// A sample's positions are cut into parts, the channels into tiles of at most NT
// pieces: a workgroup's threads are rt rows of tp pieces, and a thread keeps its
// channels over the part's positions.  The parts' statistics (of each channel,
// or of each group where a tile holds all of them) go to the workspace, are
// joined in order, and x is read again, the last part first, for y.
struct GnParts {
    int P, tp, tiles, rt, nt, parts;
    int64_t rows;     // positions of a part
    bool by_group;    // a part's statistics are kept for groups
    int entries;      // of a part: G or C
    size_t part_bytes, stat_bytes;
};

GnParts plan_parts(int64_t B, int64_t S, int C, int G, int N, int num_cus) {
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
    // eight workgroups for every CU, of 16 rows a thread at least
    const int64_t want = (8ll * num_cus + B * p.tiles - 1) / (B * p.tiles > 0 ? B * p.tiles : 1);
    const int64_t most = (S + 16ll * p.rt - 1) / (16ll * p.rt);
    int64_t parts = std::max<int64_t>(1, std::min({want, most, (int64_t)1024}));
    p.rows = std::max<int64_t>(1, (S + parts - 1) / parts);
    p.parts = (int)std::max<int64_t>(1, (S + p.rows - 1) / p.rows);
    p.by_group = p.tiles == 1;
    p.entries = p.by_group ? G : C;
    p.part_bytes = ((size_t)B * p.parts * p.entries * sizeof(float2) + 255) & ~(size_t)255;
    p.stat_bytes = ((size_t)B * G * sizeof(float2) + 255) & ~(size_t)255;
    return p;
}

// A thread's place in a job of a part and a tile.
template <int N>
struct Place {
    int64_t b, start, end;  // sample; its part's positions within the length
    int64_t last;           // past the part's last position
    int part, rt, at, skip, j;
    bool on;
    __device__ __forceinline__ Place(const GroupNormArgs &a, const GnParts &p, int64_t job) {
        const int tile = (int)(job % p.tiles);
        const int64_t q = job / p.tiles;
        b = q / p.parts;
        part = (int)(q % p.parts);
        const int64_t n = positions(a, b);
        start = (int64_t)part * p.rows;
        last = min(start + p.rows, a.S);
        end = min(last, n);
        rt = threadIdx.x / p.tp;
        j = threadIdx.x % p.tp;
        const int piece = tile * p.tp + j, c = piece * N;
        on = rt < p.rt && piece < p.P;
        at = on ? min(c, a.C - N) : 0;
        skip = on ? c - at : N;
    }
    // rows of the part that row-thread i visits
    __device__ __forceinline__ float rows(const GnParts &p, int i) const {
        const int64_t n = end - start - i;
        return n > 0 ? (float)((n + p.rt - 1) / p.rt) : 0.0f;
    }
};

constexpr int kBatch = 8;  // rows whose loads are in flight together

template <typename T, int N>
__global__ __launch_bounds__(512) void k_gn_part_stats(GroupNormArgs a, GnParts p, float2 *out, int64_t jobs) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 red[];  // [rt][tp][N], then of the channels
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Place<N> t(a, p, job);
        const E *const x = (const E *)a.x + t.b * a.S * a.C + t.at;
        float n = 0.0f, mean[N] = {}, m2[N] = {};
        if (t.on) {
            for (int64_t r = t.start + t.rt; r < t.end; r += (int64_t)kBatch * p.rt) {
                typename P::Raw raw[kBatch];
                int have = 0;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int64_t row = r + (int64_t)i * p.rt;
                    have += row < t.end;
                    raw[i] = P::load(x + (row < t.end ? row : r) * a.C);
                }
                // the batch's mean and squares about it, joined with those so far
                const float m = (float)have, all = n + m, share = m / all;
                float s[N] = {}, d[N] = {};
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    float f[N];
                    P::widen(raw[i], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) s[e] += i < have ? f[e] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] = have == kBatch ? s[e] * (1.0f / kBatch) : s[e] / m;  // equal values have their own as mean
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    float f[N];
                    P::widen(raw[i], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float v = i < have ? f[e] - s[e] : 0.0f;
                        d[e] += v * v;
                    }
                }
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float v = s[e] - mean[e];
                    mean[e] += v * share;
                    m2[e] += d[e] + v * v * n * share;
                }
                n = all;
            }
            for (int e = 0; e < N; ++e) red[(t.rt * p.tp + t.j) * N + e] = make_float2(mean[e], m2[e]);
        }
        __syncthreads();
        // the row-threads' statistics of a channel
        const int channels = p.tp * N;
        const float rows = (float)max(t.end - t.start, (int64_t)1);
        float2 *const own = red + p.rt * channels;
        for (int k = threadIdx.x; k < channels; k += blockDim.x) {
            float mu = 0.0f, q = 0.0f;
            for (int i = 0; i < p.rt; ++i) mu += red[i * channels + k].x * t.rows(p, i);
            mu /= rows;
            for (int i = 0; i < p.rt; ++i) {
                const float2 v = red[i * channels + k];
                const float d = v.x - mu;
                q += v.y + d * d * t.rows(p, i);
            }
            own[k] = make_float2(mu, q);
        }
        __syncthreads();
        const int tile = (int)(job % p.tiles);
        float2 *const o = out + (t.b * p.parts + t.part) * p.entries;
        if (!p.by_group) {
            for (int k = threadIdx.x; k < channels; k += blockDim.x) {
                const int c = (tile * p.tp) * N + k, piece = c / N;
                if (piece >= p.P) continue;
                const int at = min(piece * N, a.C - N);
                if (k % N >= piece * N - at) o[at + k % N] = own[k];
            }
        } else {
            // lanes in teams of 8 to a group
            const int lane = threadIdx.x & 7;
            for (int g = threadIdx.x >> 3; g < a.G; g += blockDim.x >> 3) {
                float mu = 0.0f, q = 0.0f;
                for (int i = lane; i < a.D; i += 8) {
                    const int c = g * a.D + i, last = a.C - N;
                    mu += own[c >= (p.P - 1) * N ? (p.P - 1) * N + c - last : c].x;
                }
                for (int d = 1; d < 8; d <<= 1) mu += __shfl_xor(mu, d);
                mu /= (float)a.D;
                for (int i = lane; i < a.D; i += 8) {
                    const int c = g * a.D + i, last = a.C - N;
                    const float2 v = own[c >= (p.P - 1) * N ? (p.P - 1) * N + c - last : c];
                    const float d = v.x - mu;
                    q += v.y + d * d * rows;
                }
                for (int d = 1; d < 8; d <<= 1) q += __shfl_xor(q, d);
                if (lane == 0) o[g] = make_float2(mu, q);
            }
        }
        __syncthreads();
    }
}

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

// f(part, entry, rows of the part) for every entry of group g, thread by thread.
template <int NT, typename F>
__device__ __forceinline__ void each_entry(const GnParts &p, int per, int64_t n, F f) {
    const int cols = per < NT ? per : NT, rp = NT / cols;
    const int c0 = threadIdx.x % cols, p0 = threadIdx.x / cols;
    if (p0 >= rp) return;
    for (int i = p0; i < p.parts; i += rp) {
        const int64_t rows = min(n - (int64_t)i * p.rows, p.rows);
        if (rows <= 0) return;
        for (int c = c0; c < per; c += cols) f(i, c, (float)rows);
    }
}

// A group's statistics from its parts'.
template <int NT>
__global__ __launch_bounds__(NT) void k_gn_join(GroupNormArgs a, GnParts p, const float2 *part, float2 *stat) {
    __shared__ float red[NT / 64];
    const int64_t jobs = a.B * a.G;
    const int per = p.by_group ? 1 : a.D;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t b = job / a.G, n = positions(a, b);
        const int g = (int)(job % a.G);
        const float2 *const v = part + b * p.parts * p.entries + (int64_t)g * per;
        float s = 0.0f, q = 0.0f;
        each_entry<NT>(p, per, n, [&](int i, int c, float rows) { s += v[(int64_t)i * p.entries + c].x * rows; });
        const float all = (float)n * (float)per;
        const float mean = n > 0 ? all_sum<NT>(s, red) / all : 0.0f;
        each_entry<NT>(p, per, n, [&](int i, int c, float rows) {
            const float2 e = v[(int64_t)i * p.entries + c];
            const float d = e.x - mean;
            q += e.y + d * d * rows * (p.by_group ? (float)a.D : 1.0f);
        });
        const float var = n > 0 ? all_sum<NT>(q, red) / ((float)n * (float)a.D) : 0.0f;
        if (threadIdx.x == 0) {
            const float rstd = n > 0 ? rsqrtf(var + a.eps) : 0.0f;
            stat[job] = make_float2(mean, rstd);
            if (a.mean) a.mean[job] = mean;
            if (a.rstd) a.rstd[job] = rstd;
        }
    }
}

template <typename T, int N>
__global__ __launch_bounds__(512) void k_gn_part_apply(GroupNormArgs a, GnParts p, const float2 *stat, int64_t jobs) {
    using P = Piece<T, N>;
    using E = typename T::T;
    for (int64_t at = blockIdx.x; at < jobs; at += gridDim.x) {
        const Place<N> t(a, p, jobs - 1 - at);  // what was read last is still in cache
        if (!t.on) continue;
        const E *const x = (const E *)a.x + t.b * a.S * a.C + t.at;
        E *const y = (E *)a.y + t.b * a.S * a.C + t.at;
        float mean[N], r[N], w[N], b[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float2 s = stat[t.b * a.G + (t.at + e) / a.D];
            mean[e] = s.x, r[e] = s.y;
            w[e] = a.w ? T::ld((const E *)a.w, t.at + e) : 1.0f;
            b[e] = a.b ? T::ld((const E *)a.b, t.at + e) : 0.0f;
        }
        for (int64_t row0 = t.start + t.rt; row0 < t.last; row0 += (int64_t)kBatch * p.rt) {
            typename P::Raw raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t row = row0 + (int64_t)i * p.rt;
                raw[i] = P::load(x + (row < t.end ? row : row0) * a.C);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t row = row0 + (int64_t)i * p.rt;
                if (row >= t.last) break;
                float f[N];
                P::widen(raw[i], f);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    f[e] = row < t.end ? activate((f[e] - mean[e]) * r[e] * w[e] + b[e], a.act) : 0.0f;
                store_own<T, N>(y + row * a.C, f, t.skip);
            }
        }
    }
}

// ---- gradients in parts ------------------------------------------------------------

// What a thread keeps of its channels.
template <typename T, int N>
struct Channels {
    float mean[N], r[N], w[N], b[N];
    __device__ __forceinline__ Channels(const GroupNormArgs &a, int64_t sample, int at) {
        using E = typename T::T;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t k = sample * a.G + (at + e) / a.D;
            mean[e] = a.mean[k], r[e] = a.rstd[k];
            w[e] = a.w ? T::ld((const E *)a.w, at + e) : 1.0f;
            b[e] = a.b ? T::ld((const E *)a.b, at + e) : 0.0f;
        }
    }
    // x becomes xh and g becomes g'
    __device__ __forceinline__ void back(float *x, float *g, int act) const {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            x[e] = (x[e] - mean[e]) * r[e];
            g[e] = activate_back(x[e] * w[e] + b[e], g[e], act);
        }
    }
};

// sum g' and sum g' xh of every channel over a part: [b][part][C].
template <typename T, int N>
__global__ __launch_bounds__(512) void k_gn_part_sums(GroupNormArgs a, GnParts p, float2 *out, int64_t jobs) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 red[];
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const Place<N> t(a, p, job);
        const int64_t base = t.b * a.S * a.C + t.at;
        const E *const x = (const E *)a.x + base, *const g = (const E *)a.g + base;
        if (t.on) {
            const Channels<T, N> ch(a, t.b, t.at);
            float s1[N] = {}, s2[N] = {};
            constexpr int U = kBatch / 2;
            for (int64_t r = t.start + t.rt; r < t.end; r += (int64_t)U * p.rt) {
                typename P::Raw xr[U], gr[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int64_t row = r + (int64_t)i * p.rt;
                    xr[i] = P::load(x + (row < t.end ? row : r) * a.C);
                    gr[i] = P::load(g + (row < t.end ? row : r) * a.C);
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (r + (int64_t)i * p.rt >= t.end) break;
                    float xh[N], u[N];
                    P::widen(xr[i], xh);
                    P::widen(gr[i], u);
                    ch.back(xh, u, a.act);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        s1[e] += u[e];
                        s2[e] += u[e] * xh[e];
                    }
                }
            }
            for (int e = 0; e < N; ++e) red[(t.rt * p.tp + t.j) * N + e] = make_float2(s1[e], s2[e]);
        }
        __syncthreads();
        const int channels = p.tp * N, tile = (int)(job % p.tiles);
        float2 *const o = out + (t.b * p.parts + t.part) * a.C;
        for (int k = threadIdx.x; k < channels; k += blockDim.x) {
            const int c = tile * channels + k, piece = c / N;
            if (piece >= p.P) continue;
            const int at = min(piece * N, a.C - N);
            if (k % N < piece * N - at) continue;
            float2 s = make_float2(0.0f, 0.0f);
            for (int i = 0; i < p.rt; ++i) {
                s.x += red[i * channels + k].x;
                s.y += red[i * channels + k].y;
            }
            o[at + k % N] = s;
        }
        __syncthreads();
    }
}

// mean u and mean(u xh) of a group.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_gn_join_back(GroupNormArgs a, GnParts p, const float2 *part, float2 *stat) {
    using E = typename T::T;
    __shared__ float red[NT / 64];
    const int64_t jobs = a.B * a.G;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t b = job / a.G, n = positions(a, b);
        const int g = (int)(job % a.G);
        const float2 *const v = part + b * p.parts * a.C + (int64_t)g * a.D;
        float s = 0.0f, q = 0.0f;
        each_entry<NT>(p, a.D, n, [&](int i, int c, float) {
            const float2 e = v[(int64_t)i * a.C + c];
            const float w = a.w ? T::ld((const E *)a.w, (int64_t)g * a.D + c) : 1.0f;
            s += e.x * w;
            q += e.y * w;
        });
        s = all_sum<NT>(s, red);
        q = all_sum<NT>(q, red);
        const float inv = n > 0 ? 1.0f / ((float)n * (float)a.D) : 0.0f;
        if (threadIdx.x == 0) stat[job] = make_float2(s * inv, q * inv);
    }
}

template <typename T, int N>
__global__ __launch_bounds__(512) void k_gn_part_back(GroupNormArgs a, GnParts p, const float2 *stat, int64_t jobs) {
    using P = Piece<T, N>;
    using E = typename T::T;
    for (int64_t k = blockIdx.x; k < jobs; k += gridDim.x) {
        const Place<N> t(a, p, jobs - 1 - k);
        if (!t.on) continue;
        const int64_t base = t.b * a.S * a.C + t.at;
        const E *const x = (const E *)a.x + base, *const g = (const E *)a.g + base;
        E *const y = (E *)a.y + base;
        const Channels<T, N> ch(a, t.b, t.at);
        float c1[N], c2[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float2 s = stat[t.b * a.G + (t.at + e) / a.D];
            c1[e] = s.x, c2[e] = s.y;
        }
        constexpr int U = kBatch / 2;
        for (int64_t row0 = t.start + t.rt; row0 < t.last; row0 += (int64_t)U * p.rt) {
            typename P::Raw xr[U], gr[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t row = row0 + (int64_t)i * p.rt;
                xr[i] = P::load(x + (row < t.end ? row : row0) * a.C);
                gr[i] = P::load(g + (row < t.end ? row : row0) * a.C);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t row = row0 + (int64_t)i * p.rt;
                if (row >= t.last) break;
                float xh[N], u[N];
                P::widen(xr[i], xh);
                P::widen(gr[i], u);
                ch.back(xh, u, a.act);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    u[e] = row < t.end ? ch.r[e] * (u[e] * ch.w[e] - c1[e] - xh[e] * c2[e]) : 0.0f;
                store_own<T, N>(y + row * a.C, u, t.skip);
            }
        }
    }
}

// The parameters' gradients: sum over `rows` rows of [C] pairs (sum g', sum g' xh).
// 16 channels of 16 row-threads; the rows of a thread, then the threads in order.
template <typename T>
__global__ __launch_bounds__(256) void k_gn_params(const float2 *sums, int64_t rows, int C, void *gw, void *gb) {
    using E = typename T::T;
    __shared__ float2 red[16][17];
    const int64_t c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const int r0 = threadIdx.x >> 4;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < C)
        for (int64_t r = r0; r < rows; r += 16) {
            const float2 v = sums[r * C + c];
            s.x += v.x, s.y += v.y;
        }
    red[r0][threadIdx.x & 15] = s;
    __syncthreads();
    if (r0 == 0 && c < C) {
        for (int i = 1; i < 16; ++i) s.x += red[i][threadIdx.x].x, s.y += red[i][threadIdx.x].y;
        if (gw) T::st((E *)gw, c, s.y);
        if (gb) T::st((E *)gb, c, s.x);
    }
}

constexpr int64_t kMaxGrid = 1 << 21;  // workgroups of a launch (of at most 1024 threads); more jobs are looped over

unsigned grid_for(int64_t jobs) { return (unsigned)std::min(jobs, kMaxGrid); }

int piece_size(int C, int dtype) {
    const int v = dtype == kF32 ? 4 : 8;
    return C >= v ? v : 1;
}

template <typename T, int N>
hipError_t run_parts(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    const GnParts p = plan_parts(a.B, a.S, a.C, a.G, N, num_cus);
    float2 *const part = (float2 *)a.ws, *const stat = (float2 *)((char *)a.ws + p.part_bytes);
    const int64_t jobs = a.B * p.parts * p.tiles;
    const size_t lds = (size_t)(p.rt + 1) * p.tp * N * sizeof(float2);
    hipLaunchKernelGGL((k_gn_part_stats<T, N>), dim3(grid_for(jobs)), dim3(p.nt), lds, stream, a, p, part, jobs);
    if ((int64_t)p.parts * (p.by_group ? 1 : a.D) <= 256)
        hipLaunchKernelGGL((k_gn_join<64>), dim3(grid_for(a.B * a.G)), dim3(64), 0, stream, a, p, part, stat);
    else
        hipLaunchKernelGGL((k_gn_join<1024>), dim3(grid_for(a.B * a.G)), dim3(1024), 0, stream, a, p, part, stat);
    hipLaunchKernelGGL((k_gn_part_apply<T, N>), dim3(grid_for(jobs)), dim3(p.nt), 0, stream, a, p, stat, jobs);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t run_parts_back(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    const GnParts p = plan_parts(a.B, a.S, a.C, a.G, N, num_cus);
    const size_t part_bytes = ((size_t)a.B * p.parts * a.C * sizeof(float2) + 255) & ~(size_t)255;
    float2 *const part = (float2 *)a.ws, *const stat = (float2 *)((char *)a.ws + part_bytes);
    const int64_t jobs = a.B * p.parts * p.tiles;
    const size_t lds = (size_t)p.rt * p.tp * N * sizeof(float2);
    if (jobs > 0) hipLaunchKernelGGL((k_gn_part_sums<T, N>), dim3(grid_for(jobs)), dim3(p.nt), lds, stream, a, p, part, jobs);
    if (a.y && jobs > 0 && a.S > 0) {
        if ((int64_t)p.parts * a.D <= 256)
            hipLaunchKernelGGL((k_gn_join_back<T, 64>), dim3(grid_for(a.B * a.G)), dim3(64), 0, stream, a, p, part, stat);
        else
            hipLaunchKernelGGL((k_gn_join_back<T, 1024>), dim3(grid_for(a.B * a.G)), dim3(1024), 0, stream, a, p, part, stat);
        hipLaunchKernelGGL((k_gn_part_back<T, N>), dim3(grid_for(jobs)), dim3(p.nt), 0, stream, a, p, stat, jobs);
    }
    if (a.gw || a.gb)
        hipLaunchKernelGGL((k_gn_params<T>), dim3((a.C + 15) / 16), dim3(256), 0, stream, part, a.B * p.parts, a.C, a.gw, a.gb);
    return hipGetLastError();
}

}  // namespace

size_t group_norm_workspace(int64_t B, int64_t S, int C, int G, int dtype, int num_cus) {
    const GnParts p = plan_parts(B, S, C, G, piece_size(C, dtype), num_cus);
    return p.part_bytes + p.stat_bytes;
}

hipError_t launch_group_norm(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    if (a.dtype == kF32) return a.C >= 4 ? run_parts<F32, 4>(a, num_cus, stream) : run_parts<F32, 1>(a, num_cus, stream);
    return a.C >= 8 ? run_parts<BF16, 8>(a, num_cus, stream) : run_parts<BF16, 1>(a, num_cus, stream);
}

size_t group_norm_backward_workspace(int64_t B, int64_t S, int C, int G, int dtype, bool, int num_cus) {
    const GnParts p = plan_parts(B, S, C, G, piece_size(C, dtype), num_cus);
    return (((size_t)B * p.parts * C * sizeof(float2) + 255) & ~(size_t)255) + p.stat_bytes;
}

hipError_t launch_group_norm_backward(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    if (a.dtype == kF32) return a.C >= 4 ? run_parts_back<F32, 4>(a, num_cus, stream) : run_parts_back<F32, 1>(a, num_cus, stream);
    return a.C >= 8 ? run_parts_back<BF16, 8>(a, num_cus, stream) : run_parts_back<BF16, 1>(a, num_cus, stream);
}

}  // namespace dc1d
