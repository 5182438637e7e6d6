// k_groupnorm.hip -- group norm over positions in channels-last order with an
// activation, x [B][S][C], G groups of D channels, and (k_groupnorm_bwd.hip) its
// gradients.
//
//   mu, r  of a sample's n positions times a group's D channels
//   z  = (x - mu) r w + b,  y = act(z)
//   g' = g act'(z),  u = g' w,  xh = (x - mu) r
//   gx = r (u - mean u - xh mean(u xh)),  gw = sum g' xh,  gb = sum g'
//
// Bound by HBM: the forward has to read x and write y, the backward to read x
// and g and write gx.  A group's values stand D at a time in rows of C, so that a
// workgroup that is to know a whole group's statistics holds a slab of channels
// of all positions.
#include "groupnorm.h"

namespace dc1d {

namespace {

// All loads first, then the sums, the squares and the rows' results, each row
// widened anew (hold() keeps the compiler from widening all of them at once, which
// took twice the registers).  8 x 4096 x 512 bf16 in 32 groups: 24 us, 2.8 TB/s, the
// vector unit busy for 54 % of it: one workgroup a CU, whose reads, sums and writes
// follow one another; 32 x 784 x 512 fp32 22 us, 4.6 TB/s; 32768 rows of 1024 bf16 33
// us, 4.1 TB/s.
template <typename T, int N, int R, int MODE, int ACT>
__global__ __launch_bounds__(1024) void k_gn_held(GroupNormArgs a, HeldPlan p, int64_t first) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float lds[];
    const int64_t job = first + (p.slabs > 1 ? by_xcd(blockIdx.x, gridDim.x) : blockIdx.x), batch = job / p.slabs;
    const int slab = (int)(job - batch * p.slabs);
    const HeldPlace<N, MODE> t(a, p, slab);
    constexpr int NV = HeldPlace<N, MODE>::NV;
    GroupSums<N, MODE> sum(p, lds);
    const int64_t b = min(batch * p.nb + t.sm, a.B - 1);
    const bool on = t.in && batch * p.nb + t.sm < a.B;
    const int n = (int)positions(a, b), s = (int)(b - batch * p.nb);
    const int64_t base = batch * p.nb * a.S * a.C * (int64_t)sizeof(E);
    const char *const x = (const char *)a.x + base;
    typename P::Raw raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = P::load((const E *)(x + t.offset(a, p, sizeof(E), s, i, on && t.rt + i * p.rt < n)));
    typename P::Raw wr, br;
    if (a.w) wr = P::load((const E *)a.w + t.at);
    if (a.b) br = P::load((const E *)a.b + t.at);
    // Rows that do not count: where pieces are whole, zeros about a mean of 0, no
    // choice for every element (8 x 4096 x 512 bf16 27 -> 24 us; 16 rows of fp32 would spill: 512 x 64 x 768 44 -> 48).
    constexpr bool pieces = (MODE == kShuffle || MODE == kWhole) && (sizeof(E) == 2 || R <= 8);
    float v[1][NV] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool see = on && t.rt + i * p.rt < n;
        if (pieces && !__all(see)) {
            const typename P::Raw zero = {};
            if (!see) raw[i] = zero;
        }
        float f[N];
        hold(raw[i]);
        P::widen(raw[i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) v[0][t.v(e)] += pieces || (see && e >= t.skip) ? f[e] : 0.0f;
#pragma unroll
        for (int e = 0; e < NV; ++e) hold(v[0][e]);
    }
    sum(p, v, t.channels, a.D, t.slot, t.of);
    const float inv = n > 0 ? 1.0f / ((float)n * (float)a.D) : 0.0f;
    float mean[NV], sq[2][NV] = {};
#pragma unroll
    for (int e = 0; e < NV; ++e) mean[e] = v[0][e] * inv;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float f[N];
        hold(raw[i]);
        P::widen(raw[i], f);
        const bool see = on && t.rt + i * p.rt < n;
        const float m = see ? mean[0] : 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = pieces ? f[e] - m : see && e >= t.skip ? f[e] - mean[t.v(e)] : 0.0f;
            sq[0][t.v(e)] += d;
            sq[1][t.v(e)] += d * d;
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            hold(sq[0][e]);
            hold(sq[1][e]);
        }
    }
    sum(p, sq, t.channels, a.D, t.slot, t.of);
    // What the first mean leaves, s = sum (x - mean), is taken out of the mean and the squares: of equal values the mean is
    // their own then (a sum over its count is not: of 4096 x 16 values of 0.1, y was 4e-4 off).  An infinite one stays.
    float r[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const float s = fabsf(sq[0][e]) < __builtin_inff() ? sq[0][e] : 0.0f, by = s * inv;
        const float left = fmaf(-s, by, sq[1][e]);  // of infinite squares they, also where s by is past 32 bits
        mean[e] += by;
        r[e] = n > 0 ? rsqrtf((left < 0.0f ? 0.0f : left) * inv + a.eps) : 0.0f;
    }
    if (!on) return;
    float w[N], c[N];
    if (a.w) P::widen(wr, w);
    if (a.b) P::widen(br, c);
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = a.w ? r[t.v(e)] * w[e] : r[t.v(e)], c[e] = a.b ? c[e] : 0.0f;
    char *const y = (char *)a.y + base;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = t.rt + i * p.rt;
        if (row >= a.S) continue;
        float f[N];
        hold(raw[i]);
        P::widen(raw[i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            f[e] = row < n ? activate<ACT>((f[e] - mean[t.v(e)]) * w[e] + c[e]) : 0.0f;
            hold(f[e]);
        }
        put<T, N, MODE>(y + t.offset(a, p, sizeof(E), s, i, true), f, t.skip, a.y == a.x || t.channels < N);  // fewer: the others' groups are not here
    }
    if (t.rt == 0) {
        // the thread that holds a group's first element
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int ch = t.at + e, g = t.group + t.of[t.v(e)];
            if (e < t.skip || ch != g * a.D) continue;
            if (a.mean) a.mean[b * a.G + g] = mean[t.v(e)];
            if (a.rstd) a.rstd[b * a.G + g] = r[t.v(e)];
        }
    }
}

// A part's mean and squares about it: of kBatch rows at a time, from registers,
// joined with those so far by (n, mean, M2) + (m, s, d): mean + (s - mean) m / (n +
// m), M2 + d + (s - mean)^2 n m / (n + m); then over the row-threads and a group's
// channels.  Every mean, here and where parts are joined, is one of its terms plus the
// mean of the differences from it: equal values have their own as mean.  8 x 16384 x
// 256 fp32: 34 us, 3.9 TB/s (parts of 257 or 265 rows, so that they do not start at
// the same distance in all channels of the memory, and twice the workgroups: no
// faster); 13 x 4092 x 255 bf16: 12 us.
template <typename T, int N>
__global__ __launch_bounds__(512) void k_gn_part_stats(GroupNormArgs a, GnParts p, float2 *channels_out, float2 *out, int64_t first) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 red[];  // [rt][tp][N], then of the channels
    const Place<T, N> t = Place<T, N>::template of<false>(a, p, first, blockIdx.x);
    const char *const x = (const char *)a.x + t.base;
    const int mine = t.on ? t.rows_of(p, t.rt, t.n) : 0;
    float n = 0.0f, mean[N] = {}, m2[N] = {};
    typename P::Raw raw[kBatch], next[kBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next[i] = P::load((const E *)(x + (t.off + (uint32_t)min(i0 + i, mine - 1) * t.step)));
    };
    if (mine) load(0);
    for (int i0 = 0; i0 < mine; i0 += kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) raw[i] = next[i];
        if (i0 + kBatch < mine) load(i0 + kBatch);
        // the batch's mean and squares about it, joined with those so far
        const int have = min(mine - i0, kBatch);
        const float m = (float)have, all = n + m, share = m / all;
        float s[N] = {}, d[N] = {};
        if (i0 == 0) P::widen(raw[0], mean);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float f[N];
            hold(raw[i]);
            P::widen(raw[i], f);
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] += i < have ? f[e] - mean[e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = mean[e] + (have == kBatch ? s[e] * (1.0f / kBatch) : s[e] / m);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float f[N];
            hold(raw[i]);
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
            m2[e] += d[e] + v * (v * (n * share));  // 0 of no rows, also where v v is infinite
        }
        n = all;
    }
    if (t.on)
#pragma unroll
        for (int e = 0; e < N; ++e) red[(t.rt * p.tp + t.j) * N + e] = make_float2(mean[e], m2[e]);
    __syncthreads();
    // the row-threads' statistics of a channel
    const int channels = p.tp * N;
    const float rows = (float)max(t.n, 1);
    float2 *const own = red + p.rt * channels;
    for (int k = threadIdx.x; k < channels; k += blockDim.x) {
        const float m0 = red[k].x;
        float mu = 0.0f, q = 0.0f;
        for (int i = 1; i < p.rt; ++i) mu += (red[i * channels + k].x - m0) * (float)t.rows_of(p, i, t.n);
        mu = m0 + mu / rows;
        for (int i = 0; i < p.rt; ++i) {
            const float2 v = red[i * channels + k];
            const float d = v.x - mu;
            q += v.y + d * (d * (float)t.rows_of(p, i, t.n));
        }
        own[k] = make_float2(mu, q);
    }
    __syncthreads();
    const int64_t row = t.b * p.parts + t.part;
    if (!p.by_group) {
        float2 *const o = channels_out + row * a.C;
        for (int k = threadIdx.x; k < channels; k += blockDim.x) {
            const int piece = t.tile * p.tp + k / N, c = piece * N;
            if (piece >= p.P) continue;
            const int at = min(c, a.C - N);
            if (k % N >= c - at) o[at + k % N] = own[k];
        }
    } else {
        float2 *const o = out + row * a.G;
        // the last piece is moved back to end with the row
        auto of = [&](int c) { return own[c >= (p.P - 1) * N ? (p.P - 1) * N + c - (a.C - N) : c]; };
        each_group(a, p, [&](int g, int lane) {
            const float m0 = of(g * a.D).x;
            float mu = 0.0f, q = 0.0f;
            for (int i = lane; i < a.D; i += p.team) mu += of(g * a.D + i).x - m0;
            mu = m0 + team_sum(p, mu) / (float)a.D;
            for (int i = lane; i < a.D; i += p.team) {
                const float2 v = of(g * a.D + i);
                const float d = v.x - mu;
                q += v.y + d * d * rows;
            }
            q = team_sum(p, q);
            if (lane == 0) o[g] = make_float2(mu, q);
        });
    }
}

// A part's groups from its channels.  (A workgroup a group for the channels of all
// parts: 8479 x 1052 fp32 in 4 groups took 65 us, not 31; 300 x 5000 in one 103, not
// 23, gradients 76, not 33.)
__global__ __launch_bounds__(256) void k_gn_fold(GroupNormArgs a, GnParts p, const float2 *channels, float2 *out) {
    const int64_t jobs = a.B * p.parts;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t b = job / p.parts, n = positions(a, b);
        const float rows = (float)max(min(n - (job - b * p.parts) * p.rows, p.rows), (int64_t)0);
        const float2 *const v = channels + job * a.C;
        each_group(a, p, [&](int g, int lane) {
            const float2 *const of = v + (int64_t)g * a.D;
            const float m0 = of[0].x;
            float mu = 0.0f, q = 0.0f;
            each_channel(p, of, a.D, lane, [&](float2 e, int) { mu += e.x - m0; });
            mu = m0 + team_sum(p, mu) / (float)a.D;
            each_channel(p, of, a.D, lane, [&](float2 e, int) {
                const float d = e.x - mu;
                q += e.y + d * d * rows;
            });
            q = team_sum(p, q);
            if (lane == 0) out[job * a.G + g] = make_float2(mu, q);
        });
    }
}

// A group's statistics from its parts'.
template <int NT>
__global__ __launch_bounds__(NT) void k_gn_join(GroupNormArgs a, GnParts p, const float2 *part, float2 *stat) {
    __shared__ float red[NT / 64];
    const int64_t jobs = a.B * a.G;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t b = job / a.G, n = positions(a, b);
        const float2 *const v = part + b * p.parts * a.G + job % a.G;
        const float m0 = v[0].x;
        float s = 0.0f, q = 0.0f;
        each_part<NT>(p, a.G, v, n, [&](float2 e, float rows) { s += (e.x - m0) * rows; });
        const float mean = n > 0 ? m0 + all_sum<NT>(s, red) / (float)n : 0.0f;
        each_part<NT>(p, a.G, v, n, [&](float2 e, float rows) {
            const float d = e.x - mean;
            q += e.y + d * d * rows * (float)a.D;
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

// The second reading, the last samples and parts first: what the first pass read
// last is in the last-level cache.  8 x 16384 x 256 fp32: 40 us, 6.7 TB/s; 13 x 4092
// x 255 bf16, whose rows stand at odd addresses: 16 us, 2.7 TB/s.
template <typename T, int N, int ACT>
__global__ __launch_bounds__(512) void k_gn_part_apply(GroupNormArgs a, GnParts p, const float2 *part, float2 *stat, int64_t first) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 joined[];
    const Place<T, N> t = Place<T, N>::template of<true>(a, p, first, gridDim.x - 1 - blockIdx.x);  // what was read last is still in cache
    const char *const x = (const char *)a.x + t.base;
    char *const y = (char *)a.y + t.base;
    const int mine = t.on ? t.rows_of(p, t.rt, t.n) : 0, every = t.on ? t.rows_of(p, t.rt, t.rows) : 0;
    typename P::Raw raw[kBatch], next[kBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next[i] = P::load((const E *)(x + (t.off + (uint32_t)max(min(i0 + i, mine - 1), 0) * t.step)));
    };
    if (every) load(0);
    if (p.joined) {
        const int64_t n = positions(a, t.b);
        float2 *const v = joined + a.G;
        fetch_parts(a, p, part, t.b, v);
        each_group(a, p, [&](int g, int lane) {
            const float m0 = v[g].x;
            float s = 0.0f, q = 0.0f;
            for (int i = lane; i < p.parts; i += p.team) {
                const int64_t rows = min(n - (int64_t)i * p.rows, p.rows);
                if (rows > 0) s += (v[i * a.G + g].x - m0) * (float)rows;
            }
            const float mean = n > 0 ? m0 + team_sum(p, s) / (float)n : 0.0f;
            for (int i = lane; i < p.parts; i += p.team) {
                const int64_t rows = min(n - (int64_t)i * p.rows, p.rows);
                const float2 e = v[i * a.G + g];
                const float d = e.x - mean;
                if (rows > 0) q += e.y + d * d * (float)rows * (float)a.D;
            }
            const float rstd = n > 0 ? rsqrtf(team_sum(p, q) / ((float)n * (float)a.D) + a.eps) : 0.0f;
            if (lane == 0) {
                joined[g] = make_float2(mean, rstd);
                if (t.lead) {
                    if (a.mean) a.mean[t.b * a.G + g] = mean;
                    if (a.rstd) a.rstd[t.b * a.G + g] = rstd;
                }
            }
        });
        __syncthreads();
    }
    if (every) {
        float mean[N], r[N], b[N];
        if (a.b) {
            P::widen(P::load((const E *)a.b + t.at), b);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) b[e] = 0.0f;
        }
        if (a.w) {
            P::widen(P::load((const E *)a.w + t.at), r);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) r[e] = 1.0f;
        }
        int g = (int)fdiv(t.at, p.by_D), c = t.at - g * a.D;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float2 s = p.joined ? joined[g] : stat[t.b * a.G + g];
            mean[e] = s.x, r[e] *= s.y;
            if (++c == a.D) c = 0, g = min(g + 1, a.G - 1);
        }
        for (int i0 = 0; i0 < every; i0 += kBatch) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) raw[i] = next[i];
            if (i0 + kBatch < every) load(i0 + kBatch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i0 + i >= every) break;
                float f[N];
                hold(raw[i]);
                P::widen(raw[i], f);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    f[e] = i0 + i < mine ? activate<ACT>((f[e] - mean[e]) * r[e] + b[e]) : 0.0f;
                    hold(f[e]);
                }
                store_own<T, N>((E *)(y + (t.off + (uint32_t)(i0 + i) * t.step)), f, t.skip, a.y == a.x);
            }
        }
    }
}

template <typename T, int N, int R, int ACT>
hipError_t run_held(const GroupNormArgs &a, const HeldPlan &p, hipStream_t stream) {
    const int64_t jobs = p.batches * p.slabs;
    for (int64_t first = 0; first < jobs; first += kMaxGrid) {
        const dim3 grid((unsigned)std::min(jobs - first, kMaxGrid)), block(p.nt);
        if (p.mode == kShuffle)
            hipLaunchKernelGGL((k_gn_held<T, N, R, kShuffle, ACT>), grid, block, p.lds, stream, a, p, first);
        else if (p.mode == kWhole)
            hipLaunchKernelGGL((k_gn_held<T, N, R, kWhole, ACT>), grid, block, p.lds, stream, a, p, first);
        else if (p.mode == kOne)
            hipLaunchKernelGGL((k_gn_held<T, N, R, kOne, ACT>), grid, block, p.lds, stream, a, p, first);
        else if constexpr (R <= 8)
            hipLaunchKernelGGL((k_gn_held<T, N, R, kMixed, ACT>), grid, block, p.lds, stream, a, p, first);
    }
    return hipGetLastError();
}

template <typename T, int N, int ACT>
hipError_t run(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    const HeldPlan h = plan_held(a.B, a.S, a.C, a.G, N, sizeof(typename T::T), 1, num_cus);
    if constexpr (N > 1) {
        switch (h.R) {
        case 1: return run_held<T, N, 1, ACT>(a, h, stream);
        case 2: return run_held<T, N, 2, ACT>(a, h, stream);
        case 4: return run_held<T, N, 4, ACT>(a, h, stream);
        case 8: return run_held<T, N, 8, ACT>(a, h, stream);
        case 16: return run_held<T, N, 16, ACT>(a, h, stream);
        }
    }
    const GnParts p = plan_parts(a.B, a.S, a.C, a.G, N, sizeof(typename T::T), num_cus);
    float2 *const channels = (float2 *)a.ws, *const part = (float2 *)((char *)a.ws + p.channel_bytes);
    float2 *const stat = (float2 *)((char *)part + p.part_bytes);
    const size_t lds = (size_t)(p.rt + 1) * p.tp * N * sizeof(float2);
    by_samples(a.B, p, 1, false, [&](int64_t b, dim3 grid) {
        hipLaunchKernelGGL((k_gn_part_stats<T, N>), grid, dim3(p.nt), lds, stream, a, p, channels, part, b);
    });
    if (!p.by_group) hipLaunchKernelGGL(k_gn_fold, dim3(grid_for(a.B * p.parts)), dim3(256), 0, stream, a, p, channels, part);
    if (!p.joined) {
        if (p.parts <= 256)
            hipLaunchKernelGGL((k_gn_join<64>), dim3(grid_for(a.B * a.G)), dim3(64), 0, stream, a, p, part, stat);
        else
            hipLaunchKernelGGL((k_gn_join<1024>), dim3(grid_for(a.B * a.G)), dim3(1024), 0, stream, a, p, part, stat);
    }
    const size_t here = p.joined ? (size_t)a.G * (1 + p.parts) * sizeof(float2) : 0;
    by_samples(a.B, p, p.split, true, [&](int64_t b, dim3 grid) {
        hipLaunchKernelGGL((k_gn_part_apply<T, N, ACT>), grid, dim3(p.nt), here, stream, a, p, part, stat, b);
    });
    return hipGetLastError();
}

}  // namespace

size_t group_norm_workspace(int64_t B, int64_t S, int C, int G, int dtype, int num_cus) {
    const int N = piece_size(C, dtype);
    if (plan_held(B, S, C, G, N, dtype == kF32 ? 4 : 2, 1, num_cus).R) return 0;
    const GnParts p = plan_parts(B, S, C, G, N, dtype == kF32 ? 4 : 2, num_cus);
    return p.channel_bytes + p.part_bytes + p.stat_bytes;
}

hipError_t launch_group_norm(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    return by_activation(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (a.dtype == kF32) return a.C >= 4 ? run<F32, 4, ACT>(a, num_cus, stream) : run<F32, 1, ACT>(a, num_cus, stream);
        return a.C >= 8 ? run<BF16, 8, ACT>(a, num_cus, stream) : run<BF16, 1, ACT>(a, num_cus, stream);
    });
}

}  // namespace dc1d
