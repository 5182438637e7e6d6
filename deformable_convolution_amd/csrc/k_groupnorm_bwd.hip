// k_groupnorm_bwd.hip -- the gradients of k_groupnorm.hip's group norm.
#include "groupnorm.h"

namespace dc1d {

namespace {

// Gradients: a workgroup strides over the batches of its slab; a thread keeps its
// channels' parameter gradients, which it leaves in the workspace at the end
// ([workgroup of the slab][C]), at most eight workgroups a CU of them.  The rows are
// taken from registers twice: in 32 bits the first time leaves xh and g' there (45.5
// -> 42.8 us below), in bf16 z is formed anew.  32768 rows of 1024 bf16: 41 us, 4.9
// TB/s; 32 x 784 x 512 fp32, silu: 43 us with the parameters' sums, 3.6 TB/s, where
// eight rows a thread of both tensors leave four waves a SIMD; 512 x 49 x 1024 bf16,
// silu: 66 us, 62 instructions an element.
template <typename T, int N, int R, int MODE, int ACT>
__global__ __launch_bounds__(512) void k_gn_held_back(GroupNormArgs a, HeldPlan p, float2 *out) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float lds[];
    const uint32_t id = p.slabs > 1 ? by_xcd(blockIdx.x, gridDim.x) : blockIdx.x;
    const int slab = (int)(id % p.slabs), w0 = (int)(id / p.slabs);
    const HeldPlace<N, MODE> t(a, p, slab);
    constexpr int NV = HeldPlace<N, MODE>::NV;
    GroupSums<N, MODE> sum(p, lds);
    float w[N], c[N], pw[N] = {}, pb[N] = {};
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 1.0f, c[e] = 0.0f;
    if (a.w) P::widen(P::load((const E *)a.w + t.at), w);
    if (a.b) P::widen(P::load((const E *)a.b + t.at), c);
    for (int64_t batch = w0; batch < p.batches; batch += p.grid_rows) {
        const int64_t b = min(batch * p.nb + t.sm, a.B - 1);
        const bool on = t.in && batch * p.nb + t.sm < a.B;
        const int n = (int)positions(a, b), s = (int)(b - batch * p.nb);
        const int64_t base = batch * p.nb * a.S * a.C * (int64_t)sizeof(E);
        const char *const x = (const char *)a.x + base, *const g = (const char *)a.g + base;
        typename P::Raw xr[R], gr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t at = t.offset(a, p, sizeof(E), s, i, on && t.rt + i * p.rt < n);
            xr[i] = P::load((const E *)(x + at));
            gr[i] = P::load((const E *)(g + at));
        }
        float mean[NV], r[NV], v[2][NV] = {};
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int64_t k = b * a.G + min(t.group + t.of[e], a.G - 1);
            mean[e] = a.mean[k], r[e] = a.rstd[k];
        }
        auto back = [&](int i, float *xh, float *u) {
            hold(xr[i]);
            hold(gr[i]);
            P::widen(xr[i], xh);
            P::widen(gr[i], u);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                xh[e] = (xh[e] - mean[t.v(e)]) * r[t.v(e)];
                u[e] = activate_back<ACT>(xh[e] * w[e] + c[e], u[e]);
            }
            if constexpr (sizeof(E) == 4) {
                xr[i] = Vec<T>::narrow(xh);
                gr[i] = Vec<T>::narrow(u);
            }
        };
        auto again = [&](int i, float *xh, float *u) {
            if constexpr (sizeof(E) == 4) {
                hold(xr[i]);
                hold(gr[i]);
                P::widen(xr[i], xh);
                P::widen(gr[i], u);
            } else {
                back(i, xh, u);
            }
        };
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool see = on && t.rt + i * p.rt < n;
            if (!__all(see)) {  // zeros add nothing, whatever stands there
                const typename P::Raw zero = {};
                if (!see) xr[i] = zero, gr[i] = zero;
            }
            float xh[N], u[N];
            back(i, xh, u);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const bool own = (MODE != kMixed && MODE != kOne) || e >= t.skip;
                const float d = own ? u[e] : 0.0f, dx = own ? u[e] * xh[e] : 0.0f;
                pb[e] += d;
                pw[e] += dx;
                v[0][t.v(e)] += d * w[e];
                v[1][t.v(e)] += dx * w[e];
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                hold(pb[e]);
                hold(pw[e]);
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                hold(v[0][e]);
                hold(v[1][e]);
            }
        }
        if (!a.y) continue;
        sum(p, v, t.channels, a.D, t.slot, t.of);
        const float inv = n > 0 ? 1.0f / ((float)n * (float)a.D) : 0.0f;
        if (on) {
            char *const y = (char *)a.y + base;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = t.rt + i * p.rt;
                if (row >= a.S) continue;
                float xh[N], u[N];
                again(i, xh, u);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    u[e] = r[t.v(e)] * (u[e] * w[e] - v[0][t.v(e)] * inv - xh[e] * (v[1][t.v(e)] * inv));
                    hold(u[e]);
                }
                if (row >= n)
#pragma unroll
                    for (int e = 0; e < N; ++e) u[e] = 0.0f;
                put<T, N, MODE>(y + t.offset(a, p, sizeof(E), s, i, true), u, t.skip, a.y == a.g || t.channels < N);
            }
        }
    }
    if (!out) return;
    float2 *const red = (float2 *)lds;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < N; ++e) red[threadIdx.x * N + e] = make_float2(pb[e], pw[e]);
    __syncthreads();
    const int last = (t.channels + N - 1) / N - 1, c0 = slab * p.gs * a.D;
    for (int j = threadIdx.x; j < t.channels; j += p.nt) {
        const int at = j >= last * N ? last * N + j - (t.channels - N) : j;
        float2 s = make_float2(0.0f, 0.0f);
        for (int q = 0; q < p.nb * p.rt; ++q) {
            const float2 d = red[q * p.P * N + at];
            s.x += d.x, s.y += d.y;
        }
        out[(int64_t)w0 * a.C + c0 + j] = s;
    }
}

// ---- gradients in parts ------------------------------------------------------------

// What a thread keeps of its channels.
template <typename T, int N>
struct Channels {
    float mean[N], r[N], w[N], b[N];
    __device__ __forceinline__ Channels(const GroupNormArgs &a, const GnParts &p, int64_t sample, int at) {
        using P = Piece<T, N>;
        using E = typename T::T;
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = 1.0f, b[e] = 0.0f;
        if (a.w) P::widen(P::load((const E *)a.w + at), w);
        if (a.b) P::widen(P::load((const E *)a.b + at), b);
        int g = (int)fdiv(at, p.by_D), c = at - g * a.D;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t k = sample * a.G + g;
            mean[e] = a.mean[k], r[e] = a.rstd[k];
            if (++c == a.D) c = 0, g = min(g + 1, a.G - 1);
        }
    }
    // x becomes xh and g becomes g'
    template <int ACT>
    __device__ __forceinline__ void back(float *x, float *g) const {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            x[e] = (x[e] - mean[e]) * r[e];
            g[e] = activate_back<ACT>(x[e] * w[e] + b[e], g[e]);
        }
    }
};

// sum g' and sum g' xh of every channel over a part, [b][part][C], and where a
// tile holds every group sum u and sum u xh of each, [b][part][G].
template <typename T, int N, int ACT>
__global__ __launch_bounds__(512) void k_gn_part_sums(GroupNormArgs a, GnParts p, float2 *out, float2 *groups, int64_t first) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 red[];
    const Place<T, N> t = Place<T, N>::template of<false>(a, p, first, blockIdx.x);
    const char *const x = (const char *)a.x + t.base, *const g = (const char *)a.g + t.base;
    const int mine = t.on ? t.rows_of(p, t.rt, t.n) : 0;
    float s1[N] = {}, s2[N] = {};
    constexpr int U = kBatch / 2;
    typename P::Raw xr[U], gr[U], xn[U], gn[U];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t at = t.off + (uint32_t)min(i0 + i, mine - 1) * t.step;
            xn[i] = P::load((const E *)(x + at));
            gn[i] = P::load((const E *)(g + at));
        }
    };
    if (mine) {
        load(0);
        const Channels<T, N> ch(a, p, t.b, t.at);
        for (int i0 = 0; i0 < mine; i0 += U) {
#pragma unroll
            for (int i = 0; i < U; ++i) xr[i] = xn[i], gr[i] = gn[i];
            if (i0 + U < mine) load(i0 + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float xh[N], u[N];
                hold(xr[i]);
                hold(gr[i]);
                P::widen(xr[i], xh);
                P::widen(gr[i], u);
                ch.template back<ACT>(xh, u);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    s1[e] += i0 + i < mine ? u[e] : 0.0f;
                    s2[e] += i0 + i < mine ? u[e] * xh[e] : 0.0f;
                    hold(s1[e]);
                    hold(s2[e]);
                }
            }
        }
    }
    if (t.on)
#pragma unroll
        for (int e = 0; e < N; ++e) red[(t.rt * p.tp + t.j) * N + e] = make_float2(s1[e], s2[e]);
    __syncthreads();
    const int channels = p.tp * N;
    float2 *const o = out + (t.b * p.parts + t.part) * a.C;
    for (int k = threadIdx.x; k < channels; k += blockDim.x) {
        const int piece = t.tile * p.tp + k / N, c = piece * N;
        if (piece >= p.P) continue;
        const int at = min(c, a.C - N);
        if (k % N < c - at) continue;
        float2 s = make_float2(0.0f, 0.0f);
        for (int i = 0; i < p.rt; ++i) {
            s.x += red[i * channels + k].x;
            s.y += red[i * channels + k].y;
        }
        o[at + k % N] = s;
        red[k] = s;  // row 0 is read by this thread alone
    }
    __syncthreads();
    if (p.by_group)
        each_group(a, p, [&](int k, int lane) {
            float u = 0.0f, ux = 0.0f;
            for (int i = lane; i < a.D; i += p.team) {
                const int c = k * a.D + i;
                const float2 s = red[c >= (p.P - 1) * N ? (p.P - 1) * N + c - (a.C - N) : c];
                const float w = a.w ? T::ld((const E *)a.w, c) : 1.0f;
                u += s.x * w;
                ux += s.y * w;
            }
            u = team_sum(p, u);
            ux = team_sum(p, ux);
            if (lane == 0) groups[(t.b * p.parts + t.part) * a.G + k] = make_float2(u, ux);
        });
}

// A part's groups from its channels.
template <typename T>
__global__ __launch_bounds__(256) void k_gn_fold_back(GroupNormArgs a, GnParts p, const float2 *channels, float2 *groups) {
    using E = typename T::T;
    const int64_t jobs = a.B * p.parts;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const float2 *const v = channels + job * a.C;
        each_group(a, p, [&](int g, int lane) {
            float u = 0.0f, ux = 0.0f;
            const int64_t c0 = (int64_t)g * a.D;
            each_channel(p, v + c0, a.D, lane, [&](float2 e, int i) {
                const float w = a.w ? T::ld((const E *)a.w, c0 + i) : 1.0f;
                u += e.x * w;
                ux += e.y * w;
            });
            u = team_sum(p, u);
            ux = team_sum(p, ux);
            if (lane == 0) groups[job * a.G + g] = make_float2(u, ux);
        });
    }
}

// mean u and mean(u xh) of a group.
template <int NT>
__global__ __launch_bounds__(NT) void k_gn_join_back(GroupNormArgs a, GnParts p, const float2 *groups, float2 *stat) {
    __shared__ float red[NT / 64];
    const int64_t jobs = a.B * a.G;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t b = job / a.G, n = positions(a, b);
        float s = 0.0f, q = 0.0f;
        each_part<NT>(p, a.G, groups + b * p.parts * a.G + job % a.G, n, [&](float2 e, float) { s += e.x, q += e.y; });
        s = all_sum<NT>(s, red);
        q = all_sum<NT>(q, red);
        const float inv = n > 0 ? 1.0f / ((float)n * (float)a.D) : 0.0f;
        if (threadIdx.x == 0) stat[job] = make_float2(s * inv, q * inv);
    }
}

template <typename T, int N, int ACT>
__global__ __launch_bounds__(512) void k_gn_part_back(GroupNormArgs a, GnParts p, const float2 *groups, const float2 *stat, int64_t first) {
    using P = Piece<T, N>;
    using E = typename T::T;
    extern __shared__ float2 joined[];
    const Place<T, N> t = Place<T, N>::template of<true>(a, p, first, gridDim.x - 1 - blockIdx.x);
    const char *const x = (const char *)a.x + t.base, *const g = (const char *)a.g + t.base;
    char *const y = (char *)a.y + t.base;
    const int mine = t.on ? t.rows_of(p, t.rt, t.n) : 0, every = t.on ? t.rows_of(p, t.rt, t.rows) : 0;
    constexpr int U = kBatch / 2;
    typename P::Raw xr[U], gr[U], xn[U], gn[U];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t at = t.off + (uint32_t)max(min(i0 + i, mine - 1), 0) * t.step;
            xn[i] = P::load((const E *)(x + at));
            gn[i] = P::load((const E *)(g + at));
        }
    };
    if (every) load(0);
    if (p.joined) {
        const int64_t n = positions(a, t.b);
        const float inv = n > 0 ? 1.0f / ((float)n * (float)a.D) : 0.0f;
        float2 *const v = joined + a.G;
        fetch_parts(a, p, groups, t.b, v);
        each_group(a, p, [&](int i, int lane) {
            float s = 0.0f, q = 0.0f;
            for (int j = lane; j < p.parts; j += p.team) s += v[j * a.G + i].x, q += v[j * a.G + i].y;
            s = team_sum(p, s);
            q = team_sum(p, q);
            if (lane == 0) joined[i] = make_float2(s * inv, q * inv);
        });
        __syncthreads();
    }
    if (every) {
        const Channels<T, N> ch(a, p, t.b, t.at);
        float c1[N], c2[N];
        int i = (int)fdiv(t.at, p.by_D), c = t.at - i * a.D;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float2 s = p.joined ? joined[i] : stat[t.b * a.G + i];
            c1[e] = s.x, c2[e] = s.y;
            if (++c == a.D) c = 0, i = min(i + 1, a.G - 1);
        }
        for (int i0 = 0; i0 < every; i0 += U) {
#pragma unroll
            for (int i = 0; i < U; ++i) xr[i] = xn[i], gr[i] = gn[i];
            if (i0 + U < every) load(i0 + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (i0 + i >= every) break;
                float xh[N], u[N];
                hold(xr[i]);
                hold(gr[i]);
                P::widen(xr[i], xh);
                P::widen(gr[i], u);
                ch.template back<ACT>(xh, u);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    u[e] = i0 + i < mine ? ch.r[e] * (u[e] * ch.w[e] - c1[e] - xh[e] * c2[e]) : 0.0f;
                    hold(u[e]);
                }
                store_own<T, N>((E *)(y + (t.off + (uint32_t)(i0 + i) * t.step)), u, t.skip, a.y == a.g);
            }
        }
    }
}

// The parameters' gradients: sum over `rows` rows of [C] pairs (sum g', sum g' xh).
// 16 channels of 64 row-threads; the rows of a thread, then the threads in order.
template <typename T>
__global__ __launch_bounds__(1024) void k_gn_params(const float2 *sums, int64_t rows, int C, void *gw, void *gb) {
    using E = typename T::T;
    __shared__ float2 red[64][17];
    const int64_t c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const int r0 = threadIdx.x >> 4;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < C) {
        int64_t r = r0;
        for (; r + 7 * 64 < rows; r += 8 * 64) {
            float2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = sums[(r + i * 64) * C + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) s.x += v[i].x, s.y += v[i].y;
        }
        for (; r < rows; r += 64) {
            const float2 v = sums[r * C + c];
            s.x += v.x, s.y += v.y;
        }
    }
    red[r0][threadIdx.x & 15] = s;
    __syncthreads();
    if (r0 == 0 && c < C) {
#pragma unroll 8
        for (int i = 1; i < 64; ++i) s.x += red[i][threadIdx.x].x, s.y += red[i][threadIdx.x].y;
        if (gw) T::st((E *)gw, c, s.y);
        if (gb) T::st((E *)gb, c, s.x);
    }
}

// The workspace: the parts' sums of channels and of groups, the joined ones.
struct BackBytes {
    size_t part, groups;
};
BackBytes back_bytes(int64_t B, int C, int G, const GnParts &p) {
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    return {up((size_t)B * p.parts * C * sizeof(float2)), up((size_t)B * p.parts * G * sizeof(float2))};
}

template <typename T, int N, int R, int ACT>
hipError_t run_held_back(const GroupNormArgs &a, const HeldPlan &p, hipStream_t stream) {
    float2 *const out = a.gw || a.gb ? (float2 *)a.ws : nullptr;
    const dim3 grid((unsigned)(p.grid_rows * p.slabs)), block(p.nt);
    if (p.mode == kShuffle)
        hipLaunchKernelGGL((k_gn_held_back<T, N, R, kShuffle, ACT>), grid, block, p.lds, stream, a, p, out);
    else if (p.mode == kWhole)
        hipLaunchKernelGGL((k_gn_held_back<T, N, R, kWhole, ACT>), grid, block, p.lds, stream, a, p, out);
    else if (p.mode == kOne)
        hipLaunchKernelGGL((k_gn_held_back<T, N, R, kOne, ACT>), grid, block, p.lds, stream, a, p, out);
    else
        hipLaunchKernelGGL((k_gn_held_back<T, N, R, kMixed, ACT>), grid, block, p.lds, stream, a, p, out);
    if (out) hipLaunchKernelGGL((k_gn_params<T>), dim3((a.C + 15) / 16), dim3(1024), 0, stream, out, (int64_t)p.grid_rows, a.C, a.gw, a.gb);
    return hipGetLastError();
}

template <typename T, int N, int ACT>
hipError_t run_back(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    const HeldPlan h = plan_held(a.B, a.S, a.C, a.G, N, sizeof(typename T::T), 2, num_cus);
    if constexpr (N > 1) {
        switch (a.B > 0 ? h.R : 0) {
        case 1: return run_held_back<T, N, 1, ACT>(a, h, stream);
        case 2: return run_held_back<T, N, 2, ACT>(a, h, stream);
        case 4: return run_held_back<T, N, 4, ACT>(a, h, stream);
        case 8: return run_held_back<T, N, 8, ACT>(a, h, stream);
        }
    }
    const GnParts p = plan_parts(a.B, a.S, a.C, a.G, N, sizeof(typename T::T), num_cus);
    const BackBytes by = back_bytes(a.B, a.C, a.G, p);
    float2 *const part = (float2 *)a.ws, *const groups = (float2 *)((char *)a.ws + by.part), *const stat = (float2 *)((char *)groups + by.groups);
    const size_t lds = (size_t)p.rt * p.tp * N * sizeof(float2);
    by_samples(a.B, p, 1, false, [&](int64_t b, dim3 grid) {
        hipLaunchKernelGGL((k_gn_part_sums<T, N, ACT>), grid, dim3(p.nt), lds, stream, a, p, part, groups, b);
    });
    if (a.y && a.B > 0 && a.S > 0) {
        if (!p.by_group) hipLaunchKernelGGL((k_gn_fold_back<T>), dim3(grid_for(a.B * p.parts)), dim3(256), 0, stream, a, p, part, groups);
        if (!p.joined) {
            if (p.parts <= 256)
                hipLaunchKernelGGL((k_gn_join_back<64>), dim3(grid_for(a.B * a.G)), dim3(64), 0, stream, a, p, groups, stat);
            else
                hipLaunchKernelGGL((k_gn_join_back<1024>), dim3(grid_for(a.B * a.G)), dim3(1024), 0, stream, a, p, groups, stat);
        }
        const size_t here = p.joined ? (size_t)a.G * (1 + p.parts) * sizeof(float2) : 0;
        by_samples(a.B, p, p.split, true, [&](int64_t b, dim3 grid) {
            hipLaunchKernelGGL((k_gn_part_back<T, N, ACT>), grid, dim3(p.nt), here, stream, a, p, groups, stat, b);
        });
    }
    if (a.gw || a.gb)
        hipLaunchKernelGGL((k_gn_params<T>), dim3((a.C + 15) / 16), dim3(1024), 0, stream, part, a.B * p.parts, a.C, a.gw, a.gb);
    return hipGetLastError();
}

}  // namespace

size_t group_norm_backward_workspace(int64_t B, int64_t S, int C, int G, int dtype, bool want_params, int num_cus) {
    const int N = piece_size(C, dtype);
    const HeldPlan h = plan_held(B, S, C, G, N, dtype == kF32 ? 4 : 2, 2, num_cus);
    if (h.R) return want_params ? (size_t)h.grid_rows * C * sizeof(float2) : 0;
    const GnParts p = plan_parts(B, S, C, G, N, dtype == kF32 ? 4 : 2, num_cus);
    const BackBytes by = back_bytes(B, C, G, p);
    return by.part + by.groups + p.stat_bytes;
}

hipError_t launch_group_norm_backward(const GroupNormArgs &a, int num_cus, hipStream_t stream) {
    return by_activation(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (a.dtype == kF32) return a.C >= 4 ? run_back<F32, 4, ACT>(a, num_cus, stream) : run_back<F32, 1, ACT>(a, num_cus, stream);
        return a.C >= 8 ? run_back<BF16, 8, ACT>(a, num_cus, stream) : run_back<BF16, 1, ACT>(a, num_cus, stream);
    });
}

}  // namespace dc1d
