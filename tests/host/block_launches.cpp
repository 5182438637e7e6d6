// The launches of group norm and the gated recurrence over sizes up to the ends
// of their documented limits, with the runtime's launch calls replaced by ones
// that only look (tests/test_block_launches.py builds and runs this; no GPU is
// used): whichever launch fails is reported, a launch holds fewer than 2^32 threads, a workgroup at most 1024 and
// 64 KB of LDS.  Group norm's plans besides: every element of a sample has one
// thread's row and piece, 32-bit offsets span what they address, and the
// workspace holds what is kept in it.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "groupnorm.h"

using namespace dc1d;

static dim3 next_grid, next_block;
static size_t next_lds;
static int failures = 0, calls = 0, launches = 0;
static bool bad = false;
static int fails_at = 0;  // the launch that fails, counted from 1
static hipError_t last_error = hipSuccess;
extern "C" hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t) {
    next_grid = grid, next_block = block, next_lds = lds;
    return hipSuccess;
}
extern "C" hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream) {
    *grid = next_grid, *block = next_block, *lds = next_lds, *stream = nullptr;
    return hipSuccess;
}
extern "C" hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **, size_t lds, hipStream_t) {
    ++launches;
    bad = bad || grid.x < 1 || grid.y != 1 || grid.z != 1 || block.y != 1 || block.z != 1 || block.x < 64 || block.x > 1024 ||
          (int64_t)grid.x * block.x >= (int64_t)1 << 32 || lds > 64 * 1024;
    if (launches == fails_at) last_error = hipErrorLaunchFailure;
    return launches == fails_at ? hipErrorLaunchFailure : hipSuccess;
}
extern "C" hipError_t hipGetLastError() {
    const hipError_t e = last_error;
    last_error = hipSuccess;
    return e;
}

// Whichever launch of a call fails, the call says so.
template <typename F>
static void every_failure(const char *what, F call) {
    fails_at = launches = 0;
    if (call() != hipSuccess) ++failures;
    const int n = launches;
    for (int i = 1; i <= n; ++i) {
        fails_at = i, launches = 0;
        ++calls;
        if (call() == hipSuccess) {
            printf("%s: launch %d of %d failed unseen\n", what, i, n);
            ++failures;
        }
        last_error = hipSuccess;
    }
    fails_at = 0;
}

static void held_plan(const HeldPlan &p, int64_t B, int64_t S, int C, int G, int N, int es, int tensors) {
    const int D = C / G;
    bad = bad || p.nt > (tensors == 1 ? 1024 : 512) || p.nb * p.rt * p.P > p.nt || (int64_t)p.rt * p.R < S || p.R > (tensors == 1 ? 16 : 8) ||
          p.P * N < p.gs * D || p.gs * D < N || (int64_t)p.slabs * p.gs < G || (int64_t)(p.slabs - 1) * p.gs >= G || p.batches * p.nb < B ||
          (p.batches - 1) * p.nb >= B || p.nb * S * C * es > (int64_t)1 << 31 || p.lds > 64 * 1024 || (p.team & (p.team - 1)) || p.team < 1 ||
          p.team > 64 || p.grid_rows < 1 || p.grid_rows > p.batches;
    if (p.mode == kShuffle || p.mode == kWhole) bad = bad || D % N || p.gs * D != p.P * N;
    if (p.mode == kOne) bad = bad || p.gs != 1 || D < N || p.per != p.P;
    if (p.mode == kShuffle) bad = bad || p.rt != 1 || 64 % p.per || p.nb * p.P > p.nt || p.P % p.per;
    if (p.mode != kShuffle) bad = bad || p.lds < (size_t)tensors * (p.nt * (p.mode == kMixed ? N : 1) + p.nb * p.gs) * sizeof(float);
}

static void part_plan(const GnParts &p, int64_t B, int64_t S, int C, int G, int N, int es) {
    bad = bad || p.rt < 1 || p.rt * p.tp > p.nt || p.nt > 512 || p.tiles * p.tp < p.P || (p.tiles - 1) * p.tp >= p.P || p.P * N < C ||
          p.parts * p.rows < S || (S > 0 && (p.parts - 1) * p.rows >= S) || p.rows * C * es > (int64_t)1 << 31 || p.split < 1 ||
          p.part_bytes < (size_t)B * p.parts * G * sizeof(float2) ||
          (!p.by_group && p.channel_bytes < (size_t)B * p.parts * C * sizeof(float2)) || p.stat_bytes < (size_t)B * G * sizeof(float2) ||
          (p.joined && (size_t)G * (1 + p.parts) * sizeof(float2) > 64 * 1024) || (p.by_group && p.tiles != 1);
}

int main() {
    static char some[16];
    const int64_t top = ((int64_t)1 << 31) - 1;
    const int64_t groups[] = {1, 2, 3, 8, 17, 32, 512, 1 << 20, 1 << 24};
    for (int dtype : {(int)kF32, (int)kBF16})
        for (int64_t C : {1, 2, 3, 4, 7, 8, 9, 33, 64, 96, 255, 256, 511, 512, 1030, 2048, 2056, 4096, 5000, 32768, 1 << 20, (1 << 24) - 1, 1 << 24})
            for (int64_t S : {(int64_t)0, (int64_t)1, (int64_t)2, (int64_t)9, (int64_t)64, (int64_t)83, (int64_t)784, (int64_t)4092, (int64_t)4096,
                              (int64_t)16384, (int64_t)16385, (int64_t)1 << 20, top})
                for (int64_t B : {(int64_t)1, (int64_t)2, (int64_t)13, (int64_t)32, (int64_t)300, (int64_t)32768, (int64_t)1 << 22, top}) {
                    // what no memory holds besides
                    if (B * std::max<int64_t>(S, 1) > top || B * S > ((int64_t)1 << 38) / C) continue;
                    for (int64_t g : groups) {
                        const int64_t G = g > C ? C : g;
                        if (C % G || B * G > top) continue;
                        ++calls;
                        bad = false;
                        const int N = piece_size((int)C, dtype), es = dtype == kF32 ? 4 : 2;
                        for (int tensors : {1, 2}) {
                            const HeldPlan h = plan_held(B, S, (int)C, (int)G, N, es, tensors, 256);
                            if (h.R)
                                held_plan(h, B, S, (int)C, (int)G, N, es, tensors);
                            else
                                part_plan(plan_parts(B, S, (int)C, (int)G, N, es, 256), B, S, (int)C, (int)G, N, es);
                        }
                        const bool plans = bad;
                        GroupNormArgs a;
                        memset((void *)&a, 0, sizeof(a));
                        a.x = a.g = a.y = some, a.mean = a.rstd = (float *)some, a.gw = a.gb = some, a.ws = some;
                        a.dtype = dtype, a.B = B, a.S = S, a.C = (int)C, a.G = (int)G, a.D = (int)(C / G), a.act = kSilu;
                        bad = false;
                        launches = 0;
                        const bool launched = launch_group_norm(a, 256, nullptr) == hipSuccess && launch_group_norm_backward(a, 256, nullptr) == hipSuccess;
                        if (plans || bad || !launched || launches < 2) {
                            printf("group norm, %lld x %lld x %lld of %lld groups, type %d: plans %d, launches %d of %d\n", (long long)B,
                                   (long long)S, (long long)C, (long long)G, dtype, plans, bad, launches);
                            ++failures;
                        }
                    }
                }
    for (int dtype : {(int)kF32, (int)kBF16})
        for (int64_t C : {(int64_t)1, (int64_t)3, (int64_t)4, (int64_t)64, (int64_t)65, (int64_t)512, (int64_t)33000, (int64_t)1 << 24})
            for (int64_t L : {(int64_t)0, (int64_t)1, (int64_t)64, (int64_t)65, (int64_t)129, (int64_t)4092, (int64_t)16384, (int64_t)1 << 20, (int64_t)1 << 29})
                for (int64_t B : {(int64_t)1, (int64_t)2, (int64_t)16, (int64_t)511, (int64_t)512, (int64_t)70000, (int64_t)1 << 24, top})
                    for (int64_t far : {(int64_t)0, (int64_t)1 << 24}) {
                        if (B * std::max<int64_t>(L, 1) > top || B * C > top || B * L > ((int64_t)1 << 38) / C) continue;
                        ++calls;
                        RecurrenceArgs a;
                        memset((void *)&a, 0, sizeof(a));
                        a.x = a.gate = a.g = some, a.y = a.gx = a.gg = some, a.states = a.last = a.g_state = (float *)some, a.ws = some;
                        a.dtype = dtype, a.B = (int)B, a.L = (int)L, a.C = (int)C;
                        for (Strides2 *s : {&a.xs, &a.gates, &a.gs, &a.ys, &a.gxs, &a.ggs}) *s = {C * L, C + far};
                        bad = false;
                        launches = 0;
                        const bool launched = launch_recurrence(a, 256, nullptr) == hipSuccess && launch_recurrence_backward(a, 256, nullptr) == hipSuccess;
                        if (bad || !launched || launches < 2) {
                            printf("recurrence, %lld x %lld x %lld, type %d, %lld apart: %d in %d launches\n", (long long)B, (long long)L,
                                   (long long)C, dtype, (long long)far, bad, launches);
                            ++failures;
                        }
                    }
    for (int64_t S : {(int64_t)1, (int64_t)784, (int64_t)65536})
        for (int64_t G : {(int64_t)1, (int64_t)512}) {
            GroupNormArgs a;
            memset((void *)&a, 0, sizeof(a));
            a.x = a.g = a.y = some, a.mean = a.rstd = (float *)some, a.gw = a.gb = some, a.ws = some;
            a.dtype = kF32, a.B = 4, a.S = S, a.C = 512, a.G = (int)G, a.D = (int)(512 / G);
            every_failure("group norm", [&] { return launch_group_norm(a, 256, nullptr); });
            every_failure("group norm gradients", [&] { return launch_group_norm_backward(a, 256, nullptr); });
        }
    for (int L : {0, 1, 90, 16384}) {
        RecurrenceArgs a;
        memset((void *)&a, 0, sizeof(a));
        a.x = a.gate = a.g = some, a.y = a.gx = a.gg = some, a.states = a.last = a.g_state = (float *)some, a.ws = some;
        a.dtype = kF32, a.B = 2, a.L = L, a.C = 64;
        for (Strides2 *s : {&a.xs, &a.gates, &a.gs, &a.ys, &a.gxs, &a.ggs}) *s = {64 * L, 64};
        every_failure("recurrence", [&] { return launch_recurrence(a, 256, nullptr); });
        every_failure("recurrence gradients", [&] { return launch_recurrence_backward(a, 256, nullptr); });
    }
    printf("block launches: %d calls, %d failure(s)\n", calls, failures);
    return failures != 0;
}
