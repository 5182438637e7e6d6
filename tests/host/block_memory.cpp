// What group norm and the gated recurrence address, on the host, over several
// counts of compute units (tests/test_block_memory.py builds and runs this; no
// GPU is used): the last byte that each form leaves in a workspace lies in what
// the library asks for, and the rows that a recurrence's tile reads and writes
// are the sequence's own, each once, whichever its length and direction.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <type_traits>
#include <vector>

// The kernels' own address arithmetic, called from here: their device functions
// are the host's too, for a thread that this program names.
static inline __host__ __device__ uint32_t high_product(uint32_t a, uint32_t b) { return (uint32_t)(((uint64_t)a * b) >> 32); }
static struct {
    unsigned x;
} this_thread;
#ifndef __HIP_DEVICE_COMPILE__
#define threadIdx this_thread
#endif
#define __umulhi high_product
#undef __device__
#define __device__ __attribute__((host)) __attribute__((device))
#include "groupnorm.h"
#include "k_recurrence.hip"

using namespace dc1d;

static int failures = 0;
static long checks = 0;

static void workspace(const char *what, int64_t last, size_t have, int64_t B, int64_t S, int64_t C, int64_t G, int dtype, int cus) {
    ++checks;
    if (last <= (int64_t)have) return;
    ++failures;
    printf("%s, %lld x %lld x %lld, %lld groups, type %d, %d CUs: %lld bytes written of %zu\n", what, (long long)B, (long long)S, (long long)C,
           (long long)G, dtype, cus, (long long)last, have);
}

constexpr int64_t kPair = 8;  // two floats
static int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

static void group_norms(int64_t B, int64_t S, int C, int G, int dtype, int cus) {
    const int es = dtype == kF32 ? 4 : 2, N = piece_size(C, dtype), D = C / G;
    const HeldPlan f = plan_held(B, S, C, G, N, es, 1, cus), b = plan_held(B, S, C, G, N, es, 2, cus);
    const GnParts p = plan_parts(B, S, C, G, N, es, cus);
    const size_t have = group_norm_workspace(B, S, C, G, dtype, cus);
    const int64_t rows = B * p.parts;
    if (!f.R) {
        const int64_t channels = p.by_group ? 0 : up(rows * C * kPair), groups = channels + up(rows * G * kPair);
        workspace("group norm, parts' groups", channels + rows * G * kPair, have, B, S, C, G, dtype, cus);
        if (!p.joined) workspace("group norm, joined", groups + B * G * kPair, have, B, S, C, G, dtype, cus);
    }
    for (int params : {0, 1}) {
        const size_t has = group_norm_backward_workspace(B, S, C, G, dtype, params != 0, cus);
        if (b.R) {
            // the workgroups of every slab leave a row of all channels
            const int64_t last = ((int64_t)(b.grid_rows - 1) * C + C) * kPair;
            if (params) workspace("group norm gradients, held", last, has, B, S, C, G, dtype, cus);
        } else {
            const int64_t groups = up(rows * C * kPair), joined = groups + up(rows * G * kPair);
            workspace("group norm gradients, parts", groups + rows * G * kPair, has, B, S, C, G, dtype, cus);
            if (!p.joined) workspace("group norm gradients, joined", joined + B * G * kPair, has, B, S, C, G, dtype, cus);
        }
    }
    if (B == 0) return;  // no launch of either form's kernels of rows
    // every row and piece of a sample has one thread, and LDS holds their sums
    for (int tensors : {1, 2}) {
        const HeldPlan &h = tensors == 1 ? f : b;
        ++checks;
        if (!h.R) continue;
        const int NV = h.mode == kMixed ? N : 1;
        const bool ok = h.nt <= (tensors == 1 ? 1024 : 512) && h.nb * h.rt * h.P <= h.nt && (int64_t)h.rt * h.R >= S && h.P * N >= h.gs * D &&
                        h.gs * D >= N && (int64_t)h.slabs * h.gs >= G && (int64_t)(h.slabs - 1) * h.gs < G && h.batches * h.nb >= B &&
                        (h.batches - 1) * h.nb < B && h.nb * S * C * es <= (int64_t)1 << 31 && h.lds <= 64 * 1024 && h.grid_rows >= 1 &&
                        h.grid_rows <= h.batches && (h.mode == kShuffle || h.lds >= (size_t)2 * (h.nt * NV + h.nb * h.gs) * sizeof(float)) &&
                        (tensors == 1 || h.lds >= (size_t)h.nt * N * kPair);
        if (!ok) {
            ++failures;
            printf("held, %d tensors, %lld x %lld x %d in %d, type %d, %d CUs\n", tensors, (long long)B, (long long)S, C, G, dtype, cus);
        }
    }
    ++checks;
    if (p.rt < 1 || p.rt * p.tp > p.nt || p.nt > 512 || p.tiles * p.tp < p.P || p.P * N < C || p.parts * p.rows < S ||
        (S > 0 && (p.parts - 1) * p.rows >= S) || p.rows * C * es > (int64_t)1 << 31 || (p.joined && (int64_t)G * (1 + p.parts) * kPair > 64 * 1024)) {
        ++failures;
        printf("parts, %lld x %lld x %d in %d, type %d, %d CUs\n", (long long)B, (long long)S, C, G, dtype, cus);
    }
}

static void recurrences(int64_t B, int64_t L, int64_t C, int dtype, int cus) {
    for (bool backward : {false, true}) {
        const size_t have = recurrence_workspace((int)B, (int)L, (int)C, dtype, backward, cus);
        for (int N : {1, 4}) {
            if (N > C) continue;
            const RecPlan p = plan_recurrence((int)B, (int)L, (int)C, N, dtype, backward, cus);
            const int64_t chains = B * ((C + N * kLanes - 1) / (N * kLanes)), tile = p.slots * (backward ? kPerBack : kPer);
            if (p.g.segs > 1)
                workspace("recurrence", (((chains - 1) * p.g.segs + p.g.segs - 1) * kLanes + kLanes) * N * kPair, have, B, L, C, p.g.segs, dtype, cus);
            // the segments cover the sequence, none of them empty
            ++checks;
            if ((int64_t)p.g.segs * p.g.tiles * tile < L || (int64_t)(p.g.segs - 1) * p.g.tiles * tile >= L || (int64_t)p.g.jobs != chains * p.g.segs ||
                (p.g.segs > 1 && p.slots != kSlots) || (p.slots != kSlots && p.slots != 2 * kSlots)) {
                ++failures;
                printf("recurrence plan, %lld x %lld x %lld, %d CUs\n", (long long)B, (long long)L, (long long)C, cus);
            }
        }
    }
}

// The rows of one tile, as Tile::load and Tile::store take them.
template <typename T, int N, int SL>
static void rows(int L, int n, bool reverse, int64_t step, int64_t batch) {
    constexpr int PER = kPer, TILE = SL * PER;
    const int C = 70, b = 1;
    static char memory[1];  // addresses only
    int lens[2] = {0, n};
    RecurrenceArgs a;
    memset((void *)&a, 0, sizeof(a));
    a.B = 2, a.L = L, a.C = C, a.reverse = reverse, a.lens = lens;
    const Strides2 st = {batch, step};
    const int slabs = (C + N * kLanes - 1) / (N * kLanes);
    const FastDiv by_slabs = make_fastdiv((uint32_t)slabs);
    std::vector<int> written(L, 0);
    bool bad = false;
    for (int slab : {0, slabs - 1})
        for (int i = 0; i * TILE < L; ++i)
            for (int thread : {0, kLanes - 1, 7 * kLanes + 3, (SL - 1) * kLanes, SL * kLanes - 1, -1})
                for (int slot = 0; slot < (thread < 0 ? SL : 1); ++slot) {
                    this_thread.x = thread < 0 ? slot * kLanes : thread;
                    const Lane<N> t(a, (uint32_t)(b * slabs + slab), by_slabs);
                    bad = bad || t.n != std::min(n, L) || t.at < 0 || t.at + N > C;
                    const int from = last_tile<TILE>(t.n, i), last = std::max(t.n, 1) - 1 - from * TILE - t.slot * PER;
                    const Walk<T, N, PER, SL> w(memory, st, a, t, from), y(memory, st, a, t, i);
                    const bool full = (i + 1) * TILE <= t.n;
                    const int left = t.n - i * TILE - t.slot * PER;
                    constexpr int64_t es = sizeof(typename T::T);
                    auto row = [&](const void *p) {
                        const int64_t at = (const char *)p - memory - (batch + t.at) * es;
                        bad = bad || at % (step * es);
                        return at / (step * es);
                    };
                    for (int k = 0; k < PER; ++k) {
                        ++checks;
                        const int64_t r = row(full ? w.at(k) : w.any(std::min(k, last)));
                        const int s = i * TILE + t.slot * PER + k;  // the position in the recurrence's order
                        const int own = reverse ? t.n - 1 - s : s;
                        bad = bad || r < 0 || r >= std::max(t.n, 1) || (s < t.n && r != own);
                        if (!full && k >= left) continue;
                        bad = bad || s >= t.n || row(y.at(k)) != own;
                        if (thread < 0 && slab == 0) ++written[s];
                    }
                }
    for (int s = 0; s < L; ++s) bad = bad || written[s] != (s < std::min(n, L));
    if (bad) {
        ++failures;
        printf("rows of a tile: L %d, length %d, reverse %d, pieces of %d, %d slots, step %lld\n", L, n, reverse, N, SL, (long long)step);
    }
}

int main() {
    for (int cus : {32, 64, 256, 304})
        for (int dtype : {(int)kF32, (int)kBF16})
            for (int C : {1, 3, 4, 7, 8, 33, 64, 90, 255, 333, 510, 890, 1024, 2056, 4105, 5000, 32768, 1 << 20, 1 << 24})
                for (int64_t S : {0, 1, 2, 9, 65, 194, 784, 2501, 4096, 16384, 1 << 20})
                    for (int64_t B : {0, 1, 2, 13, 70, 300, 32768, 1 << 22}) {
                        if (B * std::max<int64_t>(S, 1) >= (int64_t)1 << 31 || B * std::max<int64_t>(S, 1) > ((int64_t)1 << 38) / C) continue;
                        for (int G : {1, 2, 3, 8, 9, 17, 32, 111, 512, 1 << 20})
                            if (C % G == 0 && B * G < (int64_t)1 << 31) group_norms(B, S, C, G, dtype, cus);
                        if (C % 5 == 0) group_norms(B, S, C, C, dtype, cus);
                    }
    for (int cus : {32, 64, 256, 304})
        for (int dtype : {(int)kF32, (int)kBF16})
            for (int64_t C : {1, 3, 4, 20, 64, 65, 512, 33000, 1 << 24})
                for (int64_t L : {1, 64, 65, 129, 700, 4092, 16384, 1 << 20, 1 << 29})
                    for (int64_t B : {1, 2, 16, 70, 511, 70000, 1 << 24})
                        if (B * L < (int64_t)1 << 31 && B * C < (int64_t)1 << 31 && B * L <= ((int64_t)1 << 38) / C) recurrences(B, L, C, dtype, cus);
    for (int L : {1, 2, 3, 4, 5, 63, 64, 65, 127, 128, 129, 200, 257, 513})
        for (int n : {0, 1, 2, 3, 4, 5, 60, 63, 64, 65, 66, 127, 128, 129, 130, 199, 200, 256, 512, 513, 514, 1 << 30})
            for (bool reverse : {false, true}) {
                if (n > L + 1 && n < 1 << 30) continue;
                rows<F32, 4, kSlots>(L, n, reverse, 70, 70 * L), rows<F32, 4, 2 * kSlots>(L, n, reverse, 75, 3);
                rows<BF16, 4, kSlots>(L, n, reverse, 141, 141 * L + 5), rows<BF16, 4, 2 * kSlots>(L, n, reverse, 70, 70 * L);
                rows<F32, 1, kSlots>(L, n, reverse, (int64_t)1 << 33, 1), rows<BF16, 1, 2 * kSlots>(L, n, reverse, 70, 70 * L);
                // the farthest rows that 32-bit offsets serve
                rows<F32, 4, 2 * kSlots>(L, n, reverse, (((int64_t)1 << 31) / 4 - 70) / (2 * kSlots * kPer), 1);
            }
    printf("block memory: %ld checks, %d failure(s)\n", checks, failures);
    return failures != 0;
}
