// The sequence operators' launches at the ends of their documented limits,
// with the runtime's launch calls replaced by ones that only look at the grid
// (tests/test_sequence_launches.py builds and runs this; no GPU is used).  A
// launch holds fewer than 2^32 threads, and the workgroups of all of a call's
// launches have to add up to what the call needs.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "seq_internal.h"

using namespace dc1d;

struct Launch {
    int64_t blocks, threads;
};
static std::vector<Launch> seen;

static dim3 next_grid, next_block;
extern "C" hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    next_grid = grid, next_block = block;
    return hipSuccess;
}
extern "C" hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream) {
    *grid = next_grid, *block = next_block, *lds = 0, *stream = nullptr;
    return hipSuccess;
}
extern "C" hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **, size_t, hipStream_t) {
    const int64_t blocks = (int64_t)grid.x * grid.y * grid.z;
    seen.push_back({blocks, blocks * block.x * block.y * block.z});
    return hipSuccess;
}
extern "C" hipError_t hipGetLastError() { return hipSuccess; }

static int failures = 0, calls = 0;

static void check(const char *what, const AttnArgs &a, hipError_t e, int64_t want) {
    int64_t blocks = 0;
    ++calls;
    bool bad = e != hipSuccess;
    for (const Launch &l : seen) {
        blocks += l.blocks;
        bad = bad || l.blocks < 1 || l.threads >= (int64_t)1 << 32;
    }
    if (bad || blocks != want) {
        printf("%s, %d batches, %d x %d positions, %d over %d heads: %lld workgroups in %zu launches, %lld needed\n", what, a.B, a.Lq,
               a.Lk, a.Hq, a.Hkv, (long long)blocks, seen.size(), (long long)want);
        ++failures;
    }
}

int main() {
    static char some[16];
    const int64_t top = ((int64_t)1 << 24) - 1;
    const int64_t cases[][5] = {  // B, Lq, Lk, Hkv, G
        {top, 1, 1, 1, 1},       {1, 1, 1, top, 1},          {top, 31, 1, 1, 1},       {top, 1, 127, 1, 31},
        {((int64_t)1 << 23) + 1, 1, 1, 1, 1}, {(((int64_t)1 << 31) - 1) / 129, 1, 129, 1, 1}, {top, 0, 127, 1, 1}, {top, 1, 0, 1, 1},
        {(((int64_t)1 << 29) - 1) / 33, 33, 1, 1, 1}, {((int64_t)1 << 22) - 1, 1, 1, 4, 32}, {1, ((int64_t)1 << 29) - 1, 1, 1, 1},
        {1, 1, (int64_t)1 << 29, 1, 1}, {3, ((int64_t)1 << 27) + 5, (int64_t)1 << 29, 1, 1}, {1, 1, 1, 1, 1}, {16, 128, 128, 8, 1},
    };
    for (const auto &c : cases) {
        AttnArgs a;
        memset((void *)&a, 0, sizeof(a));
        a.B = (int)c[0], a.Lq = (int)c[1], a.Lk = (int)c[2], a.Hkv = (int)c[3], a.G = (int)c[4], a.Hq = a.Hkv * a.G;
        a.D = 8, a.rows = c[1] * c[4], a.by_G = make_fastdiv((uint32_t)a.G), a.scale = 1.0f, a.dtype = kBF16;
        a.gq = a.gk = a.gv = some;
        const int64_t heads = c[0] * c[3], key_tiles = (c[2] + 127) / 128, row_tiles = (a.rows + 127) / 128;
        const AttnBwdPlan b = plan_attention_backward(a, 256);
        int64_t want = (heads * a.rows + 31) / 32 + heads * key_tiles * b.splits + heads * row_tiles;
        if (b.splits > 1) want += (2 * heads * c[2] * 8 + 255) / 256;
        seen.clear();
        check("gradients", a, launch_attention_backward(a, b, some, nullptr), want);
        if (a.rows == 0) continue;
        const AttnPlan f = plan_attention(a, 256);
        seen.clear();
        check("attention", a, launch_attention(a, f, some, nullptr), f.blocks + (f.splits > 1 ? heads * a.rows : 0));
    }
    // layer norm's gradients: the workspace holds the sums of the workgroups that there are
    for (int dtype : {(int)kF32, (int)kBF16})
        for (int C : {1, 7, 40, 101, 512, 1024, 2000, 4099, 8192, 8200, 16384, 32768, 1 << 20})
            for (int64_t L : {1, 2, 5, 9, 128, 4092, 1 << 22})
                for (int64_t B : {1, 3, 300, 4096, 131072}) {
                    if (B * L * C > (int64_t)1 << 40) continue;
                    LayerNormArgs a;
                    memset((void *)&a, 0, sizeof(a));
                    a.x = a.g = a.y = some, a.gw = a.gb = some, a.mean = a.rstd = a.ws = (float *)some;
                    a.dtype = dtype, a.B = B, a.L = L, a.C = C;
                    seen.clear();
                    ++calls;
                    const size_t bytes = layer_norm_backward_workspace(B, C, L, dtype, true, 256);
                    if (launch_layer_norm_backward(a, 256, nullptr) != hipSuccess || seen.size() != 2 ||
                        bytes != (size_t)seen[0].blocks * 2 * C * sizeof(float)) {
                        printf("layer norm gradients, %lld x %d x %lld: %zu bytes for %lld workgroups\n", (long long)B, C, (long long)L,
                               bytes, seen.empty() ? -1 : (long long)seen[0].blocks);
                        ++failures;
                    }
                }
    printf("launch checks: %d calls, %d failure(s)\n", calls, failures);
    return failures != 0;
}
