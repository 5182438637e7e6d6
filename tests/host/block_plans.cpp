// Which form group norm takes for sizes at which both were timed, on 256 CUs
// (tests/test_block_plans.py builds and runs this; no GPU is used): held by
// workgroups, or in parts.
#include <stdio.h>

#include "groupnorm.h"

using namespace dc1d;

int main() {
    struct Case {
        int tensors;  // 1: forward, 2: gradients
        int64_t B, S;
        int C, G, esize;
        bool held;  // the faster one
    };
    const Case cases[] = {
        // one odd group a slab, rows of short runs
        {1, 3, 7215, 192, 16, 2, false}, {1, 1, 4096, 320, 32, 2, false}, {1, 8, 4096, 320, 32, 2, false}, {1, 64, 4096, 320, 32, 2, false},
        {1, 18, 7232, 170, 17, 2, false}, {1, 4, 4092, 255, 17, 2, false}, {1, 52, 4092, 255, 17, 2, false}, {1, 13, 2501, 76, 4, 2, false},
        {1, 23, 3016, 304, 16, 2, false}, {1, 7, 4741, 80, 8, 4, false}, {1, 1, 7922, 112, 16, 4, false}, {1, 44, 5331, 56, 8, 4, false},
        {1, 12, 2392, 48, 8, 4, true}, {1, 40, 2392, 48, 8, 4, true}, {1, 32, 2392, 88, 8, 4, true}, {1, 24, 4000, 88, 8, 4, true},
        {2, 142, 749, 160, 16, 4, false}, {2, 128, 885, 90, 9, 4, false}, {2, 472, 1212, 18, 3, 4, false}, {2, 25, 1312, 160, 32, 4, false},
        {2, 131, 918, 55, 5, 4, true}, {2, 335, 713, 14, 1, 4, true}, {2, 66, 131, 505, 5, 4, true}, {2, 231, 61, 1935, 9, 4, true},
        // most CUs without a workgroup, or a few with a second one
        {1, 14, 1641, 67, 1, 2, false}, {1, 1, 2001, 156, 4, 2, false}, {1, 7, 1010, 316, 4, 2, false}, {1, 43, 194, 516, 1, 2, false},
        {1, 70, 194, 516, 1, 2, false}, {1, 16, 4092, 510, 17, 2, false}, {1, 17, 3010, 459, 17, 2, false}, {1, 72, 643, 540, 4, 2, false},
        {1, 150, 194, 516, 1, 2, true}, {1, 250, 194, 516, 1, 2, true}, {1, 36, 554, 1197, 9, 2, true}, {1, 30, 4092, 510, 17, 2, true},
        {1, 512, 194, 516, 1, 2, true}, {1, 2, 2048, 960, 32, 2, true}, {1, 60, 80, 716, 1, 2, true}, {1, 13, 2818, 432, 16, 2, true},
        // few workgroups of fp32, and single positions
        {1, 13, 4092, 255, 17, 4, true}, {1, 46, 498, 89, 1, 4, true}, {1, 3, 619, 292, 4, 4, true}, {1, 46, 9, 1081, 1, 4, true},
        {1, 18, 646, 1054, 17, 4, true}, {1, 11031, 1, 890, 1, 2, true}, {2, 11031, 1, 890, 1, 2, true},
    };
    int failures = 0;
    for (const Case &c : cases) {
        const bool held = plan_held(c.B, c.S, c.C, c.G, piece_size(c.C, c.esize == 4 ? kF32 : kBF16), c.esize, c.tensors, 256).R != 0;
        if (held == c.held) continue;
        ++failures;
        printf("%s, %lld x %lld x %d in %d groups, %d bytes: %s\n", c.tensors == 1 ? "forward" : "gradients", (long long)c.B, (long long)c.S, c.C,
               c.G, c.esize, held ? "held" : "in parts");
    }
    printf("block plans: %d failure(s)\n", failures);
    return failures != 0;
}
