// Host-side checks of the C ABI of group norm and the gated recurrence, built
// with AddressSanitizer and UndefinedBehaviorSanitizer on the library's host
// code and on this driver (tests/test_block_sanitizers.py builds and runs it; no
// GPU is used).  Every shape, stride and argument below is malformed or at the
// integers' limits, or the call ends at the query of a device that is not there;
// the sanitizers watch the validation for overflowing arithmetic and
// out-of-bounds accesses.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "dc1d.h"

static int failures = 0, calls = 0;

static void rejected(int got, const char *what) {
    ++calls;
    if (got == DC1D_OK || got == DC1D_ERR_LAUNCH) {
        fprintf(stderr, "%s returned %d\n", what, got);
        ++failures;
    }
}

static dc1d_tensor T(uintptr_t slot, int dtype, int ndim, int64_t s0, int64_t s1 = 1, int64_t s2 = 1, int64_t s3 = 1) {
    return {(void *)(0x10000000 + (slot << 24)), dtype, ndim, {s0, s1, s2, s3}};
}
static dc1d_strided S(uintptr_t slot, int dtype, int ndim, const int64_t *s, const int64_t *t) {
    return {(void *)(0x10000000 + (slot << 24)), dtype, ndim, {s[0], s[1], s[2], 1}, {t[0], t[1], t[2], 1}};
}

int main() {
    const int64_t ends[] = {INT64_MIN, INT64_MIN / 2, -1, 0, 1, 2, 127, 129, (int64_t)1 << 24, (int64_t)1 << 29, (int64_t)1 << 31,
                            (int64_t)1 << 48, (int64_t)1 << 62, INT64_MAX};
    size_t bytes = 0;
    for (int ndim = -1; ndim <= 6; ++ndim)
        for (int64_t a : ends)
            for (int64_t b : ends)
                for (int64_t c : ends)
                    for (int64_t groups : {INT64_MIN, (int64_t)0, (int64_t)1, (int64_t)2, INT64_MAX}) {
                        const dc1d_tensor x = T(0, DC1D_F32, ndim, a, b, c, 2), y = T(1, DC1D_F32, ndim, a, b, c, 2);
                        const dc1d_tensor m = T(2, DC1D_F32, 2, a, groups), r = T(3, DC1D_F32, 2, a, groups);
                        rejected(dc1d_group_norm(&x, nullptr, nullptr, nullptr, &y, &m, &r, groups, 1e-5, DC1D_ACT_SILU, nullptr, 0, nullptr),
                                 "group_norm");
                        rejected(dc1d_group_norm_workspace_bytes(&x, groups, &bytes), "group_norm_workspace_bytes");
                        rejected(dc1d_group_norm_backward(&x, nullptr, nullptr, nullptr, &y, &m, &r, &y, nullptr, nullptr, groups,
                                                          DC1D_ACT_NONE, nullptr, 0, nullptr),
                                 "group_norm_backward");
                        rejected(dc1d_group_norm_backward_workspace_bytes(&x, groups, 1, &bytes), "group_norm_backward_workspace_bytes");
                    }
    // the recurrence: every end as a size and as a stride of each dimension, every rank
    const int64_t good[3] = {2, 5, 64}, step[3] = {1280, 256, 1};
    for (int ndim = -1; ndim <= 6; ++ndim)
        for (int d = 0; d < 3; ++d)
            for (int64_t size : ends)
                for (int64_t stride : ends)
                    for (int64_t other : {(int64_t)1, (int64_t)256, (int64_t)1 << 40, INT64_MAX, INT64_MIN}) {
                        int64_t s[3], t[3];
                        for (int i = 0; i < 3; ++i) s[i] = i == d ? size : good[i], t[i] = i == d ? stride : i == (d + 1) % 3 ? other : step[i];
                        const dc1d_strided x = S(0, DC1D_F32, ndim, s, t), gate = S(4, DC1D_F32, ndim, s, t), y = S(9, DC1D_F32, ndim, s, t);
                        const int64_t kept = s[1] > 0 ? (s[1] - 1) / 64 + 1 : 0;
                        const dc1d_tensor state = T(5, DC1D_F32, 2, s[0], s[2]), states = T(6, DC1D_F32, 3, s[0], kept, s[2]);
                        const dc1d_tensor lens = T(7, DC1D_I32, 1, s[0]);
                        for (int flags = 0; flags < 4; ++flags) {
                            rejected(dc1d_gated_recurrence(&x, &gate, &state, &lens, &y, &state, &states, flags & 1, flags >> 1, nullptr, 0, nullptr),
                                     "gated_recurrence");
                            rejected(dc1d_gated_recurrence_backward(&x, &gate, &states, &lens, &y, &state, &y, nullptr, &state, flags & 1,
                                                                    flags >> 1, nullptr, 0, nullptr),
                                     "gated_recurrence_backward");
                        }
                        rejected(dc1d_gated_recurrence_workspace_bytes(&x, &bytes), "gated_recurrence_workspace_bytes");
                        rejected(dc1d_gated_recurrence_backward_workspace_bytes(&x, &bytes), "gated_recurrence_backward_workspace_bytes");
                    }
    // nothing given
    const dc1d_tensor x = T(0, DC1D_F32, 2, 4, 8), y = T(1, DC1D_F32, 2, 4, 8);
    for (double eps : {-1.0, 1e300, __builtin_nan("")})
        rejected(dc1d_group_norm(&x, nullptr, nullptr, nullptr, &y, nullptr, nullptr, 2, eps, DC1D_ACT_NONE, nullptr, 0, nullptr), "eps");
    for (int act : {INT32_MIN, -1, 3, INT32_MAX})
        rejected(dc1d_group_norm(&x, nullptr, nullptr, nullptr, &y, nullptr, nullptr, 2, 1e-5, act, nullptr, 0, nullptr), "activation");
    rejected(dc1d_group_norm(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 1, 1e-5, 0, nullptr, 0, nullptr), "group_norm of nothing");
    rejected(dc1d_group_norm_backward(&x, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 1, 0, nullptr, 0, nullptr),
             "group_norm_backward of nothing");
    rejected(dc1d_gated_recurrence(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, nullptr, 0, nullptr), "gated_recurrence of nothing");
    rejected(dc1d_gated_recurrence_backward(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, nullptr, 0, nullptr),
             "gated_recurrence_backward of nothing");
    rejected(dc1d_group_norm_workspace_bytes(&x, 2, nullptr), "no place for the bytes");
    rejected(dc1d_gated_recurrence_workspace_bytes(nullptr, &bytes), "workspace of nothing");
    printf("block checks: %d calls, %d failure(s)\n", calls, failures);
    return failures != 0;
}
