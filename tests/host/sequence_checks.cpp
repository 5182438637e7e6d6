// Host-side checks of the sequence operators' C ABI, built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the library's host code
// and on this driver (tests/test_sequence_sanitizers.py builds and runs it; no
// GPU is used).  Every shape, stride and argument below is malformed or at the
// integers' limits and must be rejected before any device work; the sanitizers
// watch the validation for overflowing arithmetic and out-of-bounds accesses.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "dc1d.h"

static int failures = 0, calls = 0;

// Rejected, or (no device here) accepted up to the device query.
static void rejected(int got, const char *what, bool may_reach_device = false) {
    ++calls;
    if (got == DC1D_OK || got == DC1D_ERR_LAUNCH || (got == DC1D_ERR_DEVICE && !may_reach_device)) {
        fprintf(stderr, "%s returned %d\n", what, got);
        ++failures;
    }
}

static dc1d_tensor T(uintptr_t slot, int dtype, int ndim, int64_t s0, int64_t s1 = 1, int64_t s2 = 1, int64_t s3 = 1) {
    return {(void *)(0x10000000 + (slot << 24)), dtype, ndim, {s0, s1, s2, s3}};
}
static dc1d_strided S(uintptr_t slot, int dtype, int64_t s0, int64_t s1, int64_t s2, int64_t s3, int64_t t0, int64_t t1, int64_t t2,
                      int64_t t3) {
    return {(void *)(0x10000000 + (slot << 24)), dtype, 4, {s0, s1, s2, s3}, {t0, t1, t2, t3}};
}

int main() {
    const int64_t ends[] = {INT64_MIN, INT64_MIN / 2, -1, 0, 1, 2, 127, 129, (int64_t)1 << 24, (int64_t)1 << 29, (int64_t)1 << 31,
                            (int64_t)1 << 48, (int64_t)1 << 62, INT64_MAX};
    const int64_t section[4] = {16, 16, INT64_MAX, INT64_MAX};
    size_t bytes = 0;
    // layer norm: every end in every place, every rank
    for (int ndim = -1; ndim <= 6; ++ndim)
        for (int64_t a : ends)
            for (int64_t b : ends)
                for (int64_t c : ends) {
                    const dc1d_tensor x = T(0, DC1D_F32, ndim, a, b, c, 2), y = T(1, DC1D_F32, ndim, a, b, c, 2);
                    rejected(dc1d_layer_norm(&x, nullptr, nullptr, &y, nullptr, nullptr, 1e-5, nullptr), "layer_norm", true);
                    rejected(dc1d_layer_norm_backward_workspace_bytes(&x, 1, &bytes), "layer_norm_backward_workspace_bytes", true);
                    const dc1d_tensor m = T(2, DC1D_F32, ndim - 1, a, c, 2), r = T(3, DC1D_F32, ndim - 1, a, c, 2);
                    rejected(dc1d_layer_norm_backward(&x, nullptr, &y, &m, &r, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
                             "layer_norm_backward", true);
                }
    // attention and rotary: every end as a size and as a stride of each dimension
    const int64_t good[4] = {2, 5, 4, 64}, step[4] = {1280, 256, 64, 1};
    for (int d = 0; d < 4; ++d)
        for (int64_t size : ends)
            for (int64_t stride : ends) {
                int64_t s[4], t[4];
                for (int i = 0; i < 4; ++i) s[i] = i == d ? size : good[i], t[i] = i == d ? stride : step[i];
                const dc1d_strided odd = S(0, DC1D_F32, s[0], s[1], s[2], s[3], t[0], t[1], t[2], t[3]);
                const dc1d_strided odd2 = S(1, DC1D_F32, s[0], s[1], s[2], s[3], t[0], t[1], t[2], t[3]);
                const dc1d_strided odd3 = S(2, DC1D_F32, s[0], s[1], s[2], s[3], t[0], t[1], t[2], t[3]);
                const dc1d_strided out = S(9, DC1D_F32, s[0], s[1], s[2], s[3], t[0], t[1], t[2], t[3]);
                const dc1d_tensor lse = T(5, DC1D_F32, 3, s[0], s[2], s[1]);
                rejected(dc1d_attention(&odd, &odd2, &odd3, nullptr, nullptr, &out, &lse, 1, INT64_MAX, 0.1, nullptr, 0, nullptr),
                         "attention", true);
                rejected(dc1d_attention_workspace_bytes(&odd, &odd2, &odd3, &bytes), "attention_workspace_bytes", true);
                rejected(dc1d_attention_plan(&odd, &odd2, &odd3, nullptr, nullptr, nullptr), "attention_plan", true);
                rejected(dc1d_attention_backward(&odd, &odd2, &odd3, nullptr, nullptr, &out, &lse, &out, &odd, nullptr, nullptr, 0, 0,
                                                 0.1, nullptr, 0, nullptr),
                         "attention_backward onto its input", s[0] <= 0 || s[1] <= 0);
                const dc1d_tensor table = T(6, DC1D_F32, 2, 64, 32), table2 = T(7, DC1D_F32, 2, 64, 32);
                const dc1d_tensor pos = T(8, DC1D_I32, 3, s[0], s[1], 2);
                for (int32_t axes : {INT32_MIN, -1, 0, 1, 2, 4, 5, INT32_MAX})
                    rejected(dc1d_rotary(&odd, nullptr, &table, &table2, &pos, &out, nullptr, section, axes, 0, 0, nullptr), "rotary", true);
            }
    const dc1d_strided q = S(0, DC1D_F32, 2, 5, 4, 64, 1280, 256, 64, 1), o = S(9, DC1D_F32, 2, 5, 4, 64, 1280, 256, 64, 1);
    for (int64_t window : {INT64_MIN, (int64_t)-1})
        rejected(dc1d_attention(&q, &q, &q, nullptr, nullptr, &o, nullptr, 0, window, 0.1, nullptr, 0, nullptr), "window");
    printf("sequence checks: %d calls, %d failure(s)\n", calls, failures);
    return failures != 0;
}
