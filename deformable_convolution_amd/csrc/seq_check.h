// seq_check.h -- what the entries of the sequence operators share: argument
// checks on descriptors, ranges of memory that must not meet, the device.
#pragma once

#include <mutex>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dc1d.h"
#include "seq_internal.h"

namespace dc1d {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxElems = (int64_t)1 << 48, kLim31 = (int64_t)1 << 31, kLen = (int64_t)1 << 29;

inline bool log_on() {
    static const bool on = [] {
        const char *v = getenv("DC1D_LOG");
        return v && v[0] && strcmp(v, "0") != 0;
    }();
    return on;
}

// The compute units of the current device, probed once per device.
inline int current_device(int *num_cus) {
    static std::once_flag once[kMaxDevices];
    static int cus[kMaxDevices];  // 0: not a gfx950
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return DC1D_ERR_DEVICE;
    }
    std::call_once(once[dev], [dev]() {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) == hipSuccess) {
            if (strncmp(prop.gcnArchName, "gfx950", 6) == 0) cus[dev] = prop.multiProcessorCount;
        } else {
            (void)hipGetLastError();
        }
    });
    *num_cus = cus[dev];
    return cus[dev] > 0 ? DC1D_OK : DC1D_ERR_DEVICE;
}

inline bool data_dtype(int32_t dt) { return dt == DC1D_F32 || dt == DC1D_BF16; }
inline size_t elem_size(int32_t dt) { return dt == DC1D_BF16 ? 2 : 4; }

// Element count, -1 where the rank or a size is out of range; no product
// overflows.
inline int64_t count(const dc1d_tensor *t) {
    if (t->ndim < 0 || t->ndim > 4) return -1;
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) {
        const int64_t s = t->shape[i];
        if (s < 0 || (s > 0 && n > kMaxElems / s)) return -1;
        n *= s;
    }
    return n;
}

inline bool shape_is(const dc1d_tensor *t, int ndim, const int64_t *s) {
    if (t->ndim != ndim) return false;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] != s[i]) return false;
    return true;
}

// A strided tensor of rank 4: its element count, or -1; span: elements from
// its first to past its last.
inline int64_t count(const dc1d_strided *t, int64_t *span) {
    if (t->ndim != 4) return -1;
    int64_t n = 1, reach = 1;
    for (int i = 0; i < 4; ++i) {
        const int64_t s = t->shape[i], st = t->stride[i];
        if (s < 0 || st < 0 || (s > 0 && n > kMaxElems / s)) return -1;
        n *= s;
        if (s > 1) {
            if (st > kMaxElems / (s - 1)) return -1;
            reach += st * (s - 1);
            if (reach > kMaxElems) return -1;
        }
    }
    if (t->shape[3] > 1 && t->stride[3] != 1) return -1;
    *span = n > 0 ? reach : 0;
    return n;
}

// Whether no two elements share memory: taken by growing stride, each
// dimension steps past what the smaller ones cover.
inline bool distinct(const dc1d_strided *t) {
    bool used[4] = {};
    int64_t cover = 1;
    for (int k = 0; k < 4; ++k) {
        int at = -1;
        for (int i = 0; i < 4; ++i)
            if (!used[i] && (at < 0 || t->shape[i] <= 1 || (t->shape[at] > 1 && t->stride[i] < t->stride[at]))) at = i;
        used[at] = true;
        if (t->shape[at] <= 1) continue;
        if (t->stride[at] < cover) return false;
        cover = t->stride[at] * (t->shape[at] - 1) + cover;
    }
    return true;
}

struct Range {
    uintptr_t lo, hi;
};
inline bool meet(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline Range range(const dc1d_tensor *t) {
    if (!t || !t->data) return {0, 0};
    return {(uintptr_t)t->data, (uintptr_t)t->data + (size_t)count(t) * elem_size(t->dtype)};
}
inline Range range(const dc1d_strided *t) {
    int64_t span = 0;
    if (!t || !t->data || count(t, &span) <= 0) return {0, 0};
    return {(uintptr_t)t->data, (uintptr_t)t->data + (size_t)span * elem_size(t->dtype)};
}

// Whether two tensors that interleave are disjoint head slices of one buffer:
// the same positions at the same strides, and the later one's heads starting
// past the earlier one's and ending before the next position.
inline bool head_slices(const dc1d_strided *a, const dc1d_strided *b) {
    for (int i = 0; i < 2; ++i)
        if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
    if ((uintptr_t)a->data > (uintptr_t)b->data) {
        const dc1d_strided *t = a;
        a = b;
        b = t;
    }
    const int64_t es = (int64_t)elem_size(a->dtype), gap = (int64_t)((uintptr_t)b->data - (uintptr_t)a->data);
    auto inner = [](const dc1d_strided *t) { return (t->shape[2] - 1) * (t->shape[2] > 1 ? t->stride[2] : 0) + t->shape[3]; };
    if (gap < inner(a) * es) return false;
    // the two outer dimensions, sizes of 1 left out, by growing stride
    int64_t unit = kMaxElems, s[2], n[2];
    int d = 0;
    for (int i = 0; i < 2; ++i)
        if (a->shape[i] > 1) s[d] = a->stride[i], n[d++] = a->shape[i];
    if (d == 2 && s[0] > s[1]) {
        const int64_t ts = s[0], tn = n[0];
        s[0] = s[1], n[0] = n[1], s[1] = ts, n[1] = tn;
    }
    if (d == 2 && s[1] < s[0] * n[0]) return false;
    if (d > 0) unit = s[0];
    return gap + inner(b) * es <= unit * es;
}

// Whether s[0] d[0] + ... = r has a solution with lo[i] <= d[i] <= hi[i], the
// strides s falling and positive; true also where too many are left to try.
inline bool reachable(const int64_t *s, const int64_t *lo, const int64_t *hi, int n, int64_t r) {
    if (n == 0) return r == 0;
    int64_t least = 0, most = 0;  // what the dimensions after this one can add up to
    for (int i = 1; i < n; ++i) least += s[i] * lo[i], most += s[i] * hi[i];
    auto down = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    int64_t from = -down(most - r, s[0]), to = down(r - least, s[0]);
    from = from > lo[0] ? from : lo[0];
    to = to < hi[0] ? to : hi[0];
    if (to - from >= 8) return true;
    for (int64_t d = from; d <= to; ++d)
        if (reachable(s + 1, lo + 1, hi + 1, n - 1, r - s[0] * d)) return true;
    return false;
}

// Whether two tensors of one dtype at the same strides (slices of one buffer
// along any dimension) share no element: no two indices' difference times the
// strides makes up the distance between their first elements.
inline bool apart(const dc1d_strided *a, const dc1d_strided *b) {
    const int64_t es = (int64_t)elem_size(a->dtype), gap = (int64_t)((uintptr_t)b->data - (uintptr_t)a->data);
    if (gap % es) return false;
    int64_t s[4], lo[4], hi[4];
    int n = 0;
    for (int i = 0; i < 4; ++i) {
        const int64_t na = a->shape[i], nb = b->shape[i];
        const int64_t st = i == 3 ? 1 : na > 1 ? a->stride[i] : b->stride[i];
        if (i < 3 && na > 1 && nb > 1 && b->stride[i] != st) return false;
        if ((na <= 1 && nb <= 1) || st == 0) continue;
        int at = n++;
        for (; at > 0 && s[at - 1] < st; --at) s[at] = s[at - 1], lo[at] = lo[at - 1], hi[at] = hi[at - 1];
        s[at] = st, lo[at] = -(nb - 1), hi[at] = na - 1;
    }
    return !reachable(s, lo, hi, n, gap / es);
}

// An output against another tensor.
inline bool clash(const dc1d_strided *out, const dc1d_strided *t) {
    return out && t && meet(range(out), range(t)) && !head_slices(out, t) && !apart(out, t);
}
inline bool clash(const dc1d_strided *out, const dc1d_tensor *t) { return out && t && meet(range(out), range(t)); }
inline bool clash(Range w, const dc1d_strided *t) { return t && meet(w, range(t)); }
inline bool clash(Range w, const dc1d_tensor *t) { return t && meet(w, range(t)); }

inline bool same_view(const dc1d_strided *a, const dc1d_strided *b) {
    if (a->data != b->data) return false;
    for (int i = 0; i < 4; ++i)
        if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
    return true;
}

inline Strides3 strides(const dc1d_strided *t) { return {t->stride[0], t->stride[1], t->stride[2]}; }

inline int launched(hipError_t e) { return e == hipSuccess ? DC1D_OK : DC1D_ERR_LAUNCH; }

inline int workspace_ok(void *ws, size_t have, size_t need) {
    if (need == 0) return DC1D_OK;
    return ws && have >= need && !((uintptr_t)ws & 255) ? DC1D_OK : DC1D_ERR_WORKSPACE;
}

inline bool has_data(const dc1d_strided *t) {
    int64_t span;
    return !t || count(t, &span) == 0 || t->data;
}
inline bool has_data(const dc1d_tensor *t) { return !t || count(t) == 0 || t->data; }

// A dimension of size 1 is never stepped along; its stride is made 0 so that
// no arithmetic on it matters.
inline Strides3 steps(const dc1d_strided *t) {
    Strides3 s = strides(t);
    if (t->shape[0] <= 1) s.b = 0;
    if (t->shape[1] <= 1) s.l = 0;
    if (t->shape[2] <= 1) s.h = 0;
    return s;
}

}  // namespace dc1d
