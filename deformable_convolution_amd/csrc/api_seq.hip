// api_seq.hip -- the C ABI of the sequence operators (include/dc1d.h):
// argument validation, kernel choice, and launch.  No allocation, no
// synchronisation, no exceptions across the boundary.
#include <math.h>
#include <mutex>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dc1d.h"
#include "seq_internal.h"

using namespace dc1d;

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxElems = (int64_t)1 << 48, kLim31 = (int64_t)1 << 31, kLen = (int64_t)1 << 29;

bool log_on() {
    static const bool on = [] {
        const char *v = getenv("DC1D_LOG");
        return v && v[0] && strcmp(v, "0") != 0;
    }();
    return on;
}

// The compute units of the current device, probed once per device.
int current_device(int *num_cus) {
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

bool data_dtype(int32_t dt) { return dt == DC1D_F32 || dt == DC1D_BF16; }
size_t elem_size(int32_t dt) { return dt == DC1D_BF16 ? 2 : 4; }

// Element count, -1 where the rank or a size is out of range; no product
// overflows.
int64_t count(const dc1d_tensor *t) {
    if (t->ndim < 0 || t->ndim > 4) return -1;
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) {
        const int64_t s = t->shape[i];
        if (s < 0 || (s > 0 && n > kMaxElems / s)) return -1;
        n *= s;
    }
    return n;
}

bool shape_is(const dc1d_tensor *t, int ndim, const int64_t *s) {
    if (t->ndim != ndim) return false;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] != s[i]) return false;
    return true;
}

// A strided tensor of rank 4: its element count, or -1; span: elements from
// its first to past its last.
int64_t count(const dc1d_strided *t, int64_t *span) {
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
bool distinct(const dc1d_strided *t) {
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
bool meet(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

Range range(const dc1d_tensor *t) {
    if (!t || !t->data) return {0, 0};
    return {(uintptr_t)t->data, (uintptr_t)t->data + (size_t)count(t) * elem_size(t->dtype)};
}
Range range(const dc1d_strided *t) {
    int64_t span = 0;
    if (!t || !t->data || count(t, &span) <= 0) return {0, 0};
    return {(uintptr_t)t->data, (uintptr_t)t->data + (size_t)span * elem_size(t->dtype)};
}

// Whether two tensors that interleave are disjoint head slices of one buffer:
// the same positions at the same strides, and the later one's heads starting
// past the earlier one's and ending before the next position.
bool head_slices(const dc1d_strided *a, const dc1d_strided *b) {
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
bool reachable(const int64_t *s, const int64_t *lo, const int64_t *hi, int n, int64_t r) {
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
bool apart(const dc1d_strided *a, const dc1d_strided *b) {
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
bool clash(const dc1d_strided *out, const dc1d_strided *t) {
    return out && t && meet(range(out), range(t)) && !head_slices(out, t) && !apart(out, t);
}
bool clash(const dc1d_strided *out, const dc1d_tensor *t) { return out && t && meet(range(out), range(t)); }
bool clash(Range w, const dc1d_strided *t) { return t && meet(w, range(t)); }
bool clash(Range w, const dc1d_tensor *t) { return t && meet(w, range(t)); }

bool same_view(const dc1d_strided *a, const dc1d_strided *b) {
    if (a->data != b->data) return false;
    for (int i = 0; i < 4; ++i)
        if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
    return true;
}

Strides3 strides(const dc1d_strided *t) { return {t->stride[0], t->stride[1], t->stride[2]}; }

int launched(hipError_t e) { return e == hipSuccess ? DC1D_OK : DC1D_ERR_LAUNCH; }

int workspace_ok(void *ws, size_t have, size_t need) {
    if (need == 0) return DC1D_OK;
    return ws && have >= need && !((uintptr_t)ws & 255) ? DC1D_OK : DC1D_ERR_WORKSPACE;
}

// ---- layer norm ----------------------------------------------------------------

// Shape and dtype of x; positions (elements per channel over the batch).
int ln_shape(const dc1d_tensor *x, int64_t *B, int64_t *C, int64_t *L) {
    if (!x) return DC1D_ERR_NULL_PTR;
    if (!data_dtype(x->dtype)) return DC1D_ERR_BAD_DTYPE;
    if (x->ndim < 2 || x->ndim > 4 || count(x) < 0) return DC1D_ERR_BAD_SHAPE;
    *B = x->shape[0];
    *C = x->shape[1];
    *L = 1;
    if (*C < 1 || *C > (1 << 24) || *B >= kLim31) return DC1D_ERR_BAD_SHAPE;
    for (int i = 2; i < x->ndim; ++i) {
        if (x->shape[i] >= kLim31 || *L * x->shape[i] >= kLim31) return DC1D_ERR_BAD_SHAPE;
        *L *= x->shape[i];
    }
    if (*B * *L >= kLim31) return DC1D_ERR_BAD_SHAPE;
    return DC1D_OK;
}

int ln_like(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != x->dtype) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, x->ndim, x->shape) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int ln_stat(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != DC1D_F32) return DC1D_ERR_BAD_DTYPE;
    const int64_t s[3] = {x->shape[0], x->shape[2], x->shape[3]};
    return shape_is(t, x->ndim - 1, s) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int ln_param(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != x->dtype) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 1, x->shape + 1) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}

// ---- attention -------------------------------------------------------------------

int attn_shape(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v, AttnArgs *a) {
    if (!q || !k || !v) return DC1D_ERR_NULL_PTR;
    if (!data_dtype(q->dtype) || k->dtype != q->dtype || v->dtype != q->dtype) return DC1D_ERR_BAD_DTYPE;
    int64_t span;
    if (count(q, &span) < 0 || count(k, &span) < 0 || count(v, &span) < 0) return DC1D_ERR_BAD_SHAPE;
    const int64_t B = q->shape[0], Lq = q->shape[1], Hq = q->shape[2], D = q->shape[3];
    const int64_t Lk = k->shape[1], Hkv = k->shape[2];
    if (k->shape[0] != B || k->shape[3] != D) return DC1D_ERR_BAD_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (v->shape[i] != k->shape[i]) return DC1D_ERR_BAD_SHAPE;
    if (D < 1 || D > 128 || Hq < 1 || Hkv < 1 || Hq % Hkv) return DC1D_ERR_BAD_SHAPE;
    if (B >= kLim31 || Hq >= kLim31 || Lq > kLen || Lk > kLen) return DC1D_ERR_BAD_SHAPE;
    const int64_t G = Hq / Hkv;
    if (Lq * G >= kLim31) return DC1D_ERR_BAD_SHAPE;
    // keeps every kind of workgroup's number far inside 32 bits; the forward's
    // are fewer than 2^24 of 256 threads, which one launch holds
    const int64_t heads = B > 0 && Hkv > kMaxElems / B ? kMaxElems : B * Hkv;
    if (heads >= (1 << 24) || heads * (Lq * G) >= kLen || heads * Lk >= kLim31) return DC1D_ERR_BAD_SHAPE;
    memset(a, 0, sizeof(*a));
    a->q = q->data, a->k = k->data, a->v = v->data;
    a->qs = strides(q), a->ks = strides(k), a->vs = strides(v);
    a->dtype = q->dtype;
    a->B = (int)B, a->Lq = (int)Lq, a->Lk = (int)Lk, a->Hq = (int)Hq, a->Hkv = (int)Hkv, a->G = (int)G, a->D = (int)D;
    a->rows = Lq * G;
    a->by_G = make_fastdiv((uint32_t)G);
    return DC1D_OK;
}

int like_q(const dc1d_strided *t, const dc1d_strided *q) {
    if (t->dtype != q->dtype) return DC1D_ERR_BAD_DTYPE;
    int64_t span;
    if (count(t, &span) < 0) return DC1D_ERR_BAD_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (t->shape[i] != q->shape[i]) return DC1D_ERR_BAD_SHAPE;
    return DC1D_OK;
}

int attn_rest(const dc1d_strided *q, const dc1d_tensor *lens, const dc1d_tensor *start, const dc1d_tensor *lse, int causal,
              int64_t window, double scale, AttnArgs *a) {
    if (window < 0 || !(scale > 0.0) || !(scale <= 3.0e38)) return DC1D_ERR_BAD_ARG;
    const int64_t sb[1] = {q->shape[0]}, sl[3] = {q->shape[0], q->shape[2], q->shape[1]};
    for (const dc1d_tensor *t : {lens, start}) {
        if (!t) continue;
        if (t->dtype != DC1D_I32) return DC1D_ERR_BAD_DTYPE;
        if (!shape_is(t, 1, sb)) return DC1D_ERR_BAD_SHAPE;
        if (sb[0] > 0 && !t->data) return DC1D_ERR_NULL_PTR;
    }
    if (lse) {
        if (lse->dtype != DC1D_F32) return DC1D_ERR_BAD_DTYPE;
        if (!shape_is(lse, 3, sl)) return DC1D_ERR_BAD_SHAPE;
        if (count(lse) > 0 && !lse->data) return DC1D_ERR_NULL_PTR;
    }
    a->kv_lens = lens ? (const int *)lens->data : nullptr;
    a->q_start = start ? (const int *)start->data : nullptr;
    a->lse = lse ? (float *)lse->data : nullptr;
    a->causal = causal != 0;
    a->window = (int)(window > kLen ? kLen : window);
    a->scale = (float)scale;
    return a->scale > 0.0f ? DC1D_OK : DC1D_ERR_BAD_ARG;
}

bool has_data(const dc1d_strided *t) {
    int64_t span;
    return !t || count(t, &span) == 0 || t->data;
}
bool has_data(const dc1d_tensor *t) { return !t || count(t) == 0 || t->data; }

// Whether the 16-byte pieces of every row are aligned.
bool pieces(const AttnArgs &a, const dc1d_strided *const *ts, int n) {
    const int64_t es = (int64_t)elem_size(a.dtype), per = 16 / es;
    if (a.D % per) return false;
    for (int i = 0; i < n; ++i) {
        const dc1d_strided *t = ts[i];
        if (!t) continue;
        if ((uintptr_t)t->data & 15) return false;
        for (int d = 0; d < 3; ++d)
            if (t->shape[d] > 1 && t->stride[d] % per) return false;
    }
    return true;
}

// A dimension of size 1 is never stepped along; its stride is made 0 so that
// no arithmetic on it matters.
Strides3 steps(const dc1d_strided *t) {
    Strides3 s = strides(t);
    if (t->shape[0] <= 1) s.b = 0;
    if (t->shape[1] <= 1) s.l = 0;
    if (t->shape[2] <= 1) s.h = 0;
    return s;
}

}  // namespace

extern "C" {

int dc1d_layer_norm(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                    const dc1d_tensor *y, const dc1d_tensor *mean_or_null, const dc1d_tensor *rstd_or_null, double eps,
                    void *stream) {
    int64_t B, C, L;
    int st = ln_shape(x, &B, &C, &L);
    if (st) return st;
    if (!y) return DC1D_ERR_NULL_PTR;
    if (!(eps >= 0.0) || !(eps <= 3.0e38)) return DC1D_ERR_BAD_ARG;
    if ((st = ln_like(y, x))) return st;
    for (const dc1d_tensor *t : {weight_or_null, bias_or_null})
        if (t && (st = ln_param(t, x))) return st;
    for (const dc1d_tensor *t : {mean_or_null, rstd_or_null})
        if (t && (st = ln_stat(t, x))) return st;
    const dc1d_tensor *const all[6] = {x, weight_or_null, bias_or_null, y, mean_or_null, rstd_or_null};
    for (const dc1d_tensor *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 3; i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (all[i] && all[j] && !(i == 3 && j == 0 && y->data == x->data) && meet(range(all[i]), range(all[j])))
                return DC1D_ERR_ALIAS;
    int cus;
    if ((st = current_device(&cus))) return st;
    if (log_on())
        fprintf(stderr, "dc1d: layer_norm B=%lld C=%lld L=%lld %s\n", (long long)B, (long long)C, (long long)L,
                x->dtype == DC1D_F32 ? "f32" : "bf16");
    if (B * L == 0) return DC1D_OK;
    LayerNormArgs a = {};
    a.x = x->data;
    a.w = weight_or_null ? weight_or_null->data : nullptr;
    a.b = bias_or_null ? bias_or_null->data : nullptr;
    a.y = y->data;
    a.mean = mean_or_null ? (float *)mean_or_null->data : nullptr;
    a.rstd = rstd_or_null ? (float *)rstd_or_null->data : nullptr;
    a.dtype = x->dtype;
    a.B = B, a.C = (int)C, a.L = L;
    a.inv_c = 1.0f / (float)C;
    a.eps = (float)eps;
    return launched(launch_layer_norm(a, cus, (hipStream_t)stream));
}

int dc1d_layer_norm_backward_workspace_bytes(const dc1d_tensor *x, int want_params, size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    int64_t B, C, L;
    int st = ln_shape(x, &B, &C, &L), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = layer_norm_backward_workspace(B, (int)C, L, x->dtype, want_params != 0, cus);
    return DC1D_OK;
}

int dc1d_layer_norm_backward(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *grad_out,
                             const dc1d_tensor *mean, const dc1d_tensor *rstd, const dc1d_tensor *grad_x_or_null,
                             const dc1d_tensor *grad_weight_or_null, const dc1d_tensor *grad_bias_or_null,
                             void *workspace, size_t workspace_bytes, void *stream) {
    int64_t B, C, L;
    int st = ln_shape(x, &B, &C, &L);
    if (st) return st;
    if (!grad_out || !mean || !rstd) return DC1D_ERR_NULL_PTR;
    for (const dc1d_tensor *t : {grad_out, grad_x_or_null})
        if (t && (st = ln_like(t, x))) return st;
    for (const dc1d_tensor *t : {weight_or_null, grad_weight_or_null, grad_bias_or_null})
        if (t && (st = ln_param(t, x))) return st;
    for (const dc1d_tensor *t : {mean, rstd})
        if ((st = ln_stat(t, x))) return st;
    const dc1d_tensor *const all[8] = {grad_out, x, weight_or_null, mean, rstd, grad_x_or_null, grad_weight_or_null,
                                       grad_bias_or_null};
    for (const dc1d_tensor *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 5; i < 8; ++i)
        for (int j = 0; j < i; ++j)
            if (all[i] && all[j] && !(i == 5 && j == 0 && all[5]->data == all[0]->data) &&
                meet(range(all[i]), range(all[j])))
                return DC1D_ERR_ALIAS;
    int cus;
    if ((st = current_device(&cus))) return st;
    const bool params = grad_weight_or_null || grad_bias_or_null;
    const size_t need = layer_norm_backward_workspace(B, (int)C, L, x->dtype, params, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, need))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    for (const dc1d_tensor *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    if (log_on())
        fprintf(stderr, "dc1d: layer_norm_backward B=%lld C=%lld L=%lld %s ws=%zu\n", (long long)B, (long long)C,
                (long long)L, x->dtype == DC1D_F32 ? "f32" : "bf16", need);
    LayerNormArgs a = {};
    a.x = x->data;
    a.w = weight_or_null ? weight_or_null->data : nullptr;
    a.g = grad_out->data;
    a.mean = (float *)mean->data;
    a.rstd = (float *)rstd->data;
    a.y = grad_x_or_null ? grad_x_or_null->data : nullptr;
    a.gw = grad_weight_or_null ? grad_weight_or_null->data : nullptr;
    a.gb = grad_bias_or_null ? grad_bias_or_null->data : nullptr;
    a.dtype = x->dtype;
    a.B = B, a.C = (int)C, a.L = L;
    a.inv_c = 1.0f / (float)C;
    a.ws = (float *)workspace;
    if (!a.y && !params) return DC1D_OK;
    return launched(launch_layer_norm_backward(a, cus, (hipStream_t)stream));
}

int dc1d_rotary(const dc1d_strided *q, const dc1d_strided *k_or_null, const dc1d_tensor *cos, const dc1d_tensor *sin,
                const dc1d_tensor *positions, const dc1d_strided *q_out, const dc1d_strided *k_out_or_null,
                const int64_t *sections, int32_t n_axes, int interleaved, int inverse, void *stream) {
    if (!q || !q_out || !cos || !sin || !positions || !sections || !k_or_null != !k_out_or_null) return DC1D_ERR_NULL_PTR;
    const dc1d_strided *const in[2] = {q, k_or_null}, *const out[2] = {q_out, k_out_or_null};
    if (n_axes < 1 || n_axes > 4) return DC1D_ERR_BAD_ARG;
    if (!data_dtype(q->dtype)) return DC1D_ERR_BAD_DTYPE;
    const int64_t B = q->shape[0], L = q->shape[1], D = q->shape[3];
    int64_t span, heads = 0;
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        if (in[i]->dtype != q->dtype || out[i]->dtype != q->dtype) return DC1D_ERR_BAD_DTYPE;
        if (count(in[i], &span) < 0 || count(out[i], &span) < 0) return DC1D_ERR_BAD_SHAPE;
        if (in[i]->shape[0] != B || in[i]->shape[1] != L || in[i]->shape[3] != D) return DC1D_ERR_BAD_SHAPE;
        for (int d = 0; d < 4; ++d)
            if (out[i]->shape[d] != in[i]->shape[d]) return DC1D_ERR_BAD_SHAPE;
        if (in[i]->shape[2] < 1 || in[i]->shape[2] > (1 << 24)) return DC1D_ERR_BAD_SHAPE;
        heads += in[i]->shape[2];
        if (!distinct(out[i])) return DC1D_ERR_ALIAS;
    }
    if (D < 2 || D > (1 << 24) || B >= kLim31 || L >= kLim31 || B * L >= kLim31) return DC1D_ERR_BAD_SHAPE;
    if (heads * D >= (1 << 30) || heads * D * (B * L) >= (int64_t)1 << 40) return DC1D_ERR_BAD_SHAPE;
    int64_t R = 0;
    int first[4];
    for (int i = 0; i < 4; ++i) {
        if (i < n_axes && (sections[i] < 0 || sections[i] > D)) return DC1D_ERR_BAD_ARG;
        first[i] = (int)R;
        if (i < n_axes) R += sections[i];
    }
    for (int i = n_axes; i < 4; ++i) first[i] = (int)R;
    if (R < 1 || 2 * R > D) return DC1D_ERR_BAD_ARG;
    if (cos->dtype != DC1D_F32 || sin->dtype != DC1D_F32 || positions->dtype != DC1D_I32) return DC1D_ERR_BAD_DTYPE;
    if (cos->ndim != 2 || count(cos) < 0 || cos->shape[0] < 1 || cos->shape[0] >= kLim31 || cos->shape[1] != R ||
        !shape_is(sin, 2, cos->shape))
        return DC1D_ERR_BAD_SHAPE;
    const int64_t ps[3] = {B, L, n_axes}, p1[3] = {1, L, n_axes};
    if (!shape_is(positions, 3, ps) && !shape_is(positions, 3, p1)) return DC1D_ERR_BAD_SHAPE;
    for (const dc1d_strided *t : {q, k_or_null, q_out, k_out_or_null})
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (const dc1d_tensor *t : {cos, sin, positions})
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 0; i < 2; ++i) {
        if (!out[i]) continue;
        for (int j = 0; j < 2; ++j)
            if (in[j] && !(i == j && same_view(out[i], in[j])) && clash(out[i], in[j])) return DC1D_ERR_ALIAS;
        for (const dc1d_tensor *t : {cos, sin, positions})
            if (clash(out[i], t)) return DC1D_ERR_ALIAS;
    }
    if (clash(q_out, k_out_or_null)) return DC1D_ERR_ALIAS;
    int cus, st = current_device(&cus);
    if (st) return st;
    if (log_on())
        fprintf(stderr, "dc1d: rotary B=%lld L=%lld Hq=%lld Hkv=%lld D=%lld R=%lld axes=%d interleaved=%d inverse=%d %s\n",
                (long long)B, (long long)L, (long long)q->shape[2], (long long)(k_or_null ? k_or_null->shape[2] : 0),
                (long long)D, (long long)R, (int)n_axes, interleaved != 0, inverse != 0,
                q->dtype == DC1D_F32 ? "f32" : "bf16");
    if (B * L == 0) return DC1D_OK;
    RotaryArgs a = {};
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        a.t[i].x = in[i]->data;
        a.t[i].y = out[i]->data;
        a.t[i].xs = steps(in[i]);
        a.t[i].ys = steps(out[i]);
        a.t[i].H = (int)in[i]->shape[2];
    }
    a.cos = (const float *)cos->data;
    a.sin = (const float *)sin->data;
    a.pos = (const int *)positions->data;
    a.pos_b = positions->shape[0] == 1 ? 0 : L * n_axes;
    a.dtype = q->dtype;
    a.B = (int)B, a.L = (int)L, a.D = (int)D, a.R = (int)R, a.A = n_axes, a.P = (int)cos->shape[0];
    memcpy(a.first, first, sizeof(first));
    a.interleaved = interleaved != 0;
    a.sign = inverse ? -1.0f : 1.0f;
    return launched(launch_rotary(a, (hipStream_t)stream));
}

int dc1d_attention_workspace_bytes(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                                   size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    AttnArgs a;
    int st = attn_shape(q, k, v, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = plan_attention(a, cus).ws_bytes;
    return DC1D_OK;
}

int dc1d_attention_plan(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v, const char **kernel_name,
                        int64_t *grid_blocks, int32_t *splits) {
    AttnArgs a;
    int st = attn_shape(q, k, v, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    const AttnPlan pl = plan_attention(a, cus);
    if (kernel_name) *kernel_name = pl.name;
    if (grid_blocks) *grid_blocks = pl.blocks;
    if (splits) *splits = pl.splits;
    return DC1D_OK;
}

int dc1d_attention(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                   const dc1d_tensor *kv_lens_or_null, const dc1d_tensor *q_start_or_null, const dc1d_strided *out,
                   const dc1d_tensor *lse_or_null, int causal, int64_t window, double scale, void *workspace,
                   size_t workspace_bytes, void *stream) {
    AttnArgs a;
    int st = attn_shape(q, k, v, &a);
    if (st) return st;
    if (!out) return DC1D_ERR_NULL_PTR;
    if ((st = like_q(out, q))) return st;
    if ((st = attn_rest(q, kv_lens_or_null, q_start_or_null, lse_or_null, causal, window, scale, &a))) return st;
    const dc1d_strided *const all[4] = {q, k, v, out};
    for (const dc1d_strided *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    if (!distinct(out)) return DC1D_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
        if (clash(out, all[i])) return DC1D_ERR_ALIAS;
    const dc1d_tensor *const small[3] = {kv_lens_or_null, q_start_or_null, lse_or_null};
    for (const dc1d_tensor *t : small)
        if (clash(out, t)) return DC1D_ERR_ALIAS;
    if (lse_or_null) {
        for (int i = 0; i < 3; ++i)
            if (clash(range(lse_or_null), all[i])) return DC1D_ERR_ALIAS;
        for (int i = 0; i < 2; ++i)
            if (clash(range(lse_or_null), small[i])) return DC1D_ERR_ALIAS;
    }
    int cus;
    if ((st = current_device(&cus))) return st;
    const AttnPlan pl = plan_attention(a, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, pl.ws_bytes))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + pl.ws_bytes};
    for (const dc1d_strided *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    for (const dc1d_tensor *t : small)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    a.out = out->data;
    a.os = steps(out);
    a.qs = steps(q), a.ks = steps(k), a.vs = steps(v);
    a.vec = pieces(a, all, 4);
    if (log_on())
        fprintf(stderr, "dc1d: attention B=%d Lq=%d Lk=%d Hq=%d Hkv=%d D=%d causal=%d window=%d %s -> %s grid=%lld "
                        "splits=%d ws=%zu\n",
                a.B, a.Lq, a.Lk, a.Hq, a.Hkv, a.D, a.causal, a.window, a.dtype == kF32 ? "f32" : "bf16", pl.name,
                (long long)pl.blocks, pl.splits, pl.ws_bytes);
    if (a.B == 0 || a.rows == 0) return DC1D_OK;
    return launched(launch_attention(a, pl, workspace, (hipStream_t)stream));
}

int dc1d_attention_backward_workspace_bytes(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                                            size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    AttnArgs a;
    int st = attn_shape(q, k, v, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = plan_attention_backward(a, cus).ws_bytes;
    return DC1D_OK;
}

int dc1d_attention_backward(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                            const dc1d_tensor *kv_lens_or_null, const dc1d_tensor *q_start_or_null,
                            const dc1d_strided *out, const dc1d_tensor *lse, const dc1d_strided *grad_out,
                            const dc1d_strided *grad_q_or_null, const dc1d_strided *grad_k_or_null,
                            const dc1d_strided *grad_v_or_null, int causal, int64_t window, double scale,
                            void *workspace, size_t workspace_bytes, void *stream) {
    AttnArgs a;
    int st = attn_shape(q, k, v, &a);
    if (st) return st;
    if (!out || !lse || !grad_out) return DC1D_ERR_NULL_PTR;
    for (const dc1d_strided *t : {out, grad_out, grad_q_or_null})
        if (t && (st = like_q(t, q))) return st;
    for (const dc1d_strided *t : {grad_k_or_null, grad_v_or_null})
        if (t && (st = like_q(t, k))) return st;
    if ((st = attn_rest(q, kv_lens_or_null, q_start_or_null, lse, causal, window, scale, &a))) return st;
    const dc1d_strided *const all[8] = {q, k, v, out, grad_out, grad_q_or_null, grad_k_or_null, grad_v_or_null};
    const dc1d_tensor *const small[3] = {kv_lens_or_null, q_start_or_null, lse};
    for (const dc1d_strided *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 5; i < 8; ++i) {
        if (!all[i]) continue;
        if (!distinct(all[i])) return DC1D_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (clash(all[i], all[j])) return DC1D_ERR_ALIAS;
        for (const dc1d_tensor *t : small)
            if (clash(all[i], t)) return DC1D_ERR_ALIAS;
    }
    int cus;
    if ((st = current_device(&cus))) return st;
    const AttnBwdPlan pl = plan_attention_backward(a, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, pl.ws_bytes))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + pl.ws_bytes};
    for (const dc1d_strided *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    for (const dc1d_tensor *t : small)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    a.qs = steps(q), a.ks = steps(k), a.vs = steps(v), a.os = steps(out), a.gs = steps(grad_out);
    a.o = out->data;
    a.g = grad_out->data;
    if (grad_q_or_null) a.gq = grad_q_or_null->data, a.gqs = steps(grad_q_or_null);
    if (grad_k_or_null) a.gk = grad_k_or_null->data, a.gks = steps(grad_k_or_null);
    if (grad_v_or_null) a.gv = grad_v_or_null->data, a.gvs = steps(grad_v_or_null);
    a.vec = pieces(a, all, 8);
    if (log_on())
        fprintf(stderr, "dc1d: attention_backward B=%d Lq=%d Lk=%d Hq=%d Hkv=%d D=%d causal=%d window=%d %s splits=%d "
                        "ws=%zu\n",
                a.B, a.Lq, a.Lk, a.Hq, a.Hkv, a.D, a.causal, a.window, a.dtype == kF32 ? "f32" : "bf16", pl.splits,
                pl.ws_bytes);
    if (a.B == 0 || (a.rows == 0 && a.Lk == 0)) return DC1D_OK;
    return launched(launch_attention_backward(a, pl, workspace, (hipStream_t)stream));
}

}  // extern "C"
