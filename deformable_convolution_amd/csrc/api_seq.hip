// api_seq.hip -- the C ABI of the sequence operators (include/dc1d.h):
// argument validation, kernel choice, and launch.  No allocation, no
// synchronisation, no exceptions across the boundary.
#include <math.h>

#include "seq_check.h"

using namespace dc1d;

namespace {

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
