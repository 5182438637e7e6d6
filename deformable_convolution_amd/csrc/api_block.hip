// api_block.hip -- the C ABI of group norm and the gated recurrence
// (include/dc1d.h): argument validation and launch.  No allocation, no
// synchronisation, no exceptions across the boundary.
#include "seq_check.h"

using namespace dc1d;

namespace {

const char *dtype_name(int32_t dt) { return dt == DC1D_F32 ? "f32" : "bf16"; }

// ---- group norm ------------------------------------------------------------------

int gn_shape(const dc1d_tensor *x, int64_t groups, GroupNormArgs *a) {
    if (!x) return DC1D_ERR_NULL_PTR;
    if (!data_dtype(x->dtype)) return DC1D_ERR_BAD_DTYPE;
    if (x->ndim < 2 || x->ndim > 4 || count(x) < 0) return DC1D_ERR_BAD_SHAPE;
    const int64_t B = x->shape[0], C = x->shape[x->ndim - 1];
    int64_t S = 1;
    if (C < 1 || C > (1 << 24) || B >= kLim31) return DC1D_ERR_BAD_SHAPE;
    for (int i = 1; i < x->ndim - 1; ++i) {
        if (x->shape[i] >= kLim31 || S * x->shape[i] >= kLim31) return DC1D_ERR_BAD_SHAPE;
        S *= x->shape[i];
    }
    if (B * S >= kLim31) return DC1D_ERR_BAD_SHAPE;
    if (groups < 1 || groups > C || C % groups) return DC1D_ERR_BAD_ARG;
    if (B * groups >= kLim31) return DC1D_ERR_BAD_SHAPE;
    memset((void *)a, 0, sizeof(*a));
    a->dtype = x->dtype;
    a->B = B, a->S = S;
    a->C = (int)C, a->G = (int)groups, a->D = (int)(C / groups);
    return DC1D_OK;
}
int gn_like(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != x->dtype) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, x->ndim, x->shape) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int gn_param(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != x->dtype) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 1, x->shape + x->ndim - 1) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int gn_stat(const dc1d_tensor *t, const GroupNormArgs &a) {
    const int64_t s[2] = {a.B, a.G};
    if (t->dtype != DC1D_F32) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 2, s) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int gn_lens(const dc1d_tensor *t, const dc1d_tensor *x) {
    if (t->dtype != DC1D_I32) return DC1D_ERR_BAD_DTYPE;
    return x->ndim == 3 && shape_is(t, 1, x->shape) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
bool activation_ok(int act) { return act == DC1D_ACT_NONE || act == DC1D_ACT_RELU || act == DC1D_ACT_SILU; }

// ---- gated recurrence ------------------------------------------------------------

// A tensor [B, L, C] as one of rank 4, whose checks it then has.
struct Rank4 {
    dc1d_strided d;
    const dc1d_strided *p = nullptr;
    explicit Rank4(const dc1d_strided *t) {
        if (!t) return;
        d = {t->data, t->dtype, t->ndim == 3 ? 4 : -1, {t->shape[0], t->shape[1], 1, t->shape[2]}, {t->stride[0], t->stride[1], 0, t->stride[2]}};
        p = &d;
    }
};

int rec_shape(const dc1d_strided *x, RecurrenceArgs *a) {
    if (!x) return DC1D_ERR_NULL_PTR;
    if (!data_dtype(x->dtype)) return DC1D_ERR_BAD_DTYPE;
    int64_t span;
    if (count(x, &span) < 0) return DC1D_ERR_BAD_SHAPE;
    const int64_t B = x->shape[0], L = x->shape[1], C = x->shape[3];
    if (C < 1 || C > (1 << 24) || B >= kLim31 || L > kLen || B * L >= kLim31 || B * C >= kLim31) return DC1D_ERR_BAD_SHAPE;
    memset((void *)a, 0, sizeof(*a));
    a->dtype = x->dtype;
    a->B = (int)B, a->L = (int)L, a->C = (int)C;
    return DC1D_OK;
}
int rec_like(const dc1d_strided *t, const dc1d_strided *x) {
    if (t->dtype != x->dtype) return DC1D_ERR_BAD_DTYPE;
    int64_t span;
    if (count(t, &span) < 0) return DC1D_ERR_BAD_SHAPE;
    for (int i = 0; i < 4; ++i)
        if (t->shape[i] != x->shape[i]) return DC1D_ERR_BAD_SHAPE;
    return DC1D_OK;
}
int rec_state(const dc1d_tensor *t, const RecurrenceArgs &a) {
    const int64_t s[2] = {a.B, a.C};
    if (t->dtype != DC1D_F32) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 2, s) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int rec_states(const dc1d_tensor *t, const RecurrenceArgs &a) {
    const int64_t s[3] = {a.B, (a.L + kStateEvery - 1) / kStateEvery, a.C};
    if (t->dtype != DC1D_F32) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 3, s) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
int rec_lens(const dc1d_tensor *t, const RecurrenceArgs &a) {
    const int64_t s[1] = {a.B};
    if (t->dtype != DC1D_I32) return DC1D_ERR_BAD_DTYPE;
    return shape_is(t, 1, s) ? DC1D_OK : DC1D_ERR_BAD_SHAPE;
}
Strides2 steps2(const dc1d_strided *t) {
    const Strides3 s = steps(t);
    return {s.b, s.l};
}
bool same_tensor(const dc1d_tensor *a, const dc1d_tensor *b) { return a && b && a->data == b->data; }

}  // namespace

extern "C" {

int dc1d_group_norm_workspace_bytes(const dc1d_tensor *x, int64_t groups, size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    GroupNormArgs a;
    int st = gn_shape(x, groups, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = group_norm_workspace(a.B, a.S, a.C, a.G, a.dtype, cus);
    return DC1D_OK;
}

int dc1d_group_norm(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                    const dc1d_tensor *lens_or_null, const dc1d_tensor *y, const dc1d_tensor *mean_or_null,
                    const dc1d_tensor *rstd_or_null, int64_t groups, double eps, int activation, void *workspace,
                    size_t workspace_bytes, void *stream) {
    GroupNormArgs a;
    int st = gn_shape(x, groups, &a);
    if (st) return st;
    if (!y) return DC1D_ERR_NULL_PTR;
    if (!(eps >= 0.0) || !(eps <= 3.0e38) || !activation_ok(activation)) return DC1D_ERR_BAD_ARG;
    if ((st = gn_like(y, x))) return st;
    for (const dc1d_tensor *t : {weight_or_null, bias_or_null})
        if (t && (st = gn_param(t, x))) return st;
    if (lens_or_null && (st = gn_lens(lens_or_null, x))) return st;
    for (const dc1d_tensor *t : {mean_or_null, rstd_or_null})
        if (t && (st = gn_stat(t, a))) return st;
    const dc1d_tensor *const all[7] = {x, weight_or_null, bias_or_null, lens_or_null, y, mean_or_null, rstd_or_null};
    for (const dc1d_tensor *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 4; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            if (all[i] && all[j] && !(i == 4 && j == 0 && y->data == x->data) && meet(range(all[i]), range(all[j])))
                return DC1D_ERR_ALIAS;
    int cus;
    if ((st = current_device(&cus))) return st;
    const size_t need = group_norm_workspace(a.B, a.S, a.C, a.G, a.dtype, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, need))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    for (const dc1d_tensor *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    if (log_on())
        fprintf(stderr, "dc1d: group_norm B=%lld S=%lld C=%d groups=%d activation=%d lens=%d %s ws=%zu\n", (long long)a.B,
                (long long)a.S, a.C, a.G, activation, lens_or_null != nullptr, dtype_name(a.dtype), need);
    if (a.B == 0) return DC1D_OK;
    a.x = x->data;
    a.w = weight_or_null ? weight_or_null->data : nullptr;
    a.b = bias_or_null ? bias_or_null->data : nullptr;
    a.lens = lens_or_null ? (const int *)lens_or_null->data : nullptr;
    a.y = y->data;
    a.mean = mean_or_null ? (float *)mean_or_null->data : nullptr;
    a.rstd = rstd_or_null ? (float *)rstd_or_null->data : nullptr;
    a.act = activation;
    a.eps = (float)eps;
    a.ws = workspace;
    return launched(launch_group_norm(a, cus, (hipStream_t)stream));
}

int dc1d_group_norm_backward_workspace_bytes(const dc1d_tensor *x, int64_t groups, int want_params, size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    GroupNormArgs a;
    int st = gn_shape(x, groups, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = group_norm_backward_workspace(a.B, a.S, a.C, a.G, a.dtype, want_params != 0, cus);
    return DC1D_OK;
}

int dc1d_group_norm_backward(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                             const dc1d_tensor *lens_or_null, const dc1d_tensor *grad_out, const dc1d_tensor *mean,
                             const dc1d_tensor *rstd, const dc1d_tensor *grad_x_or_null,
                             const dc1d_tensor *grad_weight_or_null, const dc1d_tensor *grad_bias_or_null,
                             int64_t groups, int activation, void *workspace, size_t workspace_bytes, void *stream) {
    GroupNormArgs a;
    int st = gn_shape(x, groups, &a);
    if (st) return st;
    if (!grad_out || !mean || !rstd) return DC1D_ERR_NULL_PTR;
    if (!activation_ok(activation)) return DC1D_ERR_BAD_ARG;
    for (const dc1d_tensor *t : {grad_out, grad_x_or_null})
        if (t && (st = gn_like(t, x))) return st;
    for (const dc1d_tensor *t : {weight_or_null, bias_or_null, grad_weight_or_null, grad_bias_or_null})
        if (t && (st = gn_param(t, x))) return st;
    if (lens_or_null && (st = gn_lens(lens_or_null, x))) return st;
    for (const dc1d_tensor *t : {mean, rstd})
        if ((st = gn_stat(t, a))) return st;
    const dc1d_tensor *const all[10] = {grad_out, x,    weight_or_null, bias_or_null,        lens_or_null,
                                        mean,     rstd, grad_x_or_null, grad_weight_or_null, grad_bias_or_null};
    for (const dc1d_tensor *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 7; i < 10; ++i)
        for (int j = 0; j < i; ++j)
            if (all[i] && all[j] && !(i == 7 && j == 0 && all[7]->data == all[0]->data) &&
                meet(range(all[i]), range(all[j])))
                return DC1D_ERR_ALIAS;
    int cus;
    if ((st = current_device(&cus))) return st;
    const bool params = grad_weight_or_null || grad_bias_or_null;
    const size_t need = group_norm_backward_workspace(a.B, a.S, a.C, a.G, a.dtype, params, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, need))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    for (const dc1d_tensor *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    if (log_on())
        fprintf(stderr, "dc1d: group_norm_backward B=%lld S=%lld C=%d groups=%d activation=%d lens=%d %s ws=%zu\n",
                (long long)a.B, (long long)a.S, a.C, a.G, activation, lens_or_null != nullptr, dtype_name(a.dtype), need);
    a.x = x->data;
    a.w = weight_or_null ? weight_or_null->data : nullptr;
    a.b = bias_or_null ? bias_or_null->data : nullptr;
    a.lens = lens_or_null ? (const int *)lens_or_null->data : nullptr;
    a.g = grad_out->data;
    a.mean = (float *)mean->data;
    a.rstd = (float *)rstd->data;
    a.y = grad_x_or_null ? grad_x_or_null->data : nullptr;
    a.gw = grad_weight_or_null ? grad_weight_or_null->data : nullptr;
    a.gb = grad_bias_or_null ? grad_bias_or_null->data : nullptr;
    a.act = activation;
    a.ws = workspace;
    if (!a.y && !params) return DC1D_OK;
    return launched(launch_group_norm_backward(a, cus, (hipStream_t)stream));
}

int dc1d_gated_recurrence_workspace_bytes(const dc1d_strided *x, size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    RecurrenceArgs a;
    int st = rec_shape(Rank4(x).p, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = recurrence_workspace(a.B, a.L, a.C, a.dtype, false, cus);
    return DC1D_OK;
}

int dc1d_gated_recurrence(const dc1d_strided *x_, const dc1d_strided *gate_, const dc1d_tensor *state_or_null,
                          const dc1d_tensor *lens_or_null, const dc1d_strided *y_, const dc1d_tensor *last_or_null,
                          const dc1d_tensor *states_or_null, int blend, int reverse, void *workspace,
                          size_t workspace_bytes, void *stream) {
    const Rank4 x4(x_), gate4(gate_), y4(y_);
    const dc1d_strided *const x = x4.p, *const gate = gate4.p, *const y = y4.p;
    RecurrenceArgs a;
    int st = rec_shape(x, &a);
    if (st) return st;
    if (!gate || !y) return DC1D_ERR_NULL_PTR;
    if ((st = rec_like(gate, x)) || (st = rec_like(y, x))) return st;
    for (const dc1d_tensor *t : {state_or_null, last_or_null})
        if (t && (st = rec_state(t, a))) return st;
    if (states_or_null && (st = rec_states(states_or_null, a))) return st;
    if (lens_or_null && (st = rec_lens(lens_or_null, a))) return st;
    const dc1d_strided *const in[2] = {x, gate};
    const dc1d_tensor *const small[4] = {state_or_null, lens_or_null, last_or_null, states_or_null};
    for (const dc1d_strided *t : {x, gate, y})
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (const dc1d_tensor *t : small)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    if (!distinct(y)) return DC1D_ERR_ALIAS;
    for (const dc1d_strided *t : in)
        if (!(t == x && same_view(y, x)) && clash(y, t)) return DC1D_ERR_ALIAS;
    for (const dc1d_tensor *t : small)
        if (clash(y, t)) return DC1D_ERR_ALIAS;
    for (int i = 2; i < 4; ++i) {
        if (!small[i]) continue;
        for (const dc1d_strided *t : in)
            if (clash(range(small[i]), t)) return DC1D_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (!(i == 2 && j == 0 && same_tensor(small[2], small[0])) && clash(range(small[i]), small[j])) return DC1D_ERR_ALIAS;
    }
    int cus;
    if ((st = current_device(&cus))) return st;
    const size_t need = recurrence_workspace(a.B, a.L, a.C, a.dtype, false, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, need))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    for (const dc1d_strided *t : {x, gate, y})
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    for (const dc1d_tensor *t : small)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    if (log_on())
        fprintf(stderr, "dc1d: gated_recurrence B=%d L=%d C=%d blend=%d reverse=%d lens=%d states=%d %s ws=%zu\n", a.B, a.L, a.C,
                blend != 0, reverse != 0, lens_or_null != nullptr, states_or_null != nullptr, dtype_name(a.dtype), need);
    if (a.B == 0) return DC1D_OK;
    a.x = x->data, a.xs = steps2(x);
    a.gate = gate->data, a.gates = steps2(gate);
    a.y = y->data, a.ys = steps2(y);
    a.state = state_or_null ? (const float *)state_or_null->data : nullptr;
    a.lens = lens_or_null ? (const int *)lens_or_null->data : nullptr;
    a.last = last_or_null ? (float *)last_or_null->data : nullptr;
    a.states = states_or_null ? (float *)states_or_null->data : nullptr;
    a.blend = blend != 0, a.reverse = reverse != 0;
    a.in_place = a.y == a.x || (a.last && a.last == a.state);
    a.ws = workspace;
    return launched(launch_recurrence(a, cus, (hipStream_t)stream));
}

int dc1d_gated_recurrence_backward_workspace_bytes(const dc1d_strided *x, size_t *bytes_out) {
    if (!bytes_out) return DC1D_ERR_NULL_PTR;
    RecurrenceArgs a;
    int st = rec_shape(Rank4(x).p, &a), cus;
    if (st) return st;
    if ((st = current_device(&cus))) return st;
    *bytes_out = recurrence_workspace(a.B, a.L, a.C, a.dtype, true, cus);
    return DC1D_OK;
}

int dc1d_gated_recurrence_backward(const dc1d_strided *x_, const dc1d_strided *gate_, const dc1d_tensor *states,
                                   const dc1d_tensor *lens_or_null, const dc1d_strided *grad_out_,
                                   const dc1d_tensor *grad_last_or_null, const dc1d_strided *grad_x_or_null,
                                   const dc1d_strided *grad_gate_or_null, const dc1d_tensor *grad_state_or_null,
                                   int blend, int reverse, void *workspace, size_t workspace_bytes, void *stream) {
    const Rank4 x4(x_), gate4(gate_), g4(grad_out_), gx4(grad_x_or_null), gg4(grad_gate_or_null);
    const dc1d_strided *const x = x4.p, *const gate = gate4.p, *const g = g4.p, *const gx = gx4.p, *const gg = gg4.p;
    RecurrenceArgs a;
    int st = rec_shape(x, &a);
    if (st) return st;
    if (!gate || !g || !states) return DC1D_ERR_NULL_PTR;
    const dc1d_strided *const all[5] = {x, gate, g, gx, gg};
    const dc1d_tensor *const small[4] = {states, lens_or_null, grad_last_or_null, grad_state_or_null};
    for (const dc1d_strided *t : all)
        if (t && (st = rec_like(t, x))) return st;
    if ((st = rec_states(states, a))) return st;
    for (const dc1d_tensor *t : {grad_last_or_null, grad_state_or_null})
        if (t && (st = rec_state(t, a))) return st;
    if (lens_or_null && (st = rec_lens(lens_or_null, a))) return st;
    for (const dc1d_strided *t : all)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (const dc1d_tensor *t : small)
        if (!has_data(t)) return DC1D_ERR_NULL_PTR;
    for (int i = 3; i < 5; ++i) {
        if (!all[i]) continue;
        if (!distinct(all[i])) return DC1D_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (all[j] && !(i == 3 && j == 2 && same_view(gx, g)) && clash(all[i], all[j])) return DC1D_ERR_ALIAS;
        for (const dc1d_tensor *t : small)
            if (clash(all[i], t)) return DC1D_ERR_ALIAS;
    }
    if (grad_state_or_null) {
        const Range r = range(grad_state_or_null);
        for (int j = 0; j < 3; ++j)
            if (clash(r, all[j])) return DC1D_ERR_ALIAS;
        for (int j = 0; j < 3; ++j)
            if (!(j == 2 && same_tensor(small[2], small[3])) && clash(r, small[j])) return DC1D_ERR_ALIAS;
    }
    int cus;
    if ((st = current_device(&cus))) return st;
    const size_t need = recurrence_workspace(a.B, a.L, a.C, a.dtype, true, cus);
    if ((st = workspace_ok(workspace, workspace_bytes, need))) return st;
    const Range w = {(uintptr_t)workspace, (uintptr_t)workspace + need};
    for (const dc1d_strided *t : all)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    for (const dc1d_tensor *t : small)
        if (clash(w, t)) return DC1D_ERR_ALIAS;
    if (log_on())
        fprintf(stderr, "dc1d: gated_recurrence_backward B=%d L=%d C=%d blend=%d reverse=%d lens=%d %s ws=%zu\n", a.B, a.L, a.C,
                blend != 0, reverse != 0, lens_or_null != nullptr, dtype_name(a.dtype), need);
    a.x = x->data, a.xs = steps2(x);
    a.gate = gate->data, a.gates = steps2(gate);
    a.g = g->data, a.gs = steps2(g);
    if (gx) a.gx = gx->data, a.gxs = steps2(gx);
    if (gg) a.gg = gg->data, a.ggs = steps2(gg);
    a.states = (float *)states->data;
    a.lens = lens_or_null ? (const int *)lens_or_null->data : nullptr;
    a.g_last = grad_last_or_null ? (const float *)grad_last_or_null->data : nullptr;
    a.g_state = grad_state_or_null ? (float *)grad_state_or_null->data : nullptr;
    a.blend = blend != 0, a.reverse = reverse != 0;
    a.in_place = a.gx == a.g || (a.g_state && a.g_state == a.g_last);
    a.ws = workspace;
    if (a.B == 0 || (!a.gx && !a.gg && !a.g_state)) return DC1D_OK;
    return launched(launch_recurrence_backward(a, cus, (hipStream_t)stream));
}

}  // extern "C"
