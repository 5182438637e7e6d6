// bind_seq.cpp -- the sequence operators' Python binding, as a CPython module.
//
// Argument marshalling only: torch tensors become the descriptors of
// include/dc1d.h, outputs are allocated, the C entry is called.  It is
// compiled because small calls are bound by the host: the same steps in
// Python take two to three times as long as the launch itself.  The entries'
// addresses come from Python, which loads the library (bind()).
//
// Every function returns the status first; Python turns it into an exception.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Functions.h>

#include "dc1d.h"

namespace {

struct Entries {
    decltype(&dc1d_layer_norm) layer_norm;
    decltype(&dc1d_layer_norm_backward_workspace_bytes) layer_norm_backward_ws;
    decltype(&dc1d_layer_norm_backward) layer_norm_backward;
    decltype(&dc1d_rotary) rotary;
    decltype(&dc1d_attention_workspace_bytes) attention_ws;
    decltype(&dc1d_attention) attention;
    decltype(&dc1d_attention_backward_workspace_bytes) attention_backward_ws;
    decltype(&dc1d_attention_backward) attention_backward;
} entry;

int32_t dtype_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
    case at::kFloat: return DC1D_F32;
    case at::kBFloat16: return DC1D_BF16;
    case at::kInt: return DC1D_I32;
    default: return -1;
    }
}

// An argument that may be None: a tensor on the call's device.
struct Arg {
    at::Tensor t;
    bool given = false;
};

[[noreturn]] void refuse(const std::string &what) {
    TORCH_CHECK_VALUE(false, what);
    std::abort();  // not reached
}

struct Call {
    int device = -1;
    // required: not None.  The first tensor decides the device.
    at::Tensor tensor(PyObject *o, const char *name) {
        if (!THPVariable_Check(o)) throw torch::TypeError(std::string(name) + " must be a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse("tensors must be on the GPU");
        if (device < 0) device = t.get_device();
        if (t.get_device() != device) refuse("all tensors must be on one device");
        return t;
    }
    Arg maybe(PyObject *o, const char *name) {
        Arg a;
        if (o != Py_None) a.t = tensor(o, name), a.given = true;
        return a;
    }
};

struct Dense {
    dc1d_tensor d;
    const dc1d_tensor *p = nullptr;
    void set(const at::Tensor &t, const char *name) {
        if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        d.data = t.data_ptr();
        d.dtype = dtype_of(t);
        d.ndim = (int32_t)t.dim();
        for (int i = 0; i < 4; ++i) d.shape[i] = i < d.ndim ? t.size(i) : 0;
        p = &d;
    }
    void set(const Arg &a, const char *name) {
        if (a.given) set(a.t, name);
    }
};
struct Strided {
    dc1d_strided d;
    const dc1d_strided *p = nullptr;
    void set(const at::Tensor &t, const char *name) {
        if (t.dim() != 4) refuse(std::string(name) + " must have four dimensions");
        d.data = t.data_ptr();
        d.dtype = dtype_of(t);
        d.ndim = 4;
        for (int i = 0; i < 4; ++i) d.shape[i] = t.size(i), d.stride[i] = t.stride(i);
        p = &d;
    }
    void set(const Arg &a, const char *name) {
        if (a.given) set(a.t, name);
    }
};

at::Tensor fresh(const at::Tensor &like, at::IntArrayRef shape) { return at::empty(shape, like.options()); }

// The workspace of a call: the caller's tensor, or what `get(bytes, device)` gives.
struct Workspace {
    at::Tensor t;
    void *p = nullptr;
    size_t n = 0;
    bool take(PyObject *given, PyObject *get, size_t need, int device) {
        if (given != Py_None) {
            if (!THPVariable_Check(given)) throw torch::TypeError("workspace must be a tensor");
            t = THPVariable_Unpack(given);
            if (!t.is_cuda() || t.get_device() != device) refuse("the workspace must be on the tensors' device");
            // a view's elements need not be as many bytes of memory (expand), nor the view's alone (a step)
            if (!t.is_contiguous()) refuse("the workspace must be contiguous");
        } else if (need > 0) {
            PyObject *o = PyObject_CallFunction(get, "ni", (Py_ssize_t)need, device);
            if (!o) return false;
            t = THPVariable_Unpack(o);
            Py_DECREF(o);
        } else {
            return true;
        }
        p = t.data_ptr();
        n = t.nbytes();
        return true;
    }
};

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *result(int status, std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New(1 + (Py_ssize_t)ts.size());
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
    Py_ssize_t i = 1;
    for (const at::Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}
PyObject *failed(int status, size_t n) {
    PyObject *r = PyTuple_New(1 + (Py_ssize_t)n);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
    for (size_t i = 1; i <= n; ++i) {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, (Py_ssize_t)i, Py_None);
    }
    return r;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
void *stream_of(PyObject *o) { return (void *)(uintptr_t)integer(o); }

void expect(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) throw torch::TypeError("wrong number of arguments");
}

// x, weight, bias, eps, with_stats, out, stream -> status, y, mean, rstd
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 7);
    Call c;
    const at::Tensor x = c.tensor(a[0], "x");
    const Arg w = c.maybe(a[1], "weight"), b = c.maybe(a[2], "bias"), out = c.maybe(a[5], "out");
    Dense dx, dw, db, dy, dm, dr;
    dx.set(x, "x");
    dw.set(w, "weight");
    db.set(b, "bias");
    if (x.dim() < 2) return failed(DC1D_ERR_BAD_SHAPE, 3);
    const at::Tensor y = out.given ? out.t : fresh(x, x.sizes());
    dy.set(y, "out");
    at::Tensor mean, rstd;
    if (truth(a[4])) {
        c10::SmallVector<int64_t, 4> shape(x.sizes().begin(), x.sizes().end());
        shape.erase(shape.begin() + 1);
        mean = at::empty(shape, x.options().dtype(at::kFloat));
        rstd = at::empty(shape, x.options().dtype(at::kFloat));
        dm.set(mean, "mean");
        dr.set(rstd, "rstd");
    }
    return result(entry.layer_norm(dx.p, dw.p, db.p, dy.p, dm.p, dr.p, number(a[3]), stream_of(a[6])), {y, mean, rstd});
    END_HANDLE_TH_ERRORS
}

// x, grad_out, mean, rstd, weight, need x, need weight, need bias, workspace, get, stream
// -> status, grad x, grad weight, grad bias
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    Call c;
    const at::Tensor x = c.tensor(a[0], "x"), g = c.tensor(a[1], "grad_out"), m = c.tensor(a[2], "mean"), r = c.tensor(a[3], "rstd");
    const Arg w = c.maybe(a[4], "weight");
    Dense dx, dg, dm, dr, dw, gx, gw, gb;
    dx.set(x, "x");
    dg.set(g, "grad_out");
    dm.set(m, "mean");
    dr.set(r, "rstd");
    dw.set(w, "weight");
    if (x.dim() < 2) return failed(DC1D_ERR_BAD_SHAPE, 3);
    at::Tensor tx, tw, tb;
    if (truth(a[5])) tx = fresh(x, x.sizes()), gx.set(tx, "grad_x");
    if (truth(a[6])) tw = fresh(x, {x.size(1)}), gw.set(tw, "grad_weight");
    if (truth(a[7])) tb = fresh(x, {x.size(1)}), gb.set(tb, "grad_bias");
    size_t need = 0;
    if (tw.defined() || tb.defined())
        if (const int st = entry.layer_norm_backward_ws(dx.p, 1, &need)) return failed(st, 3);
    Workspace ws;
    if (!ws.take(a[8], a[9], need, c.device)) return nullptr;
    return result(entry.layer_norm_backward(dx.p, dw.p, dg.p, dm.p, dr.p, gx.p, gw.p, gb.p, ws.p, ws.n, stream_of(a[10])),
                  {tx, tw, tb});
    END_HANDLE_TH_ERRORS
}

// q, k, cos, sin, positions, sections (tuple), interleaved, inverse, q out, k out, stream -> status, q', k'
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    Call c;
    const at::Tensor q = c.tensor(a[0], "q"), co = c.tensor(a[2], "cos"), si = c.tensor(a[3], "sin"), po = c.tensor(a[4], "positions");
    const Arg k = c.maybe(a[1], "k"), qo = c.maybe(a[8], "out"), ko = c.maybe(a[9], "out");
    Strided dq, dk, dqo, dko;
    Dense dc, ds, dp;
    dq.set(q, "q");
    dk.set(k, "k");
    dc.set(co, "cos");
    ds.set(si, "sin");
    dp.set(po, "positions");
    const at::Tensor q2 = qo.given ? qo.t : fresh(q, q.sizes());
    dqo.set(q2, "out");
    at::Tensor k2;
    if (k.given) {
        k2 = ko.given ? ko.t : fresh(k.t, k.t.sizes());
        dko.set(k2, "out");
    }
    if (!PyTuple_Check(a[5])) throw torch::TypeError("sections must be a tuple");
    const Py_ssize_t axes = PyTuple_GET_SIZE(a[5]);
    int64_t sections[4] = {0, 0, 0, 0};
    for (Py_ssize_t i = 0; i < axes && i < 4; ++i) sections[i] = integer(PyTuple_GET_ITEM(a[5], i));
    return result(entry.rotary(dq.p, dk.p, dc.p, ds.p, dp.p, dqo.p, dko.p, sections, (int32_t)(axes < 5 ? axes : 5), truth(a[6]),
                               truth(a[7]), stream_of(a[10])),
                  {q2, k2});
    END_HANDLE_TH_ERRORS
}

// q, k, v, causal, window, scale, kv_lens, q_start, with_lse, out, workspace, get, stream -> status, out, lse
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    Call c;
    const at::Tensor q = c.tensor(a[0], "q"), k = c.tensor(a[1], "k"), v = c.tensor(a[2], "v");
    const Arg lens = c.maybe(a[6], "kv_lens"), start = c.maybe(a[7], "q_start"), given = c.maybe(a[9], "out");
    Strided dq, dk, dv, dout;
    Dense dl, dst, dlse;
    dq.set(q, "q");
    dk.set(k, "k");
    dv.set(v, "v");
    dl.set(lens, "kv_lens");
    dst.set(start, "q_start");
    size_t need = 0;
    if (const int st = entry.attention_ws(dq.p, dk.p, dv.p, &need)) return failed(st, 2);
    const at::Tensor out = given.given ? given.t : fresh(q, q.sizes());
    dout.set(out, "out");
    at::Tensor lse;
    if (truth(a[8])) {
        lse = at::empty({q.size(0), q.size(2), q.size(1)}, q.options().dtype(at::kFloat));
        dlse.set(lse, "lse");
    }
    Workspace ws;
    if (!ws.take(a[10], a[11], need, c.device)) return nullptr;
    return result(entry.attention(dq.p, dk.p, dv.p, dl.p, dst.p, dout.p, dlse.p, truth(a[3]), integer(a[4]), number(a[5]), ws.p, ws.n,
                                  stream_of(a[12])),
                  {out, lse});
    END_HANDLE_TH_ERRORS
}

// q, k, v, out, lse, grad_out, causal, window, scale, kv_lens, q_start, then for q, k and v: a
// tensor to write, True (allocate) or None (not wanted), workspace, get, stream
// -> status, grad q, grad k, grad v
PyObject *attention_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 17);
    Call c;
    const at::Tensor in[3] = {c.tensor(a[0], "q"), c.tensor(a[1], "k"), c.tensor(a[2], "v")};
    const at::Tensor out = c.tensor(a[3], "out"), lse = c.tensor(a[4], "lse"), g = c.tensor(a[5], "grad_out");
    const Arg lens = c.maybe(a[9], "kv_lens"), start = c.maybe(a[10], "q_start");
    Strided d[3], dout, dg, grad[3];
    Dense dlse, dl, dst;
    for (int i = 0; i < 3; ++i) d[i].set(in[i], i == 0 ? "q" : i == 1 ? "k" : "v");
    dout.set(out, "out");
    dg.set(g, "grad_out");
    dlse.set(lse, "lse");
    dl.set(lens, "kv_lens");
    dst.set(start, "q_start");
    at::Tensor grads[3];
    for (int i = 0; i < 3; ++i) {
        if (a[11 + i] == Py_None) continue;
        grads[i] = a[11 + i] == Py_True ? fresh(in[i], in[i].sizes()) : c.tensor(a[11 + i], "grads");
        grad[i].set(grads[i], "grads");
    }
    size_t need = 0;
    if (const int st = entry.attention_backward_ws(d[0].p, d[1].p, d[2].p, &need)) return failed(st, 3);
    Workspace ws;
    if (!ws.take(a[14], a[15], need, c.device)) return nullptr;
    return result(entry.attention_backward(d[0].p, d[1].p, d[2].p, dl.p, dst.p, dout.p, dlse.p, dg.p, grad[0].p, grad[1].p, grad[2].p,
                                           truth(a[6]), integer(a[7]), number(a[8]), ws.p, ws.n, stream_of(a[16])),
                  {grads[0], grads[1], grads[2]});
    END_HANDLE_TH_ERRORS
}

// The entries' addresses, in the order of Entries.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    void *p[8];
    expect(n, 8);
    for (int i = 0; i < 8; ++i) p[i] = stream_of(a[i]);
    static_assert(sizeof(entry) == sizeof(p), "one address an entry");
    memcpy(&entry, p, sizeof(p));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FN(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(bind), FN(layer_norm), FN(layer_norm_backward), FN(rotary), FN(attention), FN(attention_backward),
                         {nullptr, nullptr, 0, nullptr}};
#undef FN
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seq", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seq() { return PyModule_Create(&module); }
