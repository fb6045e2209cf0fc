// The common call of the linear-attention and layer-norm wrappers of binding.py, from torch tensors to the C ABI, in one
// native step: contiguous tensors of the expected types and shapes on the current device, on its current stream.  Small
// problems (a decode step's kernel takes 3 us) are bound by what a call costs on the host, and reading five tensors'
// properties from Python costs more than the launch: 12.0 us a decode call in all, 4.9 with this (layer norm 15.7 and 7.0).
// A function returns None for any other call, having done nothing: binding.py then checks, dispatches or raises.  A call that
// the library began and could not finish raises here: made again, a decode step would take its token twice.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "kdn.h"

namespace {

// the library's functions, by the addresses that binding.py has loaded them at
struct {
    decltype(&kdn_linear_workspace_size) linear_workspace_size;
    decltype(&kdn_linear_forward) linear_forward;
    decltype(&kdn_linear_decode_tokens) linear_decode_tokens;
    decltype(&kdn_linear_backward_workspace_size) linear_backward_workspace_size;
    decltype(&kdn_linear_backward) linear_backward;
    decltype(&kdn_layer_norm) layer_norm;
    decltype(&kdn_layer_norm_backward_workspace_size) layer_norm_backward_workspace_size;
    decltype(&kdn_layer_norm_backward) layer_norm_backward;
} kdn;

PyObject *error = nullptr;     // binding.KdnError(code, where)

// what a status other than KDN_OK comes to: None where the library has refused the arguments (before any launch), else the error
PyObject *refused(kdn_status_t st, const char *where) {
    if (st == KDN_ERR_INVALID_ARG || st == KDN_ERR_UNSUPPORTED || st == KDN_ERR_WORKSPACE) Py_RETURN_NONE;
    PyObject *e = error ? PyObject_CallFunction(error, "is", (int)st, where) : nullptr;
    if (e) {
        PyErr_SetObject(error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, (int)st);
    }
    return nullptr;
}

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
bool is(const at::Tensor &t, at::ScalarType type, c10::Device dev) {
    return t.layout() == at::kStrided && t.scalar_type() == type && t.device() == dev && t.is_contiguous();
}
bool is(const at::Tensor &t, at::ScalarType type, c10::Device dev, at::IntArrayRef shape) {
    return is(t, type, dev) && t.sizes() == shape;
}
// an optional tensor: its address or NULL; false if it is neither None nor such a tensor
bool optional(PyObject *o, at::ScalarType type, c10::Device dev, at::IntArrayRef shape, void **p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o);
    if (!t || !is(*t, type, dev, shape)) return false;
    *p = t->data_ptr();
    return true;
}
bool number(PyObject *o, float *x) {
    if (!PyFloat_CheckExact(o)) return false;
    *x = (float)PyFloat_AS_DOUBLE(o);
    return true;
}
bool elements(const at::Tensor &t, int *code) {
    const at::ScalarType s = t.scalar_type();
    *code = s == at::kBFloat16 ? KDN_DTYPE_BF16 : KDN_DTYPE_F32;
    return s == at::kBFloat16 || s == at::kFloat;
}
bool current(c10::Device dev) { return dev.is_cuda() && dev.index() == c10::cuda::current_device(); }
void *stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
at::Tensor scratch(size_t bytes, c10::Device dev) {
    return at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
}
at::Tensor floats(at::IntArrayRef shape, c10::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(at::kFloat).device(dev));
}

// q, k, v [B, T, H, d] (three dimensions: T = 1), g, cu_seqlens and the scale as a problem
struct Linear {
    const at::Tensor *q, *k, *v;
    void *g;
    kdn_linear_problem_t p;
    c10::Device dev = c10::Device(c10::kCPU);
    int64_t states[4];         // shape of a state
    bool read(PyObject *qo, PyObject *ko, PyObject *vo, PyObject *go, PyObject *cuo, PyObject *scale, int dims) {
        q = tensor(qo); k = tensor(ko); v = tensor(vo);
        int code;
        if (!q || !k || !v || q->dim() != dims || v->dim() != dims || !elements(*q, &code)) return false;
        dev = q->device();
        const at::ScalarType type = q->scalar_type();
        if (!current(dev) || !is(*q, type, dev) || !is(*k, type, dev, q->sizes()) || !is(*v, type, dev)) return false;
        for (int i = 0; i < dims; ++i)
            if (q->size(i) > INT_MAX || v->size(i) > INT_MAX || (i < dims - 1 && q->size(i) != v->size(i))) return false;
        p.B = (int)q->size(0);
        p.T = dims == 4 ? (int)q->size(1) : 1;
        p.H = (int)q->size(dims - 2);
        p.d_k = (int)q->size(dims - 1);
        p.d_v = (int)v->size(dims - 1);
        p.in_dtype = (kdn_dtype_t)code;
        if (!number(scale, &p.scale)) return false;
        p.cu_seqlens = nullptr;
        p.num_seqs = p.B;
        if (cuo != Py_None) {
            const at::Tensor *cu = tensor(cuo);
            if (!cu || cu->dim() != 1 || cu->size(0) < 1 || cu->size(0) > INT_MAX || p.B != 1 || !is(*cu, at::kInt, dev)) return false;
            p.cu_seqlens = static_cast<const int32_t *>(cu->data_ptr());
            p.num_seqs = (int)cu->size(0) - 1;
        }
        p.decay = KDN_DECAY_NONE;
        g = nullptr;
        if (go != Py_None) {
            const at::Tensor *t = tensor(go);
            if (!t || !is(*t, at::kFloat, dev)) return false;
            if (t->dim() == 1) {
                if (t->size(0) != p.H) return false;
                p.decay = KDN_DECAY_HEAD;
            } else {
                if (t->sizes() != q->sizes().slice(0, dims - 1)) return false;
                p.decay = KDN_DECAY_TOKEN;
            }
            g = t->data_ptr();
        }
        states[0] = p.num_seqs; states[1] = p.H; states[2] = p.d_k; states[3] = p.d_v;
        return true;
    }
    // the caller's tensor like `like`, or a new one
    bool output(PyObject *o, const at::Tensor &like, at::Tensor *out) const {
        if (o == Py_None) {
            *out = at::empty(like.sizes(), like.options());
            return true;
        }
        const at::Tensor *t = tensor(o);
        if (!t || !is(*t, like.scalar_type(), dev, like.sizes())) return false;
        *out = *t;
        return true;
    }
};

// linear_forward(q, k, v, g, cu_seqlens, S0, scale, o, S_out, want_state) -> (o, S_out)
PyObject *linear_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Linear l;
    void *s0;
    if (n != 10 || !PyBool_Check(a[9]) || !l.read(a[0], a[1], a[2], a[3], a[4], a[6], 4) || !optional(a[5], at::kFloat, l.dev, l.states, &s0)) Py_RETURN_NONE;
    at::Tensor o, s;
    void *sp;
    if (!optional(a[8], at::kFloat, l.dev, l.states, &sp)) Py_RETURN_NONE;
    size_t need;
    if (kdn.linear_workspace_size(&l.p, &need) != KDN_OK || !l.output(a[7], *l.v, &o)) Py_RETURN_NONE;
    if (a[8] != Py_None) {
        s = *tensor(a[8]);
    } else if (a[9] == Py_True) {
        s = floats(l.states, l.dev);
        sp = s.data_ptr();
    }
    const at::Tensor ws = need ? scratch(need, l.dev) : at::Tensor();
    const kdn_status_t st = kdn.linear_forward(&l.p, l.q->data_ptr(), l.k->data_ptr(), l.v->data_ptr(), static_cast<float *>(l.g), static_cast<float *>(s0),
                           o.data_ptr(), static_cast<float *>(sp), need ? ws.data_ptr() : nullptr, need, stream_of(l.dev));
    if (st != KDN_OK) return refused(st, "kdn_linear_forward");
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(o));
    PyTuple_SET_ITEM(r, 1, s.defined() ? THPVariable_Wrap(s) : Py_NewRef(Py_None));
    return r;
    END_HANDLE_TH_ERRORS
}

// linear_decode(q, k, v, g, S, scale, o, dims) -> o; token tensors of 4 dimensions, or 3 for one token
PyObject *linear_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Linear l;
    if (n != 8 || !PyLong_Check(a[7]) || !l.read(a[0], a[1], a[2], a[3], Py_None, a[5], (int)PyLong_AsLong(a[7]))) Py_RETURN_NONE;
    const at::Tensor *S = tensor(a[4]);
    at::Tensor o;
    if (!S || !is(*S, at::kFloat, l.dev, l.states) || !l.output(a[6], *l.v, &o)) Py_RETURN_NONE;
    const kdn_status_t st = kdn.linear_decode_tokens(l.p.B, l.p.T, l.p.H, l.p.d_k, l.p.d_v, l.p.in_dtype, l.p.scale, l.p.decay, l.q->data_ptr(),
                                 l.k->data_ptr(), l.v->data_ptr(), static_cast<float *>(l.g), static_cast<float *>(S->data_ptr()),
                                 o.data_ptr(), stream_of(l.dev));
    if (st != KDN_OK) return refused(st, "kdn_linear_decode_tokens");
    return THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

bool put(PyObject *d, const char *name, const at::Tensor &t) {
    PyObject *o = THPVariable_Wrap(t);
    const bool ok = o && PyDict_SetItemString(d, name, o) == 0;
    Py_XDECREF(o);
    return ok;
}

// linear_backward(q, k, v, g, d_o, cu_seqlens, S0, dS, scale, want_initial) -> dict
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Linear l;
    void *s0, *ds;
    if (n != 10 || !PyBool_Check(a[9]) || !l.read(a[0], a[1], a[2], a[3], a[5], a[8], 4) || !optional(a[6], at::kFloat, l.dev, l.states, &s0) ||
        !optional(a[7], at::kFloat, l.dev, l.states, &ds))
        Py_RETURN_NONE;
    const at::Tensor *d_o = tensor(a[4]);
    if (!d_o || !is(*d_o, l.v->scalar_type(), l.dev, l.v->sizes())) Py_RETURN_NONE;
    size_t need;
    if (kdn.linear_backward_workspace_size(&l.p, &need) != KDN_OK) Py_RETURN_NONE;
    at::Tensor dq = at::empty(l.q->sizes(), l.q->options()), dk = at::empty(l.q->sizes(), l.q->options()),
               dv = at::empty(l.v->sizes(), l.v->options()), dg, dS0;
    if (l.g) dg = floats(tensor(a[3])->sizes(), l.dev);
    if (a[9] == Py_True) dS0 = floats(l.states, l.dev);
    const at::Tensor ws = scratch(need, l.dev);
    const kdn_status_t st = kdn.linear_backward(&l.p, l.q->data_ptr(), l.k->data_ptr(), l.v->data_ptr(), static_cast<float *>(l.g), static_cast<float *>(s0),
                            d_o->data_ptr(), static_cast<float *>(ds), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                            dg.defined() ? static_cast<float *>(dg.data_ptr()) : nullptr,
                            dS0.defined() ? static_cast<float *>(dS0.data_ptr()) : nullptr, ws.data_ptr(), need,
                            stream_of(l.dev));
    if (st != KDN_OK) return refused(st, "kdn_linear_backward");
    PyObject *r = PyDict_New();
    if (r && put(r, "dq", dq) && put(r, "dk", dk) && put(r, "dv", dv) && (!dg.defined() || put(r, "dg", dg)) &&
        (!dS0.defined() || put(r, "dS0", dS0)))
        return r;
    Py_XDECREF(r);
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// x's rows: with a parameter [G, d] they are [..., G, d], else one group
struct Rows {
    const at::Tensor *x;
    long long n;
    int G, d, code;
    c10::Device dev = c10::Device(c10::kCPU);
    static constexpr int64_t most = 1 << 20;      // (the ABI's own limits are lower)
    bool read(PyObject *xo, const at::Tensor *param) {
        x = tensor(xo);
        if (!x || x->dim() < 1 || !elements(*x, &code)) return false;
        dev = x->device();
        if (!current(dev) || !is(*x, x->scalar_type(), dev) || x->size(-1) < 1 || x->size(-1) > most) return false;
        d = (int)x->size(-1);
        G = 1;
        if (param && param->dim() == 2) {
            if (x->dim() < 2 || param->size(0) != x->size(-2) || x->size(-2) < 1 || x->size(-2) > most) return false;
            G = (int)x->size(-2);
        }
        n = x->numel() / ((long long)G * d);
        return true;
    }
    bool parameter(const at::Tensor *t) const {
        if (!is(*t, at::kFloat, dev)) return false;
        return t->dim() == 2 ? t->size(0) == G && t->size(1) == d && x->dim() >= 2 && x->size(-2) == G : t->dim() == 1 && G == 1 && t->size(0) == d;
    }
};

// layer_norm(x, weight, bias, eps, y) -> (y, mean, rstd)
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    float eps;
    if (n != 5 || !number(a[3], &eps)) Py_RETURN_NONE;
    const at::Tensor *w = tensor(a[1]), *b = tensor(a[2]);
    if ((!w && a[1] != Py_None) || (!b && a[2] != Py_None)) Py_RETURN_NONE;
    Rows r;
    if (!r.read(a[0], w ? w : b) || (w && !r.parameter(w)) || (b && !r.parameter(b)) || (w && b && w->dim() != b->dim())) Py_RETURN_NONE;
    at::Tensor y;
    if (a[4] == Py_None) {
        y = at::empty(r.x->sizes(), r.x->options());
    } else {
        const at::Tensor *t = tensor(a[4]);
        if (!t || !is(*t, r.x->scalar_type(), r.dev, r.x->sizes())) Py_RETURN_NONE;
        y = *t;
    }
    const at::IntArrayRef rows = r.x->sizes().slice(0, r.x->dim() - 1);
    at::Tensor mean = floats(rows, r.dev), rstd = floats(rows, r.dev);
    const kdn_status_t st = kdn.layer_norm(r.n, r.G, r.d, (kdn_dtype_t)r.code, eps, r.x->data_ptr(), w ? static_cast<float *>(w->data_ptr()) : nullptr,
                       b ? static_cast<float *>(b->data_ptr()) : nullptr, y.data_ptr(), static_cast<float *>(mean.data_ptr()),
                       static_cast<float *>(rstd.data_ptr()), stream_of(r.dev));
    if (st != KDN_OK) return refused(st, "kdn_layer_norm");
    PyObject *t = PyTuple_New(3);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(y));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(mean));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(rstd));
    return t;
    END_HANDLE_TH_ERRORS
}

// layer_norm_backward(dy, x, weight, mean, rstd) -> dict
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor *dy = tensor(a[0]), *w = tensor(a[2]), *mean = tensor(a[3]), *rstd = tensor(a[4]);
    Rows r;
    if (!dy || (!w && a[2] != Py_None) || !mean || !rstd || !r.read(a[1], w) || (w && !r.parameter(w))) Py_RETURN_NONE;
    const at::IntArrayRef rows = r.x->sizes().slice(0, r.x->dim() - 1);
    if (!is(*dy, r.x->scalar_type(), r.dev, r.x->sizes()) || !is(*mean, at::kFloat, r.dev, rows) || !is(*rstd, at::kFloat, r.dev, rows))
        Py_RETURN_NONE;
    at::Tensor dx = at::empty(r.x->sizes(), r.x->options()), dw, db, ws;
    size_t need = 0;
    if (w) {
        if (kdn.layer_norm_backward_workspace_size(r.n, r.G, r.d, &need) != KDN_OK) Py_RETURN_NONE;
        dw = floats(w->sizes(), r.dev);
        db = floats(w->sizes(), r.dev);
        ws = scratch(need, r.dev);
    }
    const kdn_status_t st = kdn.layer_norm_backward(r.n, r.G, r.d, (kdn_dtype_t)r.code, dy->data_ptr(), r.x->data_ptr(),
                                w ? static_cast<float *>(w->data_ptr()) : nullptr, static_cast<float *>(mean->data_ptr()),
                                static_cast<float *>(rstd->data_ptr()), dx.data_ptr(), w ? static_cast<float *>(dw.data_ptr()) : nullptr,
                                w ? static_cast<float *>(db.data_ptr()) : nullptr, w ? ws.data_ptr() : nullptr, need,
                                stream_of(r.dev));
    if (st != KDN_OK) return refused(st, "kdn_layer_norm_backward");
    PyObject *d = PyDict_New();
    if (d && put(d, "dx", dx) && (!w || (put(d, "dweight", dw) && put(d, "dbias", db)))) return d;
    Py_XDECREF(d);
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the eight functions, in the order of `kdn`)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[8];
    if (n != 8 || sizeof(p) != sizeof(kdn)) {
        PyErr_SetString(PyExc_TypeError, "bind() takes eight addresses");
        return nullptr;
    }
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    memcpy(&kdn, p, sizeof(p));
    Py_RETURN_NONE;
}

// raise_with(type): the error that a failed call raises, made from (status, name of the function)
PyObject *raise_with(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 1 || !PyExceptionClass_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "raise_with() takes an exception type");
        return nullptr;
    }
    Py_XSETREF(error, Py_NewRef(a[0]));
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(raise_with), METHOD(linear_forward), METHOD(linear_decode), METHOD(linear_backward),
                         METHOD(layer_norm), METHOD(layer_norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kdn_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kdn_marshal() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "abi", KDN_MARSHAL_ABI) < 0) Py_CLEAR(m);   // the torch and interpreter it was built for
    return m;
}
