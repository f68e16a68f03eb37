// Quick way from Python to the decode-layer operators: what layer.py does for a call of
// the usual form (plain tensors on one device, with rows), without a Python call for every
// shape, stride and pointer, which cost a small call more than its launch.
// Each function returns
//   None              the call is not of that form: layer.py checks it and says what is wrong,
//                     or makes the call itself;
//   an int            the status of a call that failed (gdn_status);
//   the result        otherwise.
// The checks that keep a call in bounds are the library's own, in both ways.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn.h"

namespace {

decltype(&gdn_recurrent_fwd) recurrent_fn;
decltype(&gdn_rows_int8) rows_fn;
decltype(&gdn_int8_matmul) matmul_fn;
decltype(&gdn_int8_matmul_workspace_bytes) matmul_workspace_fn;

// What a call's tensors have in common, and whether all of them fit so far.
struct Call {
    int device = -1;
    bool grad = c10::GradMode::is_enabled(), tangents = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    bool fits = true;

    // A plain tensor on the call's device, with `least` dimensions or more, contiguous in the last,
    // and no derivative asked of it (a tangent's level is 0, the only one there is).
    const at::Tensor *any(PyObject *o, int64_t least) {
        if (!fits || !THPVariable_CheckExact(o)) { fits = false; return nullptr; }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() < least || (t.dim() && t.stride(-1) != 1) || (grad && t.requires_grad()) ||
            (tangents && t._fw_grad(0).defined())) {
            fits = false;
            return nullptr;
        }
        if (device < 0) device = t.device().index();
        fits = device == t.device().index();
        return fits ? &t : nullptr;
    }
    // With `dims` dimensions.
    const at::Tensor *tensor(PyObject *o, int64_t dims) {
        const at::Tensor *t = any(o, dims);
        if (t && t->dim() != dims) { fits = false; t = nullptr; }
        return t;
    }
    const at::Tensor *tensor(PyObject *o, int64_t dims, at::ScalarType type) {
        const at::Tensor *t = tensor(o, dims);
        if (t && t->scalar_type() != type) { fits = false; t = nullptr; }
        return t;
    }
    const at::Tensor *maybe(PyObject *o, int64_t dims, at::ScalarType type) {
        return o == Py_None ? nullptr : tensor(o, dims, type);
    }
    void need(bool x) { fits = fits && x; }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
    at::TensorOptions options(at::ScalarType type) const {
        return at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device);
    }
};

bool is_io(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
int32_t code(at::ScalarType t) { return t == at::kBFloat16 ? GDN_BF16 : GDN_F32; }
template <typename T = void>
T *ptr(const at::Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
int64_t row(const at::Tensor *t) { return t ? t->stride(0) : 0; }

// A tensor seen as rows of its last `last` dimensions: their number, and their stride where they
// are one run, else the call is left to layer.py (as one of no rows is).
struct Rows {
    int64_t rows = 1, stride = 0;
    Rows(Call &c, const at::Tensor *t, int64_t last) {
        if (!t) return;
        int64_t next = -1;               // the stride that goes on with the run
        for (int64_t d = t->dim() - last - 1; d >= 0; --d) {
            const int64_t n = t->size(d);
            if (n == 1) continue;
            c.need(n > 0 && (next < 0 || t->stride(d) == next));
            if (next < 0) stride = t->stride(d);
            next = t->stride(d) * n;
            rows *= n;
        }
        c.need(rows <= INT32_MAX);
    }
};
at::IntArrayRef lead(const at::Tensor *t, int64_t last) { return t->sizes().slice(0, t->dim() - last); }
at::DimVector shape(at::IntArrayRef lead, int64_t width) {
    at::DimVector s(lead.begin(), lead.end());
    s.push_back(width);
    return s;
}
// A Python number (eps), else the call is left to layer.py.
double number(Call &c, PyObject *o) {
    c.need(PyFloat_CheckExact(o) || PyLong_CheckExact(o));
    if (!c.fits) return 0;
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) { PyErr_Clear(); c.fits = false; }     // a whole number past the range
    return x;
}

// A size that the structs hold, else the call is left to layer.py.
int32_t size(Call &c, int64_t n) {
    c.need(n >= 0 && n <= INT32_MAX);
    return (int32_t)n;
}

// Python's lock is free while a call allocates and launches: both may wait (for memory, or for a
// full queue), and other threads, host callbacks of the stream among them, go on meanwhile.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *none() { Py_RETURN_NONE; }

// (q, k, v, alpha, beta, state, slots, cu_seqlens, qk_norm_eps, o_dtype, out)
PyObject *recurrent_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11 || !(a[9] == Py_None || THPDtype_Check(a[9]))) return none();
    Call c;
    const at::Tensor *q = c.tensor(a[0], 3), *k = c.tensor(a[1], 3), *v = c.tensor(a[2], 3), *state = c.tensor(a[5], 4, at::kFloat);
    const at::Tensor *alpha = c.maybe(a[3], 2, at::kFloat), *beta = c.maybe(a[4], 2, at::kFloat);
    const at::Tensor *slots = c.maybe(a[6], 1, at::kInt), *cu = c.maybe(a[7], 1, at::kInt);
    const at::Tensor *out = a[10] == Py_None ? nullptr : c.tensor(a[10], 3);
    const double eps = a[8] == Py_None ? 0 : number(c, a[8]);
    if (!c.fits) return none();
    const at::ScalarType io = q->scalar_type();
    const at::ScalarType od = a[9] != Py_None ? reinterpret_cast<THPDtype *>(a[9])->scalar_type : out ? out->scalar_type() : io;
    const int64_t N = q->size(0), H = v->size(1), S = cu ? cu->size(0) - 1 : N;
    c.need(is_io(io) && is_io(od) && k->scalar_type() == io && v->scalar_type() == io && k->sizes() == q->sizes() && v->size(0) == N && S >= 0);
    c.need(state->size(1) == H && state->size(2) == q->size(2) && state->size(3) == v->size(2) && state->is_contiguous());
    c.need(!alpha || (alpha->size(0) == N && alpha->size(1) == H));
    c.need(!beta || (beta->size(0) == N && beta->size(1) == H));
    c.need(!slots || slots->size(0) == S);
    c.need(!out || (out->scalar_type() == od && out->sizes() == v->sizes() && out->is_contiguous()));
    gdn_recurrent_args g{};
    g.rows = size(c, N); g.seqs = size(c, S); g.H = size(c, H); g.Hk = size(c, q->size(1));
    g.dk = size(c, q->size(2)); g.dv = size(c, v->size(2)); g.pool = size(c, state->size(0));
    if (!c.fits) return none();
    g.io_dtype = code(io); g.o_dtype = code(od);
    g.qk_norm = a[8] != Py_None;
    g.qk_eps = (float)eps;
    g.q = ptr(q); g.k = ptr(k); g.v = ptr(v);
    g.q_row = q->stride(0); g.q_head = q->stride(1); g.k_row = k->stride(0); g.k_head = k->stride(1);
    g.v_row = v->stride(0); g.v_head = v->stride(1);
    g.alpha = ptr<float>(alpha); g.beta = ptr<float>(beta); g.alpha_row = row(alpha); g.beta_row = row(beta);
    g.cu_seqlens = ptr<int32_t>(cu); g.slots = ptr<int32_t>(slots); g.state = ptr<float>(state);
    at::Tensor made;
    gdn_status s;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
        if (!out) {
            made = cu ? at::zeros(v->sizes(), c.options(od)) : at::empty(v->sizes(), c.options(od));
            out = &made;
        }
        g.o = ptr(out);
        s = recurrent_fn(&g, c.stream());
    }
    if (s != GDN_OK) return PyLong_FromLong(s);
    if (!made.defined()) { Py_INCREF(a[10]); return a[10]; }
    return wrap(made);
    END_HANDLE_TH_ERRORS
}

// Rows of steps that start on 16 bytes, and their scales, and the call that fills them.
struct Steps {
    at::Tensor q, scale;
    gdn_status make(const Call &c, at::IntArrayRef lead, int64_t rows, int64_t width, gdn_rows_args &g) {
        const int64_t pitch = (width + 15) / 16 * 16;
        at::DimVector strides = shape(lead, 1);
        int64_t next = pitch;
        for (int64_t d = (int64_t)lead.size() - 1; d >= 0; --d) { strides[d] = next; next *= lead[d]; }
        q = at::empty_strided(shape(lead, width), strides, c.options(at::kChar));
        scale = at::empty(lead, c.options(at::kFloat));
        g.rows = (int32_t)rows; g.width = (int32_t)width;
        g.q = ptr<int8_t>(&q); g.q_row = pitch; g.scale = ptr<float>(&scale);
        return rows_fn(&g, c.stream());
    }
};
PyObject *pair_of(const Steps &y) {
    PyObject *t = PyTuple_New(2);
    if (t) { PyTuple_SET_ITEM(t, 0, wrap(y.q)); PyTuple_SET_ITEM(t, 1, wrap(y.scale)); }
    return t;
}

// (x)
PyObject *quantize_int8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 1) return none();
    Call c;
    const at::Tensor *x = c.any(a[0], 1);
    const Rows xr(c, x, 1);
    if (!c.fits) return none();
    c.need(is_io(x->scalar_type()));
    size(c, x->size(-1));
    if (!c.fits) return none();
    gdn_rows_args g{};
    g.op = GDN_ROWS_PLAIN; g.x_dtype = code(x->scalar_type()); g.x = ptr(x); g.x_row = xr.stride;
    Steps y;
    gdn_status s;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
        s = y.make(c, lead(x, 1), xr.rows, x->size(-1), g);
    }
    return s == GDN_OK ? pair_of(y) : PyLong_FromLong(s);
    END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, residual_out)
PyObject *add_rms_norm_int8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5 || (a[2] == Py_None && a[4] != Py_None)) return none();
    Call c;
    const at::Tensor *x = c.any(a[0], 1), *w = a[1] == Py_None ? nullptr : c.tensor(a[1], 1);
    const at::Tensor *r = a[2] == Py_None ? nullptr : c.any(a[2], 1), *out = a[4] == Py_None ? nullptr : c.any(a[4], 1);
    const Rows xr(c, x, 1), rr(c, r, 1), outr(c, out, 1);
    const double eps = number(c, a[3]);
    if (!c.fits) return none();
    const int64_t width = x->size(-1);
    c.need(is_io(x->scalar_type()) && (!w || (is_io(w->scalar_type()) && w->size(0) == width)));
    c.need(!r || (is_io(r->scalar_type()) && r->sizes() == x->sizes()));
    c.need(!out || (out->scalar_type() == r->scalar_type() && out->sizes() == x->sizes()));
    size(c, width);
    if (!c.fits) return none();
    gdn_rows_args g{};
    g.op = GDN_ROWS_NORM; g.eps = (float)eps;
    g.x_dtype = code(x->scalar_type()); g.x = ptr(x); g.x_row = xr.stride;
    if (w) { g.weight_dtype = code(w->scalar_type()); g.weight = ptr(w); }
    if (r) { g.residual_dtype = code(r->scalar_type()); g.residual = ptr(r); g.residual_row = rr.stride; }
    Steps y;
    at::Tensor made;
    gdn_status s;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
        if (r && !out) { made = at::empty(x->sizes(), c.options(r->scalar_type())); out = &made; }
        if (out) { g.residual_out = ptr(out); g.residual_out_row = made.defined() ? width : outr.stride; }
        s = y.make(c, lead(x, 1), xr.rows, width, g);
    }
    if (s != GDN_OK) return PyLong_FromLong(s);
    PyObject *t = PyTuple_New(3);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, wrap(y.q));
    PyTuple_SET_ITEM(t, 1, wrap(y.scale));
    PyObject *h = made.defined() ? wrap(made) : a[4];
    if (!made.defined()) Py_INCREF(h);
    PyTuple_SET_ITEM(t, 2, h);
    return t;
    END_HANDLE_TH_ERRORS
}

// (x, gate, weight, eps)
PyObject *gated_rms_norm_int8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 4) return none();
    Call c;
    const at::Tensor *x = c.any(a[0], 2), *gate = c.any(a[1], 2), *w = a[2] == Py_None ? nullptr : c.tensor(a[2], 1);
    const Rows xr(c, x, 2), gr(c, gate, 2);
    const double eps = number(c, a[3]);
    if (!c.fits) return none();
    const int64_t H = x->size(-2), d = x->size(-1);
    c.need(is_io(x->scalar_type()) && gate->scalar_type() == x->scalar_type() && gate->sizes() == x->sizes());
    c.need(!w || (is_io(w->scalar_type()) && w->size(0) == d));
    c.need((x->stride(-2) == d && gate->stride(-2) == d) || H == 1);
    size(c, H * d); size(c, d);
    if (!c.fits) return none();
    gdn_rows_args g{};
    g.op = GDN_ROWS_GATED; g.head = (int32_t)d; g.eps = (float)eps;
    g.x_dtype = code(x->scalar_type()); g.x = ptr(x); g.x_row = xr.stride;
    g.gate = ptr(gate); g.gate_row = gr.stride;
    if (w) { g.weight_dtype = code(w->scalar_type()); g.weight = ptr(w); }
    Steps y;
    gdn_status s;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
        s = y.make(c, lead(x, 2), xr.rows, H * d, g);
    }
    return s == GDN_OK ? pair_of(y) : PyLong_FromLong(s);
    END_HANDLE_TH_ERRORS
}

// (x, x_scale, w, w_scale, bias, out_dtype, out)
PyObject *int8_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7 || !THPDtype_Check(a[5])) return none();
    Call c;
    const at::Tensor *x = c.any(a[0], 1), *xs = c.any(a[1], 0), *w = c.tensor(a[2], 2, at::kChar), *ws = c.tensor(a[3], 1, at::kFloat);
    const at::Tensor *bias = c.maybe(a[4], 1, at::kFloat), *out = a[6] == Py_None ? nullptr : c.any(a[6], 1);
    const at::ScalarType od = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
    const Rows xr(c, x, 1), outr(c, out, 1);
    if (!c.fits) return none();
    const int64_t K = x->size(-1), N = w->size(0);
    c.need(x->scalar_type() == at::kChar && xs->scalar_type() == at::kFloat && xs->sizes() == lead(x, 1) && xs->is_contiguous());
    c.need(is_io(od) && w->size(1) == K && ws->size(0) == N && (!bias || bias->size(0) == N));
    c.need(!out || (out->scalar_type() == od && out->size(-1) == N && lead(out, 1) == lead(x, 1)));
    gdn_int8_matmul_args g{};
    g.M = (int32_t)xr.rows; g.N = size(c, N); g.K = size(c, K);
    if (!c.fits) return none();
    g.out_dtype = code(od);
    g.x = ptr<int8_t>(x); g.w = ptr<int8_t>(w); g.x_row = xr.stride; g.w_row = row(w);
    g.x_scale = ptr<float>(xs); g.w_scale = ptr<float>(ws); g.bias = ptr<float>(bias);
    at::Tensor made, workspace;
    gdn_status s;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
        if (!out) { made = at::empty(shape(lead(x, 1), N), c.options(od)); out = &made; }
        g.out = ptr(out); g.out_row = made.defined() ? N : outr.stride;
        g.workspace_bytes = matmul_workspace_fn(&g);
        if (g.workspace_bytes) {     // not kept: a call's copies belong to its stream, or its graph
            workspace = at::empty({(int64_t)g.workspace_bytes}, c.options(at::kByte));
            g.workspace = workspace.data_ptr();
        }
        s = matmul_fn(&g, c.stream());
    }
    if (s != GDN_OK) return PyLong_FromLong(s);
    if (!made.defined()) { Py_INCREF(a[6]); return a[6]; }
    return wrap(made);
    END_HANDLE_TH_ERRORS
}

// (addresses of gdn_recurrent_fwd, gdn_rows_int8, gdn_int8_matmul, gdn_int8_matmul_workspace_bytes, GDN_ABI_VERSION
// of the library)
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long f[4];
    int abi;
    if (!PyArg_ParseTuple(args, "KKKKi", f, f + 1, f + 2, f + 3, &abi)) return nullptr;
    if (abi != GDN_ABI_VERSION) {
        PyErr_Format(PyExc_RuntimeError, "built for ABI %d, the library has %d", GDN_ABI_VERSION, abi);
        return nullptr;
    }
    recurrent_fn = reinterpret_cast<decltype(recurrent_fn)>(f[0]);
    rows_fn = reinterpret_cast<decltype(rows_fn)>(f[1]);
    matmul_fn = reinterpret_cast<decltype(matmul_fn)>(f[2]);
    matmul_workspace_fn = reinterpret_cast<decltype(matmul_workspace_fn)>(f[3]);
    return none();
}

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"recurrent_fwd", (PyCFunction)(void (*)())recurrent_fwd, METH_FASTCALL, nullptr},
                         {"quantize_int8", (PyCFunction)(void (*)())quantize_int8, METH_FASTCALL, nullptr},
                         {"add_rms_norm_int8", (PyCFunction)(void (*)())add_rms_norm_int8, METH_FASTCALL, nullptr},
                         {"gated_rms_norm_int8", (PyCFunction)(void (*)())gated_rms_norm_int8, METH_FASTCALL, nullptr},
                         {"int8_matmul", (PyCFunction)(void (*)())int8_matmul, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "Quick way to the decode-layer operators (layer.py).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Nothing of torch is touched before layer.py has compared built_for with the torch that is there.
PyMODINIT_FUNC PyInit__layer() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", GDN_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
