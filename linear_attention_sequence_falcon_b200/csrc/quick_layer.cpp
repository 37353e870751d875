// quick_layer.cpp -- the short way into the layer operators (module _quick).
//
// Behind a decode step's calls stand kernels of 2-3 us; checked and bound in
// Python (layer.py, ctypes) a call takes 10-20 us.  The functions here take the
// same arguments by position, make the same checks and the same call of
// include/falcon.h on torch's current stream.  Whatever is not as the checks
// want it (another device, a wrong shape, dtype or stride, an error of the
// call) they answer with None, before anything is enqueued or after an error
// that enqueued nothing, and layer.py goes its own way, which refuses it with
// words or handles it.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/falcon.h"

namespace {

using at::Tensor;

// What the tensors of one call share.
struct Call {
    bool ok = true;
    at::ScalarType type = at::kFloat;
    int device = -1;
    at::TensorOptions options;

    // the first argument: its dtype, its device, which has to be the current one
    const Tensor *first(PyObject *o) {
        const Tensor *t = required(o);
        if (!ok) return nullptr;
        type = t->scalar_type();
        device = t->is_cuda() && t->layout() == at::kStrided ? t->get_device() : -1;
        ok = (type == at::kFloat || type == at::kBFloat16) && device >= 0 && device == c10::cuda::current_device();
        options = t->options();
        return t;
    }
    const Tensor *required(PyObject *o) {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    const Tensor *optional(PyObject *o) { return o == Py_None ? nullptr : required(o); }
    falcon_dtype dtype() const { return type == at::kBFloat16 ? FALCON_BF16 : FALCON_F32; }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }

    void like(const Tensor *t, at::IntArrayRef shape, at::ScalarType want) {
        if (ok && t) ok = t->scalar_type() == want && t->is_cuda() && t->layout() == at::kStrided && t->get_device() == device && t->sizes() == shape;
    }
    // a contiguous array (or none)
    void need(const Tensor *t, at::IntArrayRef shape, at::ScalarType want) {
        like(t, shape, want);
        if (ok && t) ok = t->is_contiguous();
    }
    // rows: the stride from token to token of [n, D] or [n, L, D]
    long long rows(const Tensor *t, at::IntArrayRef shape) {
        like(t, shape, type);
        if (!ok || !t) return 0;
        const auto st = t->strides();
        const int64_t D = shape.back(), n = shape[0];
        int64_t step = st[0];
        if (st.back() != 1 && D > 1) ok = false;
        if (shape.size() == 3 && shape[1] > 1) {
            step = st[1];
            if (n > 1 && st[0] != step * shape[1]) ok = false;
        } else if (n <= 1) {
            return D;
        }
        if (step < D) ok = false;
        return step;
    }
    // sizes fit the library's int arguments
    void sizes(at::IntArrayRef s) {
        for (const int64_t n : s)
            if (n > 0x7fffffff) ok = false;
    }
    Tensor empty(at::IntArrayRef shape) const { return at::empty(shape, options); }
    Tensor empty_f32(at::IntArrayRef shape) const { return at::empty(shape, options.dtype(at::kFloat)); }
};

bool truth(PyObject *o) { return PyObject_IsTrue(o) == 1; }
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
float *f32(const Tensor *t) { return t ? static_cast<float *>(t->data_ptr()) : nullptr; }

// new references; None for no tensor
PyObject *object(const Tensor *t, PyObject *given) {
    if (given && given != Py_None) return Py_NewRef(given);
    if (!t || !t->defined()) return Py_NewRef(Py_None);
    return THPVariable_Wrap(*t);
}

PyObject *tuple(std::initializer_list<PyObject *> items) {
    PyObject *r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (r) PyTuple_SET_ITEM(r, i++, o);
        else Py_XDECREF(o);
    }
    return r;
}

// the result, unless a conversion failed (out of memory)
PyObject *checked(PyObject *r) {
    if (PyErr_Occurred()) {
        Py_XDECREF(r);
        return nullptr;
    }
    return r;
}

// The library's call with Python's lock released, as ctypes makes it: a launch
// waits where the device's queue is full, and other threads run meanwhile (the
// one among them that the queue waits for, where a host function needs the lock).
class Unlock {
    PyThreadState *const state_ = PyEval_SaveThread();

public:
    ~Unlock() { PyEval_RestoreThread(state_); }
};
template <typename... P, typename... A> int unlocked(int (*call)(P...), A... args) {
    const Unlock held;
    return call(args...);
}

#define ARGUMENTS(count)                                                        \
    if (n != (count)) {                                                         \
        PyErr_SetString(PyExc_TypeError, "_quick: wrong number of arguments");  \
        return nullptr;                                                         \
    }                                                                           \
    at::AutoDispatchBelowADInplaceOrView no_autograd;                           \
    Call c
#define ELSEWHERE Py_RETURN_NONE

// scan(x, f, reset, initial_state, out, final_state, marks, want_state, want_marks) -> (out, final_state, marks)
PyObject *scan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(9);
    const Tensor *x = c.first(a[0]);
    if (!c.ok || x->dim() != 3) ELSEWHERE;
    const auto shape = x->sizes();
    const int64_t N = shape[0], L = shape[1], D = shape[2], blocks = (L + FALCON_SCAN_BLOCK - 1) / FALCON_SCAN_BLOCK;
    c.sizes(shape);
    const Tensor *f = c.required(a[1]), *reset = c.optional(a[2]), *init = c.optional(a[3]), *out = c.optional(a[4]),
                 *last = c.optional(a[5]), *marks = c.optional(a[6]);
    if (!c.ok) ELSEWHERE;
    const long long ldx = c.rows(x, shape), ldf = c.rows(f, shape);
    if (reset && reset->scalar_type() != at::kBool && reset->scalar_type() != at::kByte) ELSEWHERE;
    if (reset) c.need(reset, {N, L}, reset->scalar_type());
    c.need(init, {N, D}, at::kFloat);
    c.need(last, {N, D}, at::kFloat);
    c.need(out, shape, c.type);
    c.need(marks, {N, blocks, D}, at::kFloat);
    if (!c.ok) ELSEWHERE;
    Tensor new_out, new_last, new_marks;
    if (!out) new_out = c.empty(shape), out = &new_out;
    if (!last && truth(a[7])) new_last = c.empty_f32({N, D}), last = &new_last;
    if (!marks && truth(a[8])) new_marks = c.empty_f32({N, blocks, D}), marks = &new_marks;
    if (unlocked(falcon_scan, c.dtype(), ptr(x), ptr(f), static_cast<const unsigned char *>(ptr(reset)), f32(init), (int)N,
                 (int)L, (int)D, ldx, ldf, ptr(out), f32(last), f32(marks), c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(tuple({object(out, a[4]), object(last, a[5]), object(marks, a[6])}));
    END_HANDLE_TH_ERRORS
}

// scan_bwd(x, f, dout, dstate, reset, initial_state, marks, dx, df, workspace) -> (dx, df, dinitial)
PyObject *scan_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(10);
    const Tensor *x = c.first(a[0]);
    if (!c.ok || x->dim() != 3 || a[9] != Py_None) ELSEWHERE;
    const auto shape = x->sizes();
    const int64_t N = shape[0], L = shape[1], D = shape[2], blocks = (L + FALCON_SCAN_BLOCK - 1) / FALCON_SCAN_BLOCK;
    c.sizes(shape);
    const Tensor *f = c.required(a[1]), *dout = c.required(a[2]), *dstate = c.optional(a[3]), *reset = c.optional(a[4]),
                 *init = c.optional(a[5]), *marks = c.optional(a[6]), *dx = c.optional(a[7]), *df = c.optional(a[8]);
    if (!c.ok) ELSEWHERE;
    const long long ldx = c.rows(x, shape), ldf = c.rows(f, shape);
    const long long lddx = dx ? c.rows(dx, shape) : D, lddf = df ? c.rows(df, shape) : D;
    if (reset && reset->scalar_type() != at::kBool && reset->scalar_type() != at::kByte) ELSEWHERE;
    if (reset) c.need(reset, {N, L}, reset->scalar_type());
    c.need(dout, shape, c.type);
    c.need(dstate, {N, D}, at::kFloat);
    c.need(init, {N, D}, at::kFloat);
    c.need(marks, {N, blocks, D}, at::kFloat);
    if (!c.ok) ELSEWHERE;
    size_t bytes = 0;
    if (falcon_scan_bwd_workspace_size(c.dtype(), (int)N, (int)L, (int)D, marks != nullptr, &bytes) != FALCON_OK) ELSEWHERE;
    Tensor new_dx, new_df, ws;
    if (!dx) new_dx = c.empty(shape), dx = &new_dx;
    if (!df) new_df = c.empty(shape), df = &new_df;
    const Tensor dinitial = c.empty_f32({N, D});
    if (bytes) ws = c.empty_f32({(int64_t)(bytes + 3) / 4});
    if (unlocked(falcon_scan_bwd_ws, c.dtype(), ptr(x), ptr(f), static_cast<const unsigned char *>(ptr(reset)), f32(init),
                 f32(marks), (int)N, (int)L, (int)D, ldx, ldf, ptr(dout), f32(dstate), ptr(dx), lddx, ptr(df), lddf,
                 f32(&dinitial), bytes ? ws.data_ptr() : nullptr, bytes, c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(tuple({object(dx, a[7]), object(df, a[8]), object(&dinitial, nullptr)}));
    END_HANDLE_TH_ERRORS
}

// scan_step(x, f, state, state_out, out) -> (out, state_out)
PyObject *scan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(5);
    const Tensor *x = c.first(a[0]);
    if (!c.ok || x->dim() != 2) ELSEWHERE;
    const auto shape = x->sizes();
    c.sizes(shape);
    const Tensor *f = c.required(a[1]), *state = c.required(a[2]), *next = c.optional(a[3]), *out = c.optional(a[4]);
    if (!c.ok) ELSEWHERE;
    const long long ldx = c.rows(x, shape), ldf = c.rows(f, shape);
    c.need(state, shape, at::kFloat);
    c.need(next, shape, at::kFloat);
    c.need(out, shape, c.type);
    if (!c.ok) ELSEWHERE;
    Tensor new_out;
    if (!out) new_out = c.empty(shape), out = &new_out;
    if (unlocked(falcon_scan_step, c.dtype(), ptr(x), ptr(f), f32(state), (int)shape[0], (int)shape[1], ldx, ldf,
                 f32(next ? next : state), ptr(out), c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(tuple({object(out, a[4]), Py_NewRef(next ? a[3] : a[2])}));
    END_HANDLE_TH_ERRORS
}

// the shapes of the gated norm's arrays; eps from its argument
struct Gate {
    const Tensor *o = nullptr, *gate = nullptr, *weight = nullptr;
    int64_t B = 0, H = 0, L = 0, d = 0, wide = 0;
    long long ldg = 0;
    float eps = 0.f;
    int per_head = 0;

    void begin(Call &c, PyObject *po, PyObject *pg, PyObject *pw, PyObject *pe) {
        o = c.first(po);
        c.ok = c.ok && o->dim() == 4;
        if (!c.ok) return;
        c.sizes(o->sizes());
        B = o->size(0), H = o->size(1), L = o->size(2), d = o->size(3), wide = H * d;
        ldg = wide;
        if (d < 1 || d > FALCON_NORM_MAX_D || (d > 1 && o->stride(3) != 1)) c.ok = false;
        gate = c.optional(pg);
        weight = c.optional(pw);
        const double e = PyFloat_AsDouble(pe);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            c.ok = false;
        }
        if (!c.ok || !(e >= 0.0)) {
            c.ok = false;
            return;
        }
        eps = (float)e;
        if (gate) ldg = c.rows(gate, {B, L, wide});
        per_head = weight && weight->dim() == 2;
        if (per_head) c.need(weight, {H, d}, at::kFloat);
        else c.need(weight, {d}, at::kFloat);
    }
};

// norm_gate(o, gate, weight, eps, out) -> out
PyObject *norm_gate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(5);
    Gate g;
    g.begin(c, a[0], a[1], a[2], a[3]);
    const Tensor *out = c.ok ? c.optional(a[4]) : nullptr;
    c.need(out, {g.B, g.L, g.wide}, c.type);
    if (!c.ok) ELSEWHERE;
    Tensor new_out;
    if (!out) new_out = c.empty({g.B, g.L, g.wide}), out = &new_out;
    if (unlocked(falcon_norm_gate, c.dtype(), ptr(g.o), g.o->stride(0), g.o->stride(1), g.o->stride(2), ptr(g.gate),
                 g.ldg, f32(g.weight), g.per_head, g.eps, (int)g.B, (int)g.H, (int)g.L, (int)g.d, ptr(out), c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(object(out, a[4]));
    END_HANDLE_TH_ERRORS
}

// norm_gate_bwd(o, gate, weight, eps, dout, want_dweight) -> (do, dgate, dweight)
PyObject *norm_gate_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(6);
    Gate g;
    g.begin(c, a[0], a[1], a[2], a[3]);
    const Tensor *dout = c.ok ? c.required(a[4]) : nullptr;
    c.need(dout, {g.B, g.L, g.wide}, c.type);
    if (!c.ok) ELSEWHERE;
    size_t bytes = 0;
    if (falcon_norm_gate_bwd_workspace_size(c.dtype(), (int)g.B, (int)g.H, (int)g.L, (int)g.d, &bytes) != FALCON_OK)
        ELSEWHERE;
    const Tensor d_o = c.empty({g.B, g.H, g.L, g.d});
    Tensor dgate, dweight, ws;
    if (g.gate) dgate = c.empty({g.B, g.L, g.wide});
    if (g.weight && truth(a[5])) dweight = c.empty_f32(g.weight->sizes());
    if (bytes) ws = c.empty_f32({(int64_t)(bytes + 3) / 4});
    if (unlocked(falcon_norm_gate_bwd_ws, c.dtype(), ptr(g.o), g.o->stride(0), g.o->stride(1), g.o->stride(2), ptr(g.gate),
                 g.ldg, f32(g.weight), g.per_head, g.eps, (int)g.B, (int)g.H, (int)g.L, (int)g.d, ptr(dout), d_o.data_ptr(),
                 d_o.stride(0), d_o.stride(1), d_o.stride(2), dgate.defined() ? dgate.data_ptr() : nullptr, g.wide,
                 dweight.defined() ? f32(&dweight) : nullptr, bytes ? ws.data_ptr() : nullptr, bytes, c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(tuple({object(&d_o, nullptr), object(&dgate, nullptr), object(&dweight, nullptr)}));
    END_HANDLE_TH_ERRORS
}

// the shapes of the residual norm's arrays
struct Residual {
    const Tensor *r = nullptr, *y = nullptr, *scale = nullptr, *weight = nullptr;
    int64_t R = 0, D = 0;
    float eps = 0.f;

    void begin(Call &c, PyObject *pr, PyObject *pw, PyObject *pe, PyObject *py, PyObject *ps) {
        r = c.first(pr);
        c.ok = c.ok && r->dim() >= 1;
        if (!c.ok) return;
        D = r->size(-1);
        if (D < 1 || D > FALCON_NORM_MAX_D) {
            c.ok = false;
            return;
        }
        R = r->numel() / D;
        c.sizes({R});
        weight = c.optional(pw);
        y = c.optional(py);
        scale = c.optional(ps);
        const double e = PyFloat_AsDouble(pe);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            c.ok = false;
        }
        if (!c.ok || !(e >= 0.0) || (scale && !y)) {
            c.ok = false;
            return;
        }
        eps = (float)e;
        c.need(r, r->sizes(), c.type);
        c.need(y, r->sizes(), c.type);
        c.need(scale, {D}, at::kFloat);
        c.need(weight, {D}, at::kFloat);
    }
};

// residual_norm(r, weight, eps, y, scale) -> (r_out, h)
PyObject *residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(5);
    Residual g;
    g.begin(c, a[0], a[1], a[2], a[3], a[4]);
    if (!c.ok) ELSEWHERE;
    const Tensor h = c.empty(g.r->sizes());
    Tensor stream;
    if (g.y) stream = c.empty(g.r->sizes());
    if (unlocked(falcon_residual_norm, c.dtype(), ptr(g.r), ptr(g.y), f32(g.scale), f32(g.weight), g.eps, (int)g.R,
                 (int)g.D, g.y ? stream.data_ptr() : nullptr, h.data_ptr(), c.stream()) != FALCON_OK)
        ELSEWHERE;
    return checked(tuple({object(&stream, g.y ? nullptr : a[0]), object(&h, nullptr)}));
    END_HANDLE_TH_ERRORS
}

// residual_norm_bwd(r_out, weight, eps, dh, dr_out, y, scale) -> (dr, dy, dscale, dweight)
PyObject *residual_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ARGUMENTS(7);
    Residual g;
    g.begin(c, a[0], a[1], a[2], a[5], a[6]);
    if (!c.ok) ELSEWHERE;
    const Tensor *dh = c.required(a[3]), *dr_out = c.optional(a[4]);
    c.need(dh, g.r->sizes(), c.type);
    c.need(dr_out, g.r->sizes(), c.type);
    if (!c.ok) ELSEWHERE;
    size_t bytes = 0;
    if (falcon_residual_norm_bwd_workspace_size(c.dtype(), (int)g.R, (int)g.D, &bytes) != FALCON_OK) ELSEWHERE;
    const Tensor dr = c.empty(g.r->sizes());
    Tensor dy, dscale, dweight, ws;
    if (g.scale) dy = c.empty(g.r->sizes()), dscale = c.empty_f32({g.D});
    if (g.weight) dweight = c.empty_f32({g.D});
    if (bytes) ws = c.empty_f32({(int64_t)(bytes + 3) / 4});
    if (unlocked(falcon_residual_norm_bwd_ws, c.dtype(), ptr(g.r), ptr(g.y), f32(g.scale), f32(g.weight), ptr(dh),
                 ptr(dr_out), g.eps, (int)g.R, (int)g.D, dr.data_ptr(), g.scale ? dy.data_ptr() : nullptr,
                 g.scale ? f32(&dscale) : nullptr, g.weight ? f32(&dweight) : nullptr, bytes ? ws.data_ptr() : nullptr,
                 bytes, c.stream()) != FALCON_OK)
        ELSEWHERE;
    PyObject *first = object(&dr, nullptr);
    PyObject *second = g.scale ? object(&dy, nullptr) : Py_NewRef(g.y && first ? first : Py_None);
    return checked(tuple({first, second, object(&dscale, nullptr), object(&dweight, nullptr)}));
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(scan),          METHOD(scan_bwd),      METHOD(scan_step),
                         METHOD(norm_gate),     METHOD(norm_gate_bwd), METHOD(residual_norm),
                         METHOD(residual_norm_bwd), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick", "The short way into the layer operators (layer.py).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick() { return PyModule_Create(&module); }
