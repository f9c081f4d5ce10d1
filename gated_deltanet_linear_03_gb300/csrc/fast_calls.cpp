// The Python binding's short way into the calls that are made for every layer of every generated token (ssm.py, linear.py): the
// checks and the marshalling of those modules in C++, for calls in which nothing is wrong and nothing unusual is asked for.
// A call of one token is a few microseconds of work on the GPU, less than Python needs to look its arguments over.
//
// Every function returns the output tensor, or None where it does not take the call: then the module's own code does, or says what
// is wrong with it.  Nothing has been launched in that case: a call that failed for another reason than its arguments raises
// GdnError here, since a kernel that updates states in place must not run twice.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <limits.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn.h"

namespace {

decltype(&gdn_short_conv) short_conv_fn;
decltype(&gdn_ssm_scan) scan_fn;
decltype(&gdn_ssm_scan_workspace_size) scan_workspace_fn;
decltype(&gdn_q4_linear) linear_fn;
decltype(&gdn_q4_gated) gated_fn;
decltype(&gdn_q4_workspace_size) q4_workspace_fn;
PyObject *error_type;

using at::ScalarType;

// What is looked at of a call's arguments; `fine` turns false at the first thing that is not as it should be.
struct Call {
    int device = -1;
    bool fine = true;

    const at::Tensor *tensor(PyObject *o, ScalarType type, int dim) {
        if (!THPVariable_Check(o)) return fail();
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.scalar_type() != type || t.dim() != dim) return fail();
        if (device < 0) device = t.get_device();
        return t.get_device() == device ? &t : fail();
    }
    const at::Tensor *dense(PyObject *o, ScalarType type, int dim) {
        const at::Tensor *t = tensor(o, type, dim);
        return t && t->is_contiguous() ? t : fail();
    }
    // An argument that may be None.
    const at::Tensor *optional(PyObject *o, ScalarType type, int dim) { return o == Py_None ? nullptr : dense(o, type, dim); }
    void want(bool b) { fine = fine && b; }
    const at::Tensor *fail() {
        fine = false;
        return nullptr;
    }
    // [tokens, width] with contiguous rows: their distance.
    long long rows(const at::Tensor *t, long long tokens, long long width) {
        if (!t) return 0;
        want(t->size(0) == tokens && t->size(1) == width && (t->stride(1) == 1 || width <= 1));
        return tokens > 1 ? t->stride(0) : width;
    }
    // An fp32 parameter for each channel.
    const float *per_channel(PyObject *o, long long channels) {
        const at::Tensor *t = optional(o, ScalarType::Float, 1);
        if (!t) return nullptr;
        want(t->size(0) == channels);
        return static_cast<const float *>(t->data_ptr());
    }
};

template <class T>
T *address(const at::Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }

int to_int(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    return v < 0 ? -1 : v > INT_MAX ? INT_MAX : (int)v;
}

bool in_int(long long v) { return v <= INT_MAX; }

// Sequences and their states [slots, d0, d1].
struct Sequences {
    int n = 0, n_slots = 0;
    const int32_t *cu = nullptr, *slots = nullptr;
    void *in = nullptr, *out = nullptr;
    Sequences(Call &c, PyObject *cu_obj, PyObject *slots_obj, PyObject *in_obj, PyObject *out_obj, ScalarType type, long long tokens,
              long long d0, long long d1) {
        const at::Tensor *t = c.optional(cu_obj, ScalarType::Int, 1);
        long long count = tokens;
        if (t) {
            count = t->size(0) - 1;
            cu = address<const int32_t>(t);
        }
        c.want(count >= 0 && in_int(count));
        n = (int)count;
        if ((t = c.optional(slots_obj, ScalarType::Int, 1))) {
            c.want(t->size(0) == count);
            slots = address<const int32_t>(t);
        }
        long long have = -1;
        for (PyObject *o : {in_obj, out_obj}) {
            if (!(t = c.optional(o, type, 3))) continue;
            c.want(t->size(1) == d0 && t->size(2) == d1 && in_int(t->size(0)) && (have < 0 || have == t->size(0)));
            have = t->size(0);
            (o == in_obj ? in : out) = t->data_ptr();
            if (in_obj == out_obj) in = out = t->data_ptr();
        }
        n_slots = have < 0 ? 0 : (int)have;
    }
};

// The tensor given for an output (of this shape, bf16 or fp32), or a new one of type `code`.
at::Tensor output(Call &c, PyObject *given, at::IntArrayRef shape, int &code) {
    if (given != Py_None) {
        if (!THPVariable_Check(given)) {
            c.fail();
            return {};
        }
        const at::Tensor &t = THPVariable_Unpack(given);
        code = t.scalar_type() == ScalarType::BFloat16 ? GDN_DTYPE_BF16 : t.scalar_type() == ScalarType::Float ? GDN_DTYPE_F32 : -1;
        c.want(code >= 0 && t.is_cuda() && t.get_device() == c.device && t.is_contiguous() && t.sizes() == shape);
        return t;
    }
    c.want(code == GDN_DTYPE_BF16 || code == GDN_DTYPE_F32);
    if (!c.fine) return {};
    return at::empty(shape, at::TensorOptions(code == GDN_DTYPE_F32 ? ScalarType::Float : ScalarType::BFloat16).device(at::kCUDA, c.device));
}

at::Tensor scratch(const Call &c, size_t bytes) {
    return at::empty({(long long)bytes}, at::TensorOptions(ScalarType::Byte).device(at::kCUDA, c.device));
}

// The library launches on the current device: another one is the module's business.
bool here(const Call &c) { return c.fine && c.device >= 0 && c10::cuda::current_device() == c.device; }

PyObject *answer(gdn_status st, const at::Tensor &out, const char *name) {
    if (st == GDN_OK) return THPVariable_Wrap(out);
    if (st == GDN_ERR_INVALID_ARG || st == GDN_ERR_UNSUPPORTED || st == GDN_ERR_ALIGNMENT || st == GDN_ERR_WORKSPACE) Py_RETURN_NONE;
    if (PyObject *e = PyObject_CallFunction(error_type, "is", (int)st, name)) {
        PyErr_SetObject(error_type, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// x, weight, cu_seqlens, bias, act, state_in, state_out, slots, out
PyObject *short_conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor *x = c.tensor(a[0], ScalarType::BFloat16, 2), *w = c.dense(a[1], ScalarType::Float, 2);
        if (!c.fine) Py_RETURN_NONE;
        const long long T = x->size(0), C = x->size(1), stride = c.rows(x, T, C), width = w->size(1);
        c.want(in_int(T) && in_int(C) && w->size(0) == C && width <= 4);
        const float *bias = c.per_channel(a[3], C);
        const Sequences s(c, a[2], a[7], a[5], a[6], ScalarType::BFloat16, T, width - 1, C);
        if (!here(c)) Py_RETURN_NONE;
        int code = GDN_DTYPE_BF16;
        const int64_t shape[] = {T, C};
        const at::Tensor out = output(c, a[8], shape, code);
        if (!c.fine || code != GDN_DTYPE_BF16) Py_RETURN_NONE;
        return answer(short_conv_fn(s.n, (int)T, (int)C, (int)width, x->data_ptr(), stride, address<const float>(w), bias, to_int(a[4]), s.cu,
                                    s.in, s.out, s.slots, s.n_slots, out.data_ptr(), c10::cuda::getCurrentCUDAStream(c.device).stream()), out, "gdn_short_conv");
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// x, dt, a, b, c, cu_seqlens, d, z, dt_bias, dt_softplus, state_in, state_out, slots, max_len, out, type of the output
PyObject *scan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 16) Py_RETURN_NONE;
    try {
        Call c;
        const at::Tensor *x = c.tensor(a[0], ScalarType::BFloat16, 2), *dt = c.tensor(a[1], ScalarType::BFloat16, 2);
        const at::Tensor *av = c.dense(a[2], ScalarType::Float, 2), *z = a[7] == Py_None ? nullptr : c.tensor(a[7], ScalarType::BFloat16, 2);
        const at::Tensor *b = c.tensor(a[3], ScalarType::BFloat16, 3), *cv = c.tensor(a[4], ScalarType::BFloat16, 3);
        if (!c.fine) Py_RETURN_NONE;
        const long long T = x->size(0), C = x->size(1), G = b->size(1), N = b->size(2);
        const long long xs = c.rows(x, T, C), ds = c.rows(dt, T, C), zs = c.rows(z, T, C);
        long long vs[2];
        for (int i = 0; i < 2; ++i) {
            const at::Tensor *t = i ? cv : b;
            c.want(t->size(0) == T && t->size(1) == G && t->size(2) == N && t->stride(2) == 1 && (G <= 1 || t->stride(1) == N));
            vs[i] = T > 1 ? t->stride(0) : G * N;
        }
        c.want(in_int(T) && in_int(C) && in_int(G) && in_int(N) && av->size(0) == C && av->size(1) == N);
        const float *skip = c.per_channel(a[6], C), *bias = c.per_channel(a[8], C);
        const Sequences s(c, a[5], a[12], a[10], a[11], ScalarType::Float, T, C, N);
        if (!here(c)) Py_RETURN_NONE;
        if (!PyBool_Check(a[9])) Py_RETURN_NONE;
        int code = to_int(a[15]), max_len = s.cu ? to_int(a[13]) : 1;
        if (max_len > T) max_len = (int)T;
        const int64_t shape[] = {T, C};
        const at::Tensor out = output(c, a[14], shape, code);
        if (!c.fine) Py_RETURN_NONE;
        size_t need = 0;
        at::Tensor work;
        if (s.cu) {
            gdn_status st = GDN_OK;
            need = scan_workspace_fn(s.n, (int)T, (int)C, (int)N, (int)G, max_len, &st);
            if (st != GDN_OK) Py_RETURN_NONE;
            if (need) work = scratch(c, need);
        }
        return answer(scan_fn(s.n, (int)T, (int)C, (int)N, (int)G, x->data_ptr(), xs, dt->data_ptr(), ds, address<const float>(av),
                              b->data_ptr(), vs[0], cv->data_ptr(), vs[1], skip, z ? z->data_ptr() : nullptr, zs, bias, a[9] == Py_True, s.cu, max_len,
                              static_cast<const float *>(s.in), static_cast<float *>(s.out), s.slots, s.n_slots, out.data_ptr(), code,
                              need ? work.data_ptr() : nullptr, need, c10::cuda::getCurrentCUDAStream(c.device).stream()), out, "gdn_ssm_scan");
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// A matrix in 4 bits: a tuple of codes, scales, offsets.
struct Matrix {
    const void *codes = nullptr, *scales = nullptr, *offsets = nullptr;
    long long n_out = 0, group = 0;
    Matrix(Call &c, PyObject *o, long long k) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
            c.fail();
            return;
        }
        const at::Tensor *q = c.dense(PyTuple_GET_ITEM(o, 0), ScalarType::Byte, 2), *s = c.dense(PyTuple_GET_ITEM(o, 1), ScalarType::BFloat16, 2);
        if (!c.fine) return;
        const long long groups = s->size(1);
        n_out = q->size(0);
        c.want(2 * q->size(1) == k && s->size(0) == n_out && groups > 0 && k % groups == 0 && in_int(n_out));
        if (!c.fine) return;
        group = k / groups;
        codes = q->data_ptr();
        scales = s->data_ptr();
        if (const at::Tensor *f = c.optional(PyTuple_GET_ITEM(o, 2), ScalarType::BFloat16, 2)) {
            c.want(f->sizes() == s->sizes());
            offsets = f->data_ptr();
        }
    }
};

// x, matrix (and the second one), act, out, type of the output
PyObject *q4(PyObject *const *a, bool gated) {
    try {
        Call c;
        if (!THPVariable_Check(a[0])) Py_RETURN_NONE;
        const at::Tensor &x = THPVariable_Unpack(a[0]);
        const int dim = (int)x.dim();
        if (!x.is_cuda() || x.scalar_type() != ScalarType::BFloat16 || dim < 1) Py_RETURN_NONE;
        c.device = x.get_device();
        const long long k = x.size(dim - 1);
        if (k <= 0 || !in_int(k)) Py_RETURN_NONE;
        const long long rows = x.numel() / k;
        const bool dense = x.is_contiguous();
        if (!in_int(rows) || (!dense && (dim != 2 || x.stride(1) != 1))) Py_RETURN_NONE;
        const long long stride = dense || rows <= 1 ? k : x.stride(0);
        const Matrix w(c, a[1], k), up = gated ? Matrix(c, a[2], k) : w;
        c.want(up.n_out == w.n_out && up.group == w.group && (up.offsets == nullptr) == (w.offsets == nullptr));
        if (!here(c)) Py_RETURN_NONE;
        at::DimVector shape(x.sizes().begin(), x.sizes().end());
        shape[dim - 1] = w.n_out;
        PyObject *const *rest = a + (gated ? 3 : 2);
        int code = to_int(rest[2]);
        const at::Tensor out = output(c, rest[1], shape, code);
        if (!c.fine) Py_RETURN_NONE;
        gdn_status st = GDN_OK;
        const size_t need = q4_workspace_fn((int)rows, (int)w.n_out, (int)k, (int)w.group, code, &st);
        if (st != GDN_OK) Py_RETURN_NONE;
        at::Tensor work;
        if (need) work = scratch(c, need);
        void *ws = need ? work.data_ptr() : nullptr, *stream = c10::cuda::getCurrentCUDAStream(c.device).stream();
        if (gated)
            st = gated_fn((int)rows, (int)w.n_out, (int)k, (int)w.group, x.data_ptr(), stride, w.codes, w.scales, w.offsets, up.codes, up.scales,
                          up.offsets, to_int(rest[0]), out.data_ptr(), code, ws, need, stream);
        else
            st = linear_fn((int)rows, (int)w.n_out, (int)k, (int)w.group, x.data_ptr(), stride, w.codes, w.scales, w.offsets, out.data_ptr(), code,
                           ws, need, stream);
        return answer(st, out, gated ? "gdn_q4_gated" : "gdn_q4_linear");
    } catch (...) {
        Py_RETURN_NONE;
    }
}

PyObject *q4_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) Py_RETURN_NONE;
    return q4(a, false);
}
PyObject *q4_gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) Py_RETURN_NONE;
    return q4(a, true);
}

// The addresses of the library's functions, in the order below, and GdnError.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *at[6];
    if (n != 7 || !PyExceptionClass_Check(a[6])) return PyErr_Format(PyExc_TypeError, "six addresses and an exception's class");
    for (int i = 0; i < 6; ++i)
        if (!(at[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "an address is null");
    short_conv_fn = reinterpret_cast<decltype(short_conv_fn)>(at[0]);
    scan_fn = reinterpret_cast<decltype(scan_fn)>(at[1]);
    scan_workspace_fn = reinterpret_cast<decltype(scan_workspace_fn)>(at[2]);
    linear_fn = reinterpret_cast<decltype(linear_fn)>(at[3]);
    gated_fn = reinterpret_cast<decltype(gated_fn)>(at[4]);
    q4_workspace_fn = reinterpret_cast<decltype(q4_workspace_fn)>(at[5]);
    Py_XSETREF(error_type, Py_NewRef(a[6]));
    Py_RETURN_NONE;
}

template <class F>
PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", method(bind), METH_FASTCALL, nullptr},
                         {"short_conv", method(short_conv), METH_FASTCALL, nullptr},
                         {"scan", method(scan), METH_FASTCALL, nullptr},
                         {"q4_linear", method(q4_linear), METH_FASTCALL, nullptr},
                         {"q4_gated", method(q4_gated), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
