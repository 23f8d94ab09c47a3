// Argument marshalling of the layer operators (router by scores, microscaled
// formats, their product, RMSNorm) from torch tensors to the C ABI.
//
// A serving step makes these calls for a few microseconds of GPU work each;
// reading a tensor's pointer, sizes and strides from Python and converting them
// one by one for ctypes took 4 to 6 us a call, here it takes well under one.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gale.h"

namespace {

PyObject* g_error = nullptr;   // the package's GaleError(code, where)

PyObject* fail(int code, const char* where) {
    PyObject* e = PyObject_CallFunction(g_error, "is", code, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}
struct Refused {
    const char* why;
};

// A tensor argument, or none.
struct Arg {
    const at::Tensor* t = nullptr;
    void* data = nullptr;      // read with the tensor: a tensor without memory of its own raises
    explicit operator bool() const { return t != nullptr; }
    void* ptr() const { return data; }
    int64_t size(int i) const { return t->size(i); }
    int dtype() const {
        switch (t->scalar_type()) {
            case at::kFloat: return GALE_F32;
            case at::kBFloat16: return GALE_BF16;
            case at::kHalf: return GALE_F16;
            default: throw Refused{"float32, bfloat16 or float16"};
        }
    }
};

struct Call {
    int device = -1;      // of the first tensor; the others and the current device have to agree

    Arg tensor(PyObject* o, bool optional = false) {
        if (optional && o == Py_None) return Arg{};
        if (!THPVariable_Check(o)) throw Refused{"a tensor is missing"};
        Arg a;
        a.t = &THPVariable_Unpack(o);
        if (!a.t->defined() || a.t->layout() != at::kStrided) throw Refused{"a dense tensor"};
        // (a view that negates when read: its memory holds the other sign)
        if (a.t->is_neg()) throw Refused{"a tensor without a pending negation"};
        const int d = a.t->is_cuda() ? int(a.t->get_device()) : -2;
        if (device == -1) device = d;
        else if (device != d) throw Refused{"tensors on one device"};
        a.data = a.t->data_ptr();
        return a;
    }
    // [rows, cols] whose rows are contiguous: the row stride in elements
    static int64_t rows(const Arg& a, int64_t r, int64_t c) {
        if (a.t->dim() != 2 || a.size(0) != r || a.size(1) != c) throw Refused{"a tensor of another shape"};
        if (c > 1 && a.t->stride(1) != 1) throw Refused{"rows must be contiguous"};
        const int64_t ld = a.t->stride(0);
        return r > 1 || ld >= c ? ld : c;
    }
    static int64_t bytes(const Arg& a) {
        if (!a.t->is_contiguous()) throw Refused{"a contiguous buffer"};
        return int64_t(a.t->nbytes());
    }
    // a packed buffer that holds its layout
    static void room(const Arg& a, bool mx4, int64_t rows, int64_t cols) {
        gale_mx_layout_t L;
        if (rows == 0) return;
        if ((mx4 ? gale_mx4_layout(rows, cols, &L) : gale_mx8_layout(rows, cols, &L)) != GALE_OK) throw Refused{"sizes"};
        if (bytes(a) < L.s_offset + L.s_bytes) throw Refused{"packed buffer smaller than its layout"};
    }
    static void flat(const Arg& a, at::ScalarType type, int64_t n) {
        if (a.t->scalar_type() != type || a.t->numel() != n || !a.t->is_contiguous())
            throw Refused{"a contiguous tensor of another type or size"};
    }
    // the stream argument: none (the current one), a handle, or an object with cuda_stream
    void* stream(PyObject* o) const {
        if (device < 0) throw Refused{"tensors on a CUDA device"};
        if (device != int(c10::cuda::current_device())) throw Refused{"tensors on the current device"};
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream();
        if (PyLong_Check(o)) return handle(o);
        PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) {
            PyErr_Clear();
            throw Refused{"a stream"};
        }
        void* p = nullptr;
        const bool good = PyLong_Check(h);
        if (good) p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!good) throw Refused{"a stream"};
        return checked(p);
    }
    static void* handle(PyObject* o) { return checked(PyLong_AsVoidPtr(o)); }
    // no Python error may be left behind by a call that goes on
    static void* checked(void* p) {
        if (!p && PyErr_Occurred()) {
            PyErr_Clear();
            throw Refused{"a stream"};
        }
        return p;
    }
};

int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{"an integer"};
    }
    return v;
}
int whole32(PyObject* o) {
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{"an integer of 32 bits"};
    return int(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Refused{"a truth value"};
    }
    return v != 0;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{"a number"};
    }
    return float(v);
}

// Runs one call; refusals and status codes become GaleError.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t have, Py_ssize_t want, F f) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd expected", name, have, want);
        return nullptr;
    }
    try {
        const int rc = f();
        if (rc != GALE_OK) return fail(rc, name);
    } catch (const Refused& r) {
        char where[160];
        snprintf(where, sizeof where, "%s (%s)", name, r.why);
        return fail(GALE_ERR_ARG, where);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

// The library's call, with other Python threads running meanwhile (a full launch queue
// blocks).  `f` touches no Python object and no tensor; should it throw all the same, the
// exception is handled with the interpreter's lock held.
template <typename F>
int unlocked(F f) {
    struct Lock {
        PyThreadState* state = PyEval_SaveThread();
        ~Lock() { PyEval_RestoreThread(state); }
    } lock;
    return f();
}

PyObject* route_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("gale_route_select", n, 11, [&] {
        Call c;
        const Arg logits = c.tensor(a[0]), ids = c.tensor(a[1]), gates = c.tensor(a[2]), bias = c.tensor(a[3], true);
        if (logits.t->dim() != 2 || ids.t->dim() != 2 || ids.size(0) != logits.size(0))
            throw Refused{"logits [B, E], ids [B, K]"};
        const int64_t B = logits.size(0), E = logits.size(1), K = ids.size(1);
        if (B > INT32_MAX || E > INT32_MAX) throw Refused{"sizes"};
        const int64_t ld = Call::rows(logits, B, E);
        Call::rows(gates, B, K);
        Call::flat(ids, at::kInt, B * K);
        Call::flat(gates, at::kFloat, B * K);
        if (bias) Call::flat(bias, at::kFloat, E);
        const int dt = logits.dtype();
        const int score = whole32(a[4]), groups = whole32(a[5]), keep = whole32(a[6]), top = whole32(a[7]);
        const int renorm = truth(a[8]);
        const float scale = real(a[9]);
        void* s = c.stream(a[10]);
        return unlocked([&] {
            return gale_route_select(logits.ptr(), dt, ld, static_cast<const float*>(bias.ptr()), int(B), int(E), int(K),
                                     score, groups, keep, top, renorm, scale, static_cast<int32_t*>(ids.ptr()),
                                     static_cast<float*>(gates.ptr()), s);
        });
    });
}

PyObject* quantize(const char* name, bool mx4, PyObject* const* a, Py_ssize_t n) {
    return guarded(name, n, 3, [&] {
        Call c;
        const Arg x = c.tensor(a[0]), packed = c.tensor(a[1]);
        if (x.t->dim() != 2) throw Refused{"a [rows, cols] tensor"};
        const int64_t r = x.size(0), k = x.size(1), ld = Call::rows(x, r, k);
        Call::room(packed, mx4, r, k);
        const int dt = x.dtype();
        void* s = c.stream(a[2]);
        return unlocked([&] {
            return mx4 ? gale_mx4_quantize(x.ptr(), dt, ld, r, k, packed.ptr(), s)
                       : gale_mx8_quantize(x.ptr(), dt, ld, r, k, packed.ptr(), s);
        });
    });
}
PyObject* mx4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return quantize("gale_mx4_quantize", true, a, n); }
PyObject* mx8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return quantize("gale_mx8_quantize", false, a, n); }

PyObject* mx4_unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("gale_mx4_unpack", n, 3, [&] {
        Call c;
        const Arg packed = c.tensor(a[0]), out = c.tensor(a[1]);
        if (out.t->dim() != 2) throw Refused{"a [rows, cols] tensor"};
        const int64_t r = out.size(0), k = out.size(1), ld = Call::rows(out, r, k);
        Call::room(packed, true, r, k);
        const int dt = out.dtype();
        void* s = c.stream(a[2]);
        return unlocked([&] { return gale_mx4_unpack(packed.ptr(), r, k, out.ptr(), dt, ld, s); });
    });
}

PyObject* mx_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("gale_mx_gemm", n, 7, [&] {
        Call c;
        const Arg w4 = c.tensor(a[0]);
        const int64_t rows = whole(a[1]), cols = whole(a[2]);
        const Arg x8 = c.tensor(a[3]), y = c.tensor(a[4]), ws = c.tensor(a[5]);
        if (y.t->dim() != 2 || y.size(1) != rows) throw Refused{"y is [tokens, rows]"};
        const int64_t tokens = y.size(0), ldy = Call::rows(y, tokens, rows);
        Call::room(w4, true, rows, cols);
        Call::room(x8, false, tokens, cols);
        const int dt = y.dtype();
        const int64_t room = Call::bytes(ws);
        void* s = c.stream(a[6]);
        return unlocked([&] {
            return gale_mx_gemm(w4.ptr(), rows, cols, x8.ptr(), tokens, y.ptr(), dt, ldy, ws.ptr(), size_t(room), s);
        });
    });
}

PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("gale_rmsnorm", n, 8, [&] {
        Call c;
        const Arg x = c.tensor(a[0]), y = c.tensor(a[1], true), r = c.tensor(a[2], true), w = c.tensor(a[3], true),
                  h = c.tensor(a[4], true), q = c.tensor(a[5], true);
        if (x.t->dim() != 2) throw Refused{"x is [tokens, cols]"};
        const int64_t t = x.size(0), k = x.size(1), ldx = Call::rows(x, t, k);
        const int dt = x.dtype();
        if ((r && r.dtype() != dt) || (h && h.dtype() != dt)) throw Refused{"residual and sum_out have x's type"};
        if (w) Call::flat(w, w.t->scalar_type(), k);
        if (q) Call::room(q, false, t, k);
        const int64_t ldr = r ? Call::rows(r, t, k) : 0, ldh = h ? Call::rows(h, t, k) : 0, ldy = y ? Call::rows(y, t, k) : 0;
        const int wt = w ? w.dtype() : 0, yt = y ? y.dtype() : 0;
        const float eps = real(a[6]);
        void* s = c.stream(a[7]);
        return unlocked([&] {
            return gale_rmsnorm(x.ptr(), r.ptr(), dt, ldx, ldr, w.ptr(), wt, eps, t, k, h.ptr(), ldh, y.ptr(), yt, ldy,
                                q.ptr(), s);
        });
    });
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define FAST(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FAST(route_select), FAST(mx4_quantize), FAST(mx8_quantize), FAST(mx4_unpack), FAST(mx_gemm),
                         FAST(rmsnorm), {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
