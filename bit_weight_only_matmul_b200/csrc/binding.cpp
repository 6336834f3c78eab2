// binding.cpp -- the Python binding's checks and argument marshalling for the
// MXFP4 operators and the block norm, as a CPython extension module.
//
// A decode step makes many calls of a few microseconds of GPU time each; the
// same checks written in Python over ctypes took 2.0 us of a
// quantize call and 4.9 us of a block norm's, longer than the launch.  Nothing
// here touches CUDA: each function checks its tensors, finds the stream and
// calls the C entry point of its name; the Python functions around it carry
// the documentation and raise on a status.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxfp4.h"

namespace {

// Types an operand may have, as a mask over Q4_TYPE_*.
constexpr int kF32 = 1 << Q4_TYPE_F32, kBF16 = 1 << Q4_TYPE_BF16, kF16 = 1 << Q4_TYPE_F16, kBytes = 1 << Q4_TYPE_MXFP4;

PyObject *g_get_device = nullptr, *g_get_stream = nullptr;   // torch._C's functions
PyObject *g_cuda_stream = nullptr;                           // the attribute's name

int type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return Q4_TYPE_F32;
        case at::kBFloat16: return Q4_TYPE_BF16;
        case at::kHalf: return Q4_TYPE_F16;
        case at::kByte: return Q4_TYPE_MXFP4;
        default: return -1;
    }
}

// The arguments of one call: the first thing that is wrong sets a Python
// exception, and what is asked after that does nothing.
class Call {
  public:
    bool ok() const { return ok_; }

    int64_t number(PyObject *o) {
        if (!ok_) return 0;
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) ok_ = false;
        return v;
    }
    float real(PyObject *o) {
        if (!ok_) return 0.f;
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) ok_ = false;
        return static_cast<float>(v);
    }

    // A contiguous tensor on the current device, of one of `types`, with at
    // least rows * cols elements (sizes below zero are the library's to refuse).
    void *tensor(PyObject *o, const char *what, int types, int64_t rows, int64_t cols, int *type = nullptr) {
        const at::Tensor *t = checked(o, what, types, type);
        if (!t) return nullptr;
        return sized(*t, what, rows > 0 && cols > 0 ? static_cast<__int128>(rows) * cols : 0);
    }
    // The same for an MXFP4 matrix of R rows by K values.
    void *matrix(PyObject *o, const char *what, int64_t R, int64_t K) {
        const at::Tensor *t = checked(o, what, kBytes, nullptr);
        if (!t) return nullptr;
        const __int128 tiles = R > 0 && K > 0 ? static_cast<__int128>((R + 127) / 128) * ((K + 255) / 256) : 0;
        return sized(*t, what, tiles * 17408);
    }
    // x of the block norm: values, or an MXFP4 matrix.
    void *values_or_matrix(PyObject *o, const char *what, int64_t rows, int64_t cols, int *type) {
        if (!ok_) return nullptr;
        if (THPVariable_Check(o) && type_of(THPVariable_Unpack(o)) == Q4_TYPE_MXFP4) {
            *type = Q4_TYPE_MXFP4;
            return matrix(o, what, rows, cols);
        }
        return tensor(o, what, kF32 | kBF16, rows, cols, type);
    }

    // None: the current stream of the current device; an address; or an object
    // with one.
    q4_0_stream_t stream(PyObject *o) {
        if (!ok_) return nullptr;
        PyObject *v;
        if (o == Py_None) {
            if (device_ < 0 && !find_device()) return nullptr;
            PyObject *d = PyLong_FromLong(device_);
            v = d ? PyObject_CallOneArg(g_get_stream, d) : nullptr;
            Py_XDECREF(d);
        } else if (PyLong_Check(o)) {
            v = Py_NewRef(o);
        } else {
            v = PyObject_GetAttr(o, g_cuda_stream);
        }
        void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
        Py_XDECREF(v);
        if (PyErr_Occurred()) ok_ = false;
        return static_cast<q4_0_stream_t>(p);
    }

  private:
    bool find_device() {
        PyObject *d = PyObject_CallNoArgs(g_get_device);
        if (d) {
            device_ = PyLong_AsLong(d);
            Py_DECREF(d);
        }
        if (PyErr_Occurred()) ok_ = false;
        return ok_;
    }
    template <class... A>
    std::nullptr_t refuse(const char *format, A... args) {
        PyErr_Format(PyExc_ValueError, format, args...);
        ok_ = false;
        return nullptr;
    }
    const at::Tensor *checked(PyObject *o, const char *what, int types, int *type) {
        if (!ok_) return nullptr;
        if (!THPVariable_Check(o)) return refuse("%s: expected a CUDA tensor, got %s", what, Py_TYPE(o)->tp_name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) return refuse("%s: expected a CUDA tensor", what);
        if (device_ < 0 && !find_device()) return nullptr;
        if (t.get_device() != device_)
            return refuse("%s: on device %d, the current device is %d", what, static_cast<int>(t.get_device()), static_cast<int>(device_));
        const int k = type_of(t);
        if (k < 0 || !(types >> k & 1)) return refuse("%s: dtype %s is not supported here", what, c10::toString(t.scalar_type()));
        if (t.is_nested() || !t.is_contiguous()) return refuse("%s: expected a contiguous tensor", what);
        if (type) *type = k;
        return &t;
    }
    void *sized(const at::Tensor &t, const char *what, __int128 count) {
        if (t.numel() < count)
            return refuse("%s: %lld elements, %lld are needed", what, static_cast<long long>(t.numel()),
                          count > INT64_MAX ? static_cast<long long>(INT64_MAX) : static_cast<long long>(count));
        return t.data_ptr();
    }

    bool ok_ = true;
    long device_ = -1;
};

// The entry point's status, called without the interpreter's lock (a launch
// may wait for room in the queue).
template <class F>
PyObject *status(const Call &c, F &&f) {
    if (!c.ok()) return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 5)) return nullptr;
    Call c;
    const int64_t R = c.number(a[2]), K = c.number(a[3]);
    int type = 0;
    const void *x = c.tensor(a[0], "X", kF32 | kBF16 | kF16, R, K, &type);
    void *w = c.matrix(a[1], "W", R, K);
    const q4_0_stream_t s = c.stream(a[4]);
    return status(c, [&] { return mxfp4_quantize(x, type, w, R, K, s); });
}

PyObject *dequant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 5)) return nullptr;
    Call c;
    const int64_t R = c.number(a[2]), K = c.number(a[3]);
    int type = 0;
    const void *w = c.matrix(a[0], "W", R, K);
    void *out = c.tensor(a[1], "out", kF32 | kBF16 | kF16, R, K, &type);
    const q4_0_stream_t s = c.stream(a[4]);
    return status(c, [&] { return mxfp4_dequant(w, out, type, R, K, s); });
}

PyObject *pack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 6)) return nullptr;
    Call c;
    const int64_t R = c.number(a[3]), K = c.number(a[4]);
    const void *codes = c.tensor(a[0], "codes", kBytes, R, K / 2), *scales = c.tensor(a[1], "scales", kBytes, R, K / 32);
    void *w = c.matrix(a[2], "W", R, K);
    const q4_0_stream_t s = c.stream(a[5]);
    return status(c, [&] { return mxfp4_pack(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), w, R, K, s); });
}

PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 7)) return nullptr;
    Call c;
    const int64_t M = c.number(a[3]), N = c.number(a[4]), K = c.number(a[5]);
    int type = 0;
    const void *w = c.matrix(a[0], "W", N, K), *x = c.matrix(a[1], "X", M, K);
    void *y = c.tensor(a[2], "Y", kF32 | kBF16, M, N, &type);
    const q4_0_stream_t s = c.stream(a[6]);
    return status(c, [&] { return mxfp4_gemm(w, x, y, type, M, N, K, s); });
}

// r, M, D, y, post_weight, gate, gate_span, scale, pre_weight, x, r_out, eps, stream
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 13)) return nullptr;
    Call c;
    q4_0_block b = {};
    const int64_t M = b.M = c.number(a[1]), D = b.D = c.number(a[2]), span = b.gate_span = c.number(a[6]);
    b.scale = c.real(a[7]);
    b.eps = c.real(a[11]);
    int type = 0;
    b.r = c.tensor(a[0], "r", kF32 | kBF16, M, D, &type);
    b.r_type = type;
    if (a[3] != Py_None) {
        b.y = c.tensor(a[3], "y", kF32 | kBF16, M, D, &type);
        b.y_type = type;
    }
    if (a[4] != Py_None) b.post_weight = static_cast<const float *>(c.tensor(a[4], "post_weight", kF32, 1, D));
    if (a[5] != Py_None)
        b.gate = static_cast<const float *>(c.tensor(a[5], "gate", kF32, span > 0 ? M / span + (M % span != 0) : 1, D));
    if (a[8] != Py_None) b.pre_weight = static_cast<const float *>(c.tensor(a[8], "pre_weight", kF32, 1, D));
    if (a[9] != Py_None) {
        b.x = c.values_or_matrix(a[9], "x", M, D, &type);
        b.x_type = type;
    }
    if (a[10] != Py_None) b.r_out = c.tensor(a[10], "r_out", 1 << b.r_type, M, D);
    const q4_0_stream_t s = c.stream(a[12]);
    return status(c, [&] { return q4_0_block_norm(&b, s); });
}

// A tensor without plain storage (sparse, fake) throws when it is asked
// for its strides or its address: an error of the caller's, not the process's end.
template <PyObject *F(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const c10::Error &e) {
        PyErr_Format(PyExc_ValueError, "expected tensors with storage: %s", e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD("mxfp4_quantize", quantize), METHOD("mxfp4_dequant", dequant), METHOD("mxfp4_pack", pack),
                           METHOD("mxfp4_gemm", gemm), METHOD("q4_0_block_norm", block_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *c = PyImport_ImportModule("torch._C");
    if (!c) return nullptr;
    g_get_device = PyObject_GetAttrString(c, "_cuda_getDevice");
    g_get_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    Py_DECREF(c);
    if (!g_get_device || !g_get_stream || !g_cuda_stream) return nullptr;
    return PyModule_Create(&g_module);
}
