// py_calls.cpp -- the plain case of the layer norm's and the microscaled calls'
// Python entry points, as a CPython module.
//
// A small call's time is the host's: in Python the checks of five to eight tensors
// take as long as the launch.  Here they take a few tens of ns each (layer norm of 17 x
// 5120: 7.0 us a call without this, 3.8 with it).  Only the plain case is decided here:
// contiguous device tensors of the right shapes and types on the current device, its
// current stream.  Everything else (what is refused among it, and calls on another
// device or stream) returns None with nothing done, and the Python function goes
// on as if this module was not there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mx4.h"

namespace {

using at::ScalarType;

// The library's functions, by their addresses in it.
decltype(&nf4_layer_norm) f_norm;
decltype(&nf4_layer_norm_grad) f_norm_grad;
decltype(&mx4_quantize) f_quantize;
decltype(&mx4_dequantize) f_dequantize;
decltype(&mx4_matmul) f_matmul;
decltype(&mx4_matmul4) f_matmul4;
PyObject* current_stream;   // of a device's index, as an address

// The checks of one call.  `ok` stays true while all is plain.
struct Call {
    bool ok = true;
    int dev = -1;

    const at::Tensor* tensor(PyObject* o)
    {
        if (!ok || !THPVariable_CheckExact(o)) return fail();
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || !t.is_contiguous()) return fail();
        if (dev < 0) dev = t.get_device();
        return t.get_device() == dev ? &t : fail();
    }

    const at::Tensor* fail()
    {
        ok = false;
        return nullptr;
    }

    // The first tensor of a call: two dimensions, bfloat16 or float16.
    const at::Tensor* first16(PyObject* o)
    {
        const at::Tensor* t = tensor(o);
        if (!t) return nullptr;
        const bool good = t->dim() == 2 && (t->scalar_type() == ScalarType::BFloat16 || t->scalar_type() == ScalarType::Half);
        return good ? t : fail();
    }

    // The address of a tensor of this type and shape.
    void* at(PyObject* o, ScalarType type, int64_t rows, int64_t cols)
    {
        const at::Tensor* t = tensor(o);
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != rows || t->size(1) != cols) return (fail(), nullptr);
        return t->mutable_data_ptr();
    }
    void* at(PyObject* o, ScalarType type, int64_t n)
    {
        const at::Tensor* t = tensor(o);
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n) return (fail(), nullptr);
        return t->mutable_data_ptr();
    }
    void* at_or_none(PyObject* o, ScalarType type, int64_t rows, int64_t cols)
    {
        return o == Py_None ? nullptr : at(o, type, rows, cols);
    }

    struct Pair {
        uint8_t *codes, *scales;
        int64_t rows, cols;
    };
    Pair pair(PyObject* codes, PyObject* scales)
    {
        const at::Tensor* c = tensor(codes);
        if (!c || c->scalar_type() != ScalarType::Byte || c->dim() != 2 || c->size(1) % 16) return (fail(), Pair{});
        Pair p{static_cast<uint8_t*>(c->mutable_data_ptr()), nullptr, c->size(0), 2 * c->size(1)};
        p.scales = static_cast<uint8_t*>(at(scales, ScalarType::Byte, p.rows, p.cols / 32));
        return p;
    }

    struct Space {
        void* p;
        size_t bytes;
    };
    Space space(PyObject* o)
    {
        if (o == Py_None) return Space{nullptr, 0};
        const at::Tensor* t = tensor(o);
        return t ? Space{t->mutable_data_ptr(), static_cast<size_t>(t->nbytes())} : Space{};
    }

    // The last check, and the current stream.
    bool stream(PyObject* given, hipStream_t* s)
    {
        if (!ok || given != Py_None) return false;
        if (c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() != dev) return false;
        PyObject* i = PyLong_FromLong(dev);
        PyObject* v = i ? PyObject_CallOneArg(current_stream, i) : nullptr;
        Py_XDECREF(i);
        if (!v) return (PyErr_Clear(), false);
        *s = static_cast<hipStream_t>(PyLong_AsVoidPtr(v));
        Py_DECREF(v);
        if (PyErr_Occurred()) return (PyErr_Clear(), false);
        return true;
    }
};

int dtype_of(ScalarType t) { return t == ScalarType::BFloat16 ? NF4_BF16 : NF4_FP16; }

// The call without the interpreter's lock, its status as Python's.
template <class F>
PyObject* enqueue(F&& call)
{
    nf4_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// A function of so many arguments that may throw (torch's accessors do): None then, and Python finds out.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f)
{
    if (n == want) {
        try {
            if (PyObject* r = f()) return r;
            if (PyErr_Occurred()) return nullptr;
        } catch (const std::exception&) {
        }
    }
    Py_RETURN_NONE;
}

// x, weight, bias, out, stats, eps, residual, total, stream
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const at::Tensor* x = c.first16(a[0]);
        if (!x) return nullptr;
        const ScalarType t = x->scalar_type();
        const int64_t m = x->size(0), k = x->size(1);
        void *w = c.at(a[1], t, k), *b = c.at(a[2], t, k), *out = c.at(a[3], t, m, k), *st = c.at(a[4], ScalarType::Float, m, 2);
        void *res = c.at_or_none(a[6], t, m, k), *total = c.at_or_none(a[7], t, m, k);
        if (!PyFloat_Check(a[5]) || !c.stream(a[8], &s)) return nullptr;
        const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[5]));
        void* xp = x->mutable_data_ptr();
        return enqueue([&] { return f_norm(xp, res, w, b, m, k, dtype_of(t), eps, out, total, static_cast<float*>(st), s); });
    });
}

// dy, x, weight, stats, dx, dweight, dbias, ws, residual, stream
PyObject* layer_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const at::Tensor* dy = c.first16(a[0]);
        if (!dy) return nullptr;
        const ScalarType t = dy->scalar_type();
        const int64_t m = dy->size(0), k = dy->size(1);
        void *x = c.at(a[1], t, m, k), *w = c.at(a[2], t, k), *st = c.at(a[3], ScalarType::Float, m, 2), *dx = c.at(a[4], t, m, k);
        void *dw = c.at(a[5], ScalarType::Float, k), *db = c.at(a[6], ScalarType::Float, k), *res = c.at_or_none(a[8], t, m, k);
        const Call::Space ws = c.space(a[7]);
        if (!c.stream(a[9], &s)) return nullptr;
        void* yp = dy->mutable_data_ptr();
        return enqueue([&] {
            return f_norm_grad(yp, x, w, static_cast<float*>(st), res, m, k, dtype_of(t), dx, static_cast<float*>(dw),
                               static_cast<float*>(db), ws.p, ws.bytes, s);
        });
    });
}

// x, codes, scales, err, ws, stream
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const at::Tensor* x = c.first16(a[0]);
        const Call::Pair w = c.pair(a[1], a[2]);
        if (!c.ok || x->size(0) != w.rows || x->size(1) != w.cols) return nullptr;
        void* err = a[3] == Py_None ? nullptr : c.at(a[3], ScalarType::Double, 1);
        const Call::Space ws = c.space(a[4]);
        if (!c.stream(a[5], &s)) return nullptr;
        void* xp = x->mutable_data_ptr();
        const int dt = dtype_of(x->scalar_type());
        return enqueue([&] {
            return f_quantize(xp, w.rows, w.cols, dt, w.codes, w.scales, static_cast<double*>(err), ws.p, ws.bytes, s);
        });
    });
}

// codes, scales, out, stream
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 4, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const at::Tensor* out = c.first16(a[2]);
        const Call::Pair w = c.pair(a[0], a[1]);
        if (!c.ok || out->size(0) != w.rows || out->size(1) != w.cols || !c.stream(a[3], &s)) return nullptr;
        void* op = out->mutable_data_ptr();
        const int dt = dtype_of(out->scalar_type());
        return enqueue([&] { return f_dequantize(w.codes, w.scales, w.rows, w.cols, dt, op, s); });
    });
}

// codes, scales, x, out, ws, backward, stream
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const at::Tensor* x = c.first16(a[2]);
        const Call::Pair w = c.pair(a[0], a[1]);
        const at::Tensor* out = c.tensor(a[3]);
        if (!c.ok || !PyBool_Check(a[5])) return nullptr;
        const bool back = a[5] == Py_True, f32 = out->scalar_type() == ScalarType::Float;
        const ScalarType t = x->scalar_type();
        const int64_t m = x->size(0);
        if (x->size(1) != (back ? w.rows : w.cols)) return nullptr;
        void* op = c.at(a[3], f32 ? ScalarType::Float : t, m, back ? w.cols : w.rows);
        const Call::Space ws = c.space(a[4]);
        if (!c.stream(a[6], &s)) return nullptr;
        void* xp = x->mutable_data_ptr();
        return enqueue([&] {
            return f_matmul(w.codes, w.scales, w.rows, w.cols, dtype_of(t), back, xp, m, op, f32, ws.p, ws.bytes, s);
        });
    });
}

// codes, scales, xcodes, xscales, out, ws, stream
PyObject* matmul4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject* {
        Call c;
        hipStream_t s;
        const Call::Pair w = c.pair(a[0], a[1]), x = c.pair(a[2], a[3]);
        const at::Tensor* out = c.tensor(a[4]);
        if (!c.ok || x.cols != w.cols) return nullptr;
        const ScalarType t = out->scalar_type();
        if (t != ScalarType::Float && t != ScalarType::BFloat16 && t != ScalarType::Half) return nullptr;
        void* op = c.at(a[4], t, x.rows, w.rows);
        const Call::Space ws = c.space(a[5]);
        if (!c.stream(a[6], &s)) return nullptr;
        const int dt = t == ScalarType::Half ? NF4_FP16 : NF4_BF16;
        return enqueue([&] {
            return f_matmul4(w.codes, w.scales, w.rows, w.cols, x.codes, x.scales, x.rows, dt, op, t == ScalarType::Float,
                             ws.p, ws.bytes, s);
        });
    });
}

// setup(the six functions' addresses in the order above, current_stream)
PyObject* setup(PyObject*, PyObject* args)
{
    unsigned long long p[6];
    PyObject* cs;
    if (!PyArg_ParseTuple(args, "KKKKKKO", p, p + 1, p + 2, p + 3, p + 4, p + 5, &cs)) return nullptr;
    f_norm = reinterpret_cast<decltype(f_norm)>(p[0]);
    f_norm_grad = reinterpret_cast<decltype(f_norm_grad)>(p[1]);
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[2]);
    f_dequantize = reinterpret_cast<decltype(f_dequantize)>(p[3]);
    f_matmul = reinterpret_cast<decltype(f_matmul)>(p[4]);
    f_matmul4 = reinterpret_cast<decltype(f_matmul4)>(p[5]);
    Py_INCREF(cs);
    Py_XDECREF(current_stream);
    current_stream = cs;
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                         FAST(layer_norm),
                         FAST(layer_norm_grad),
                         FAST(quantize),
                         FAST(dequantize),
                         FAST(matmul),
                         FAST(matmul4),
                         {nullptr, nullptr, 0, nullptr}};
#undef FAST

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
