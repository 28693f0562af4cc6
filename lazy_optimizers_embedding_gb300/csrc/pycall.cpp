// pycall.cpp -- the operators around the table step called from Python: tensors to pointers, checked as the
// binding checks them, and the C entry point, without a Python frame or a foreign-function
// conversion per argument (a call of sparse_layer_norm: 2.1 us of host time against 5.6, the launch among them).
//
// Every function returns the entry point's status, or None for any argument that is not of the common
// kind (a contiguous CUDA tensor of the type wanted, None, a plain number, the current stream):
// the binding's own path then takes the call, converts what can be converted and says what is
// wrong with the rest.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>

#include <ATen/core/TensorBody.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sparseopt.h"

namespace {

PyObject *ns_config = nullptr, *muon_config = nullptr;   // the binding's structures

struct Args {
    PyObject* const* a;
    bool ok = true;

    const at::Tensor* tensor(int i)
    {
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda() || !t.is_contiguous()) ok = false;
        return &t;
    }
    template <class T>
    T* pointer(int i, at::ScalarType type)
    {
        if (a[i] == Py_None) return nullptr;
        const at::Tensor* t = tensor(i);
        if (!ok || t->scalar_type() != type) {
            ok = false;
            return nullptr;
        }
        return static_cast<T*>(t->data_ptr());
    }
    float* floats(int i) { return pointer<float>(i, at::kFloat); }
    int32_t* ints(int i) { return pointer<int32_t>(i, at::kInt); }
    int64_t* longs(int i) { return pointer<int64_t>(i, at::kLong); }
    // fp32 or bf16; `like`: of that type only
    void* typed(int i, sparse_dtype_t& type, bool like = false)
    {
        if (!like) type = SPARSE_F32;
        if (a[i] == Py_None) return nullptr;
        const at::Tensor* t = tensor(i);
        if (!ok) return nullptr;
        const at::ScalarType s = t->scalar_type();
        const sparse_dtype_t mine = s == at::kBFloat16 ? SPARSE_BF16 : SPARSE_F32;
        if ((s != at::kBFloat16 && s != at::kFloat) || (like && mine != type)) {
            ok = false;
            return nullptr;
        }
        type = mine;
        return t->data_ptr();
    }
    void* workspace(int i, size_t& bytes)
    {
        void* p = pointer<void>(i, at::kByte);
        bytes = ok && a[i] != Py_None ? static_cast<size_t>(THPVariable_Unpack(a[i]).numel()) : 0;
        return p;
    }
    int64_t number(int i)
    {
        if (!PyLong_Check(a[i])) {
            ok = false;
            return 0;
        }
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(a[i], &over);
        if (over != 0) ok = false;
        return v;
    }
    double real(int i)
    {
        if (!PyFloat_Check(a[i])) {
            ok = false;
            return 0.0;
        }
        return PyFloat_AS_DOUBLE(a[i]);
    }
    template <class C>
    C config(int i, PyObject* type)
    {
        C c{};
        Py_buffer view;
        if (type == nullptr || reinterpret_cast<PyObject*>(Py_TYPE(a[i])) != type ||
            PyObject_GetBuffer(a[i], &view, PyBUF_SIMPLE) != 0) {
            PyErr_Clear();
            ok = false;
            return c;
        }
        if (view.len == static_cast<Py_ssize_t>(sizeof(C)))
            std::memcpy(&c, view.buf, sizeof(C));
        else
            ok = false;
        PyBuffer_Release(&view);
        return c;
    }
    cudaStream_t stream(int i)
    {
        if (a[i] != Py_None) ok = false;
        return ok ? c10::cuda::getCurrentCUDAStream().stream() : nullptr;
    }
};

// `f` reads the arguments and returns the entry point's call; nothing thrown reaches Python.
template <class F>
PyObject* run(PyObject* const* a, Py_ssize_t have, Py_ssize_t want, F f)
{
    if (have != want) Py_RETURN_NONE;
    Args args{a};
    try {
        auto call = f(args);
        if (!args.ok) Py_RETURN_NONE;
        sparse_status_t code;
        Py_BEGIN_ALLOW_THREADS
        code = call();
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(code);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 13, [](Args& g) {
        sparse_dtype_t xt, yt;
        void* x = g.typed(0, xt);
        void* y = g.typed(8, yt);
        return [=, r = g.number(1), c = g.number(2), idx = g.longs(3), rows = g.number(4), gamma = g.floats(5),
                beta = g.floats(6), eps = g.real(7), mean = g.floats(9), rstd = g.floats(10), err = g.ints(11),
                s = g.stream(12)] {
            return sparse_layer_norm(x, xt, r, c, idx, rows, gamma, beta, eps, y, yt, mean, rstd, err, s);
        };
    });
}

PyObject* layer_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 15, [](Args& g) {
        sparse_dtype_t xt, yt;
        size_t bytes;
        void* dy = g.typed(0, yt);
        void* x = g.typed(1, xt);
        void* dx = g.typed(9, xt, true);
        void* ws = g.workspace(12, bytes);
        return [=, r = g.number(2), c = g.number(3), idx = g.longs(4), rows = g.number(5), gamma = g.floats(6),
                mean = g.floats(7), rstd = g.floats(8), dgamma = g.floats(10), dbeta = g.floats(11), err = g.ints(13),
                s = g.stream(14)] {
            return sparse_layer_norm_grad(dy, yt, x, xt, r, c, idx, rows, gamma, mean, rstd, dx, dgamma, dbeta, ws,
                                          bytes, err, s);
        };
    });
}

PyObject* expert_sort(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 10, [](Args& g) {
        size_t bytes;
        void* ws = g.workspace(7, bytes);
        return [=, expert = g.longs(0), rows = g.number(1), k = g.number(2), experts = g.number(3), offsets = g.longs(4),
                src = g.ints(5), pos = g.ints(6), err = g.ints(8), s = g.stream(9)] {
            return sparse_expert_sort(expert, rows, k, experts, offsets, src, pos, ws, bytes, err, s);
        };
    });
}

PyObject* expert_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 10, [](Args& g) {
        sparse_dtype_t t;
        void* x = g.typed(0, t);
        void* xs = g.typed(7, t, true);
        return [=, rows = g.number(1), k = g.number(2), c = g.number(3), pos = g.ints(4), offsets = g.longs(5),
                experts = g.number(6), err = g.ints(8), s = g.stream(9)] {
            return sparse_expert_dispatch(x, t, rows, k, c, pos, offsets, experts, xs, err, s);
        };
    });
}

PyObject* expert_combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 9, [](Args& g) {
        sparse_dtype_t t;
        void* ys = g.typed(0, t);
        void* y = g.typed(6, t, true);
        return [=, rows = g.number(1), k = g.number(2), c = g.number(3), pos = g.ints(4), weights = g.floats(5),
                err = g.ints(7), s = g.stream(8)] {
            return sparse_expert_combine(ys, t, rows, k, c, pos, weights, y, err, s);
        };
    });
}

PyObject* expert_combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 13, [](Args& g) {
        sparse_dtype_t t;
        void* ys = g.typed(1, t);
        void* dy = g.typed(0, t, true);
        void* dys = g.typed(9, t, true);
        return [=, rows = g.number(2), k = g.number(3), c = g.number(4), pos = g.ints(5), offsets = g.longs(6),
                experts = g.number(7), weights = g.floats(8), dweights = g.floats(10), err = g.ints(11),
                s = g.stream(12)] {
            return sparse_expert_combine_grad(dy, ys, t, rows, k, c, pos, offsets, experts, weights, dys, dweights, err, s);
        };
    });
}

PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 9, [](Args& g) {
        sparse_dtype_t ut, ot;
        size_t bytes;
        void* u = g.typed(0, ut);
        void* out = g.typed(5, ot);
        void* ws = g.workspace(6, bytes);
        return [=, batch = g.number(1), r = g.number(2), c = g.number(3), err = g.ints(7),
                cfg = g.config<sparse_ns_config_t>(4, ns_config), s = g.stream(8)] {
            return sparse_orthogonalize(u, ut, batch, r, c, cfg, out, ot, ws, bytes, err, s);
        };
    });
}

PyObject* muon_step(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(a, n, 10, [](Args& g) {
        sparse_dtype_t gt;
        size_t bytes;
        void* grad = g.typed(2, gt);
        void* ws = g.workspace(7, bytes);
        return [=, w = g.floats(0), buf = g.floats(1), batch = g.number(3), r = g.number(4), c = g.number(5),
                cfg = g.config<sparse_muon_config_t>(6, muon_config), err = g.ints(8), s = g.stream(9)] {
            return sparse_muon_step(w, buf, grad, gt, batch, r, c, cfg, ws, bytes, err, s);
        };
    });
}

// The binding's NsConfig and MuonConfig.
PyObject* configs(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "configs(NsConfig, MuonConfig)");
        return nullptr;
    }
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_XDECREF(ns_config);
    Py_XDECREF(muon_config);
    ns_config = a[0];
    muon_config = a[1];
    Py_RETURN_NONE;
}

#define SO_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SO_METHOD(layer_norm),      SO_METHOD(layer_norm_grad), SO_METHOD(expert_sort),
                         SO_METHOD(expert_dispatch), SO_METHOD(expert_combine),  SO_METHOD(expert_combine_grad),
                         SO_METHOD(orthogonalize),   SO_METHOD(muon_step),       SO_METHOD(configs),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall() { return PyModule_Create(&module); }
