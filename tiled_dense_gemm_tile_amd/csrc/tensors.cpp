// What the Python binding does for every tensor of a call, in C++: the checks
// of a matrix, a vector or a list of gradients, the allocation of results, and
// the call of the C function (a matrix checked here takes 0.1 us in place of
// 0.4, a result allocated 1.0 in place of 1.8, a call of 18 arguments 0.2 in
// place of 0.9 through ctypes; the smallest calls wait for the host).
//
// Checks say yes or no: where one fails, or torch throws, the function returns
// None, and the Python form of the same check raises the error that names it.
// An error that Python code raised below is passed on.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cstring>
#include <tuple>
#include <type_traits>

#include "../../include/tilegemm_layers.h"

namespace {

// Leading dimension of one row that is not taken as given: the products' rows
// are below 8 MiB.
constexpr int64_t kLdLimit = 1 << 21;

bool of_type(const at::Tensor &t, PyObject *types) {
    if (!PyTuple_Check(types)) return false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(types); ++i) {
        PyObject *o = PyTuple_GET_ITEM(types, i);
        if (THPDtype_Check(o) && ((THPDtype *)o)->scalar_type == t.scalar_type()) return true;
    }
    return false;
}

bool plain(PyObject *o) { return THPVariable_Check(o) && THPVariable_Unpack(o).layout() == c10::kStrided; }

template <class F>
PyObject *or_none(F &&f) {
    try {
        return f();
    } catch (...) {
        if (PyErr_Occurred()) return nullptr;          // (thrown by Python code that torch called)
        Py_RETURN_NONE;
    }
}

// matrix(tensor, shape, dtypes, device index) -> (address, leading dimension)
PyObject *checked_matrix(PyObject *const *a, Py_ssize_t n) {
    if (n != 4 || !plain(a[0]) || !PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2) Py_RETURN_NONE;
    const at::Tensor &t = THPVariable_Unpack(a[0]);
    const long long rows = PyLong_AsLongLong(PyTuple_GET_ITEM(a[1], 0)), cols = PyLong_AsLongLong(PyTuple_GET_ITEM(a[1], 1)),
                    dev = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.get_device() != dev || !of_type(t, a[2]))
        Py_RETURN_NONE;
    int64_t ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1) Py_RETURN_NONE;
    if (rows <= 1 && !(cols <= ld && ld < kLdLimit)) ld = cols;
    PyObject *p = PyTuple_New(2);
    if (!p) return nullptr;
    PyTuple_SET_ITEM(p, 0, PyLong_FromVoidPtr(t.data_ptr()));
    PyTuple_SET_ITEM(p, 1, PyLong_FromLongLong(ld));
    return p;
}

PyObject *matrix(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return or_none([&] { return checked_matrix(a, n); });
}

// vector(tensor, length, dtypes, device index) -> address
PyObject *checked_vector(PyObject *const *a, Py_ssize_t n) {
    if (n != 4 || !plain(a[0])) Py_RETURN_NONE;
    const at::Tensor &t = THPVariable_Unpack(a[0]);
    const long long len = PyLong_AsLongLong(a[1]), dev = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (t.dim() != 1 || t.size(0) != len || (len > 1 && t.stride(0) != 1) || t.get_device() != dev || !of_type(t, a[2]))
        Py_RETURN_NONE;
    return PyLong_FromVoidPtr(t.data_ptr());
}

PyObject *vector(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return or_none([&] { return checked_vector(a, n); });
}

// Without the interpreter's lock, as torch's own functions run: an allocation
// may wait for the GPU.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// empty(length or shape, dtype, device index) -> tensor
PyObject *checked_empty(PyObject *const *a, Py_ssize_t n) {
    if (n != 3 || !THPDtype_Check(a[1])) Py_RETURN_NONE;
    int64_t size[2] = {};
    size_t dims = 1;
    if (PyTuple_Check(a[0])) {
        dims = (size_t)PyTuple_GET_SIZE(a[0]);
        if (dims > 2) Py_RETURN_NONE;
        for (size_t i = 0; i < dims; ++i) size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a[0], i));
    } else {
        size[0] = PyLong_AsLongLong(a[0]);
    }
    const long long dev = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    const auto options = at::TensorOptions(((THPDtype *)a[1])->scalar_type).device(at::kCUDA, (int8_t)dev);
    at::Tensor t;
    {
        Unlocked u;
        t = at::empty(c10::IntArrayRef(size, dims), options);
    }
    return THPVariable_Wrap(std::move(t));
}

PyObject *empty(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return or_none([&] { return checked_empty(a, n); });
}

// gradients(list) -> (device index, addresses, sizes, types), the last three
// bytes objects of int64, int64 and int, where all are contiguous
PyObject *gradients(PyObject *, PyObject *list) {
    if (!PyList_Check(list) || PyList_GET_SIZE(list) == 0) Py_RETURN_NONE;
    const Py_ssize_t n = PyList_GET_SIZE(list);
    PyObject *at = PyBytes_FromStringAndSize(nullptr, n * 8), *sizes = PyBytes_FromStringAndSize(nullptr, n * 8),
             *types = PyBytes_FromStringAndSize(nullptr, n * 4);
    int64_t dev = -1;
    auto take = [&](Py_ssize_t i) {
        PyObject *o = PyList_GET_ITEM(list, i);
        if (!plain(o)) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (i == 0) dev = t.get_device();
        const auto k = t.scalar_type();
        const int code = k == at::kFloat ? GEMM_TYPE_F32 : k == at::kBFloat16 ? GEMM_TYPE_BF16 : k == at::kHalf ? GEMM_TYPE_FP16 : -1;
        const int64_t p = (int64_t)(uintptr_t)t.data_ptr(), size = t.numel();
        memcpy(PyBytes_AS_STRING(at) + i * 8, &p, 8);
        memcpy(PyBytes_AS_STRING(sizes) + i * 8, &size, 8);
        memcpy(PyBytes_AS_STRING(types) + i * 4, &code, 4);
        return t.get_device() == dev && dev >= 0 && code >= 0 && t.is_contiguous();
    };
    bool fine = at && sizes && types;
    try {
        for (Py_ssize_t i = 0; fine && i < n; ++i) fine = take(i);
    } catch (...) {
        fine = false;
    }
    PyObject *r = fine ? Py_BuildValue("(LOOO)", (long long)dev, at, sizes, types) : nullptr;
    Py_XDECREF(at);
    Py_XDECREF(sizes);
    Py_XDECREF(types);
    if (r || PyErr_Occurred()) return r;
    Py_RETURN_NONE;
}

// ---- calls ----------------------------------------------------------------

template <class T>
T argument(PyObject *o) {
    if constexpr (std::is_pointer_v<T>) {
        if (o == Py_None) return nullptr;
        if (PyBytes_Check(o)) return (T)PyBytes_AS_STRING(o);
        return (T)PyLong_AsVoidPtr(o);
    } else if constexpr (std::is_floating_point_v<T>) {
        return (T)PyFloat_AsDouble(o);
    } else {
        return (T)PyLong_AsLongLong(o);
    }
}

template <class F> struct Call;
template <class R, class... A>
struct Call<R (*)(A...)> {
    typedef R (*F)(A...);
    template <size_t... I>
    static PyObject *go(F f, PyObject *const *a, std::index_sequence<I...>) {
        std::tuple<A...> v{argument<A>(a[I])...};
        if (PyErr_Occurred()) return nullptr;
        if constexpr (std::is_same_v<R, size_t>) {     // (workspace bytes)
            return PyLong_FromSize_t(f(std::get<I>(v)...));
        } else {
            R st;
            Py_BEGIN_ALLOW_THREADS
            st = f(std::get<I>(v)...);
            Py_END_ALLOW_THREADS
            return PyLong_FromLong(st);
        }
    }
    static PyObject *go(F f, PyObject *const *a, Py_ssize_t n) {
        if (!f || n != sizeof...(A)) {
            PyErr_Format(PyExc_TypeError, "%zd arguments in place of %zu, or not bound", n, sizeof...(A));
            return nullptr;
        }
        return go(f, a, std::index_sequence_for<A...>());
    }
};

// The C functions, at the addresses that bind(name, address) gave (those of the
// library that the binding has loaded).
#define TG_ENTRIES(X)                                                                                \
    X(gemm_glu) X(gemm_glu_backward) X(int8_quantize) X(gemm_int8) X(grad_norm) X(grad_clip)         \
    X(gemm_glu_workspace_bytes) X(gemm_glu_backward_workspace_bytes) X(gemm_int8_workspace_bytes)    \
    X(grad_workspace_bytes)
#define TG_ENTRY(name)                                                                     \
    decltype(&::name) at_##name = nullptr;                                                 \
    PyObject *call_##name(PyObject *, PyObject *const *a, Py_ssize_t n) {                  \
        return Call<decltype(&::name)>::go(at_##name, a, n);                               \
    }
TG_ENTRIES(TG_ENTRY)

PyObject *bind(PyObject *, PyObject *args) {
    const char *name;
    unsigned long long address;
    if (!PyArg_ParseTuple(args, "sK", &name, &address)) return nullptr;
#define TG_BIND(f) \
    if (!strcmp(name, #f)) at_##f = (decltype(&::f))(uintptr_t)address;
    TG_ENTRIES(TG_BIND)
    Py_RETURN_NONE;
}

#define TG_METHOD(f) {#f, (PyCFunction)(void (*)(void))call_##f, METH_FASTCALL, nullptr},
PyMethodDef methods[] = {{"matrix", (PyCFunction)(void (*)(void))matrix, METH_FASTCALL, nullptr},
                         {"vector", (PyCFunction)(void (*)(void))vector, METH_FASTCALL, nullptr},
                         {"empty", (PyCFunction)(void (*)(void))empty, METH_FASTCALL, nullptr},
                         {"gradients", gradients, METH_O, nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         TG_ENTRIES(TG_METHOD){nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
