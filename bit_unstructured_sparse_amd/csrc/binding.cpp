// binding.cpp -- the steps that every call of the Python binding repeats, natively: checking a
// tensor against what an entry point takes, making an output, and the call itself with the
// stream and device it runs on. Optional: without this module the binding's own Python
// functions do the same, several times slower (a tensor's check 0.6 us against 0.06, an output 2.6
// against 0.9, a call of 13 arguments 2.2 against 0.2, where a launch takes 2).
//
// Each function here handles the common case and hands every other one -- a wrong type or shape, a
// stream of the caller's, another current device, a tensor subclass -- to the Python function it
// stands for, with the same arguments, so that what is refused and how is written once.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <iterator>
#include <type_traits>
#include <utility>

#include "bitmap_spmm.h"

namespace {

PyObject *py_flat, *py_rows, *py_matrix_rows, *py_new_output, *py_launch;      // the Python functions
PyObject *torch_dict, *torch_empty;      // torch's own empty, as long as nobody replaced it

// ---- the library's entry points, called with the types of their declarations ----

struct Arg {
    int64_t i;
    double d;
};

template <class T>
T as(const Arg &a) {
    if constexpr (std::is_pointer_v<T>)
        return reinterpret_cast<T>(static_cast<uintptr_t>(a.i));
    else if constexpr (std::is_floating_point_v<T>)
        return static_cast<T>(a.d);
    else
        return static_cast<T>(a.i);
}

template <class... A, size_t... I>
int invoke_with(int (*f)(A...), const Arg *v, std::index_sequence<I...>) {
    return f(as<A>(v[I])...);
}

template <class... A>
constexpr int arity(int (*)(A...)) {
    return (int)sizeof...(A);
}

#define MOST_ARGS 20

enum Kind : char { WHOLE, REAL, ADDRESS };

template <class T>
constexpr Kind kind_of = std::is_pointer_v<T> ? ADDRESS : std::is_floating_point_v<T> ? REAL : WHOLE;

template <class Fn>
struct Kinds;
template <class... A>
struct Kinds<int (*)(A...)> {
    static constexpr Kind of[] = {kind_of<A>...};
};

struct Entry {
    const char *name;
    int args;
    const Kind *kinds;      // of its arguments
    int (*invoke)(void *, const Arg *);
    PyObject *object;      // the library's function object, as the binding passes it
    void *address;
};

template <class Fn>
int invoke(void *address, const Arg *v) {
    return invoke_with(reinterpret_cast<Fn>(address), v, std::make_index_sequence<arity(Fn{})>{});
}

// (declarations only: the addresses come from the library that the binding has loaded)
#define ENTRY(name) {#name, arity(decltype(&name){}), Kinds<decltype(&name)>::of, invoke<decltype(&name)>, nullptr, nullptr}

Entry entries[] = {
    ENTRY(kv_cache_append),     ENTRY(kv_cache_gather),         ENTRY(attention_tree_f16),
    ENTRY(kv_pages_step),       ENTRY(qk_norm_rope_f16),        ENTRY(qk_norm_rope_append_f16),
    ENTRY(quantize_tokens_f16), ENTRY(dequantize_tokens_f16),   ENTRY(gemm_w8a8_dq),
};

// What ctypes takes for an argument of its kind, as a plain integer, None or bytes (addresses) or float; false for
// anything else.
bool argument(PyObject *o, Kind kind, Arg &a) {
    a.d = 0.0;
    if (PyLong_CheckExact(o)) {
        a.i = (int64_t)PyLong_AsUnsignedLongLongMask(o);
        int overflow = 0;
        (void)PyLong_AsLongLongAndOverflow(o, &overflow);
        a.d = (double)a.i;
        return overflow == 0;
    }
    if (kind == ADDRESS && o == Py_None) return a.i = 0, true;
    if (kind == ADDRESS && PyBytes_CheckExact(o)) return a.i = (int64_t)(uintptr_t)PyBytes_AS_STRING(o), true;
    if (kind == REAL && PyFloat_CheckExact(o)) return a.i = 0, a.d = PyFloat_AS_DOUBLE(o), true;
    return false;
}

const at::Tensor *plain(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool integer(PyObject *o, int64_t &v) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    v = PyLong_AsLongLongAndOverflow(o, &overflow);
    return overflow == 0;
}

// A tensor on device `index` of type `dtype`.
const at::Tensor *on_device(PyObject *o, at::ScalarType type, int64_t index) {
    const at::Tensor *t = plain(o);
    if (t == nullptr || !t->is_cuda() || t->scalar_type() != type || t->device().index() != index) return nullptr;
    return t;
}

// (t, name, dtype, numel, index) -> address
PyObject *flat(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t numel, index;
    if (n == 5 && THPDtype_Check(a[2]) && integer(a[3], numel) && integer(a[4], index)) {
        const at::Tensor *t = on_device(a[0], reinterpret_cast<THPDtype *>(a[2])->scalar_type, index);
        if (t != nullptr && t->numel() == numel && t->is_contiguous())
            return PyLong_FromVoidPtr(t->data_ptr());
    }
    return PyObject_Vectorcall(py_flat, a, (size_t)n, nullptr);
    END_HANDLE_TH_ERRORS
}

// (t, name, n or None, heads, dim, index) -> stride between tokens
PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t m = -1, heads, dim, index;
    if (n == 6 && (a[2] == Py_None || integer(a[2], m)) && integer(a[3], heads) && integer(a[4], dim) && integer(a[5], index)) {
        const at::Tensor *t = on_device(a[0], at::kHalf, index);
        if (t != nullptr && t->dim() == 3 && t->size(1) == heads && t->size(2) == dim &&
            (a[2] == Py_None || t->size(0) == m)) {
            const int64_t width = heads * dim;
            if (t->is_contiguous()) return PyLong_FromLongLong(width);
            if (t->stride(2) == 1 && (heads == 1 || t->stride(1) == dim)) {
                if (t->size(0) <= 1) return PyLong_FromLongLong(width);
                if (t->stride(0) >= width) return PyLong_FromLongLong(t->stride(0));
            }
        }
    }
    return PyObject_Vectorcall(py_rows, a, (size_t)n, nullptr);
    END_HANDLE_TH_ERRORS
}

// (t, name, dtype, n, width, index) -> stride between rows
PyObject *matrix_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t m, width, index;
    if (n == 6 && THPDtype_Check(a[2]) && integer(a[3], m) && integer(a[4], width) && integer(a[5], index)) {
        const at::Tensor *t = on_device(a[0], reinterpret_cast<THPDtype *>(a[2])->scalar_type, index);
        if (t != nullptr && t->dim() == 2 && t->size(0) == m && t->size(1) == width) {
            if (t->is_contiguous()) return PyLong_FromLongLong(width);
            if (t->stride(1) == 1 || width <= 1) {
                if (m <= 1) return PyLong_FromLongLong(width);
                if (t->stride(0) >= width) return PyLong_FromLongLong(t->stride(0));
            }
        }
    }
    return PyObject_Vectorcall(py_matrix_rows, a, (size_t)n, nullptr);
    END_HANDLE_TH_ERRORS
}

// (shape, dtype, device, stream) -> tensor
PyObject *new_output(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n == 4 && a[3] == Py_None && PyTuple_CheckExact(a[0]) && THPDtype_Check(a[1]) && THPDevice_Check(a[2]) &&
        PyDict_GetItemString(torch_dict, "empty") == torch_empty) {
        const c10::Device device = reinterpret_cast<THPDevice *>(a[2])->device;
        const Py_ssize_t dims = PyTuple_GET_SIZE(a[0]);
        int64_t size[4];
        bool good = device.is_cuda() && device.has_index() && dims <= 4;
        for (Py_ssize_t i = 0; good && i < dims; ++i)
            good = integer(PyTuple_GET_ITEM(a[0], i), size[i]) && size[i] >= 0;
        if (good)
            return THPVariable_Wrap(at::empty(c10::IntArrayRef(size, (size_t)dims),
                                              at::TensorOptions(reinterpret_cast<THPDtype *>(a[1])->scalar_type).device(device)));
    }
    return PyObject_Vectorcall(py_new_output, a, (size_t)n, nullptr);
    END_HANDLE_TH_ERRORS
}

// (function, index, stream, arguments ...) -> status
PyObject *launch(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int64_t index;
    if (n >= 3 && a[2] == Py_None && integer(a[1], index)) {
        for (const Entry &e : entries) {
            if (e.object != a[0] || e.address == nullptr) continue;
            Arg v[MOST_ARGS];
            bool good = e.args == (int)n - 2 && e.args <= MOST_ARGS;
            for (Py_ssize_t i = 3; good && i < n; ++i) good = argument(a[i], e.kinds[i - 3], v[i - 3]);
            if (!good || c10::hip::current_device() != index) break;
            v[e.args - 1].i = (int64_t)(uintptr_t)c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream();
            int status;
            Py_BEGIN_ALLOW_THREADS      // (a full queue makes a launch wait)
            status = e.invoke(e.address, v);
            Py_END_ALLOW_THREADS
            return PyLong_FromLong(status);
        }
    }
    return PyObject_Vectorcall(py_launch, a, (size_t)n, nullptr);
    END_HANDLE_TH_ERRORS
}

// bind(library handle, {name: function object}, (flat, rows, matrix_rows, new_output, launch), torch): the
// Python functions that the ones here stand for, and the library they call.
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long handle;
    PyObject *functions, *f[5], *torch;
    if (!PyArg_ParseTuple(args, "KO!(OOOOO)O", &handle, &PyDict_Type, &functions, f, f + 1, f + 2, f + 3, f + 4, &torch))
        return nullptr;
    PyObject *const dict = PyModule_GetDict(torch), *const empty = PyDict_GetItemString(dict, "empty");
    if (empty == nullptr) return PyErr_SetString(PyExc_ValueError, "torch has no empty"), nullptr;
    PyObject **const to[] = {&py_flat, &py_rows, &py_matrix_rows, &py_new_output, &py_launch, &torch_dict, &torch_empty};
    PyObject *const from[] = {f[0], f[1], f[2], f[3], f[4], dict, empty};
    for (size_t i = 0; i < std::size(to); ++i) {
        Py_INCREF(from[i]);
        Py_XDECREF(*to[i]);
        *to[i] = from[i];
    }
    for (Entry &e : entries) {
        PyObject *o = PyDict_GetItemString(functions, e.name);
        Py_XINCREF(o);
        Py_XDECREF(e.object);
        e.object = o;
        e.address = o == nullptr ? nullptr : dlsym(reinterpret_cast<void *>((uintptr_t)handle), e.name);
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"flat", (PyCFunction)(void (*)(void))flat, METH_FASTCALL, nullptr},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL, nullptr},
    {"matrix_rows", (PyCFunction)(void (*)(void))matrix_rows, METH_FASTCALL, nullptr},
    {"new_output", (PyCFunction)(void (*)(void))new_output, METH_FASTCALL, nullptr},
    {"launch", (PyCFunction)(void (*)(void))launch, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Native steps of the binding's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
