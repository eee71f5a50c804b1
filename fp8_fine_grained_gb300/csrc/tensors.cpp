// CPython helper of the binding: the argument checks of its short calls, their
// outputs' allocation, the calls themselves, and the table that fp8fg_grad_clip
// reads, from torch tensors.
//
// Looking at one property of a tensor from Python takes 0.07 to 0.15 us, a
// check of its type, layout and extent half a microsecond with the call, a
// foreign call with 18 arguments 1.5 us: for a decoding step's norm that was
// more than the kernel, and for the gradients of a whole model many times the
// library's own work. Here it takes a few nanoseconds. A norm of one row takes
// 3.8 us in all (6.2 by ctypes), half of it the launch, and its four outputs 6
// more (15 by torch.empty). This module is compiled against the installed
// torch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <exception>
#include <tuple>
#include <type_traits>
#include <utility>

#include <ATen/ops/empty.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8fg.h"

namespace {

PyObject *refuse(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return nullptr;
}

// f(), with a C++ exception (a tensor without storage, for example) as ValueError
template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

// describe(grads, outs) -> bytes: one fp8fg_grad per tensor of the two lists
// (of the same length; outs may be grads itself), written into `table`, which
// is returned. Raises ValueError for what the kernels cannot take; the device
// is looked at last.
PyObject *describe_into(PyObject *table, PyObject *grads, PyObject *outs)
{
    const Py_ssize_t n = PyList_GET_SIZE(grads);
    fp8fg_grad *row = reinterpret_cast<fp8fg_grad *>(PyBytes_AS_STRING(table));
    const char *bad = nullptr;
    bool cuda = true, one_device = true;
    c10::Device device(c10::DeviceType::CPU);
    for (Py_ssize_t i = 0; i < n && !bad; ++i) {
        PyObject *go = PyList_GET_ITEM(grads, i), *oo = PyList_GET_ITEM(outs, i);
        if (!THPVariable_Check(go) || !THPVariable_Check(oo)) {
            bad = "grads and out must hold tensors";
            break;
        }
        const at::Tensor &g = THPVariable_Unpack(go), &o = THPVariable_Unpack(oo);
        const at::ScalarType type = g.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16)
            bad = "gradients must be float32 or bfloat16";
        else if (o.scalar_type() != type || o.numel() != g.numel())
            bad = "out must match the gradients' sizes and types";
        else if (g.layout() != at::kStrided || o.layout() != at::kStrided || !g.is_contiguous() || !o.is_contiguous())
            bad = "gradients and out must be contiguous";
        if (bad)
            break;
        if (i == 0)
            device = g.device();
        cuda = cuda && g.is_cuda() && o.is_cuda();
        one_device = one_device && g.device() == device && o.device() == device;
        row[i].g = g.const_data_ptr();
        row[i].out = o.mutable_data_ptr();
        row[i].n = g.numel();
        row[i].kind = type == at::kFloat ? FP8FG_OUT_F32 : FP8FG_OUT_BF16;
        row[i].unused = 0;
    }
    if (!bad && !cuda)
        bad = "grads and out must be CUDA tensors";
    if (!bad && !one_device)
        bad = "grads and out must be on one device";
    return bad ? refuse(bad) : table;
}

PyObject *describe(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 2 || !PyList_Check(args[0]) || !PyList_Check(args[1]) ||
        PyList_GET_SIZE(args[0]) != PyList_GET_SIZE(args[1]))
        return refuse("describe takes two lists of the same length");
    PyObject *table =
        PyBytes_FromStringAndSize(nullptr, PyList_GET_SIZE(args[0]) * (Py_ssize_t)sizeof(fp8fg_grad));
    if (!table)
        return nullptr;
    PyObject *rows = guarded([&] { return describe_into(table, args[0], args[1]); });
    if (!rows)
        Py_DECREF(table);
    return rows;
}

// Arguments (tensor, dtype, size, ..., name) shared by matrix and vector:
// false, with the error set, when they are not that or the dtype differs.
bool typed_tensor(PyObject *const *args, Py_ssize_t nargs, Py_ssize_t want)
{
    if (nargs != want || !THPDtype_Check(args[1]) || !PyUnicode_Check(args[want - 1])) {
        refuse("bad call of the argument check");
        return false;
    }
    if (!THPVariable_Check(args[0])) {
        PyErr_Format(PyExc_ValueError, "%U must be a tensor", args[want - 1]);
        return false;
    }
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    if (t.scalar_type() != reinterpret_cast<THPDtype *>(args[1])->scalar_type) {
        PyErr_Format(PyExc_ValueError, "%U must be %S", args[want - 1], args[1]);
        return false;
    }
    return true;
}

// matrix(t, dtype, rows, cols, name) -> row pitch of a 2-D row-major tensor of
// the dtype that covers [rows, cols]; for a tensor of one row, whose stride
// means nothing, one that every entry point takes
PyObject *matrix(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded([&]() -> PyObject * {
        if (!typed_tensor(args, nargs, 5))
            return nullptr;
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        const long long rows = PyLong_AsLongLong(args[2]), cols = PyLong_AsLongLong(args[3]);
        if (PyErr_Occurred())
            return nullptr;
        if (t.layout() != at::kStrided || t.dim() != 2 || t.stride(1) != 1)
            return PyErr_Format(PyExc_ValueError, "%U must be a 2-D row-major tensor (unit inner stride)", args[4]);
        if (t.size(0) < rows || t.size(1) < cols)
            return PyErr_Format(PyExc_ValueError, "%U must cover [%lld, %lld], got (%lld, %lld)", args[4], rows, cols,
                                (long long)t.size(0), (long long)t.size(1));
        // (one row has no pitch: torch lets its stride be anything)
        return PyLong_FromLongLong(t.size(0) == 1 ? (t.size(1) + 15) / 16 * 16 : t.stride(0));
    });
}

// vector(t, dtype, n, name): a contiguous vector of at least n entries
PyObject *vector(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded([&]() -> PyObject * {
        if (!typed_tensor(args, nargs, 4))
            return nullptr;
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        const long long n = PyLong_AsLongLong(args[2]);
        if (PyErr_Occurred())
            return nullptr;
        if (t.layout() != at::kStrided || t.dim() != 1 || t.numel() < n || !t.is_contiguous())
            return PyErr_Format(PyExc_ValueError, "%U must be a contiguous vector of at least %lld entries", args[3],
                                n);
        Py_RETURN_NONE;
    });
}

// norm_weight(gamma, D) -> FP8FG_OUT_F32 or FP8FG_OUT_BF16: a norm's weight, a
// contiguous vector of exactly D entries
PyObject *norm_weight(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded([&]() -> PyObject * {
        if (nargs != 2)
            return refuse("bad call of the argument check");
        if (!THPVariable_Check(args[0]))
            return refuse("gamma must be a tensor");
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        const long long n = PyLong_AsLongLong(args[1]);
        if (PyErr_Occurred())
            return nullptr;
        if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
            return refuse("gamma must be float32 or bfloat16");
        if (t.layout() != at::kStrided || t.dim() != 1 || t.numel() != n || !t.is_contiguous())
            return PyErr_Format(PyExc_ValueError, "gamma must be a contiguous vector of %lld entries", n);
        return PyLong_FromLong(t.scalar_type() == at::kFloat ? FP8FG_OUT_F32 : FP8FG_OUT_BF16);
    });
}

// on_gpu(t, name, t, name, ...): every tensor (None is skipped) is a CUDA
// tensor, all on one device, and that is the current one: the call's stream,
// its workspace's size and its launch are the current device's
PyObject *on_gpu(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    return guarded([&]() -> PyObject * {
        c10::Device device(c10::DeviceType::CPU);
        for (Py_ssize_t i = 0; i + 1 < nargs; i += 2) {
            if (args[i] == Py_None)
                continue;
            if (!THPVariable_Check(args[i]) || !THPVariable_Unpack(args[i]).is_cuda())
                return PyErr_Format(PyExc_ValueError, "%U must be a CUDA tensor", args[i + 1]);
            const c10::Device d = THPVariable_Unpack(args[i]).device();
            if (device.is_cpu())
                device = d;
            if (d != device)
                return PyErr_Format(PyExc_ValueError, "%U must be on the other tensors' device", args[i + 1]);
        }
        if (!device.is_cpu()) {
            const int current = c10::impl::getDeviceGuardImpl(device.type())->getDevice().index();
            if (device.index() != current)
                return PyErr_Format(PyExc_ValueError, "the tensors must be on the current device (cuda:%d), not on cuda:%d",
                                    current, (int)device.index());
        }
        Py_RETURN_NONE;
    });
}

// empty(like, dtype, n) or empty(like, dtype, rows, cols) -> a contiguous
// tensor on like's device
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS  // (out of memory stays torch's own error)
    if ((nargs != 3 && nargs != 4) || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1]))
        return refuse("bad call of the allocation");
    int64_t size[2] = {0, 0};
    for (Py_ssize_t i = 2; i < nargs; ++i)
        size[i - 2] = PyLong_AsLongLong(args[i]);
    if (PyErr_Occurred())
        return nullptr;
    const at::TensorOptions options = at::TensorOptions()
                                          .dtype(reinterpret_cast<THPDtype *>(args[1])->scalar_type)
                                          .device(THPVariable_Unpack(args[0]).device());
    return THPVariable_Wrap(at::empty(at::IntArrayRef(size, (size_t)nargs - 2), options));
    END_HANDLE_TH_ERRORS
}

// An argument of a library call: pointers come from a tensor (its data), None,
// a bytes object or an address.
template <typename T>
bool take(PyObject *o, T &v)
{
    if constexpr (std::is_pointer_v<T>) {
        if (THPVariable_Check(o)) {
            const at::Tensor &t = THPVariable_Unpack(o);
            if constexpr (std::is_const_v<std::remove_pointer_t<T>>)
                v = static_cast<T>(t.const_data_ptr());
            else
                v = static_cast<T>(t.mutable_data_ptr());
        } else if (o == Py_None) {
            v = nullptr;
        } else if (PyBytes_Check(o)) {
            v = reinterpret_cast<T>(PyBytes_AS_STRING(o));
        } else {
            v = static_cast<T>(PyLong_AsVoidPtr(o));
        }
    } else if constexpr (std::is_floating_point_v<T>) {
        v = (T)PyFloat_AsDouble(o);
    } else {
        v = (T)PyLong_AsLongLong(o);
    }
    return !PyErr_Occurred();
}

template <typename R, typename... A, size_t... I>
PyObject *invoke(R (*fn)(A...), PyObject *const *args, Py_ssize_t nargs, std::index_sequence<I...>)
{
    if (!fn || nargs != (Py_ssize_t)sizeof...(A))
        return refuse(fn ? "bad call of the library" : "the library is not bound");
    return guarded([&]() -> PyObject * {
        std::tuple<A...> v;
        if (!(take(args[I], std::get<I>(v)) && ...))
            return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS;  // (a launch waits when the stream's queue is full)
        r = fn(std::get<I>(v)...);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLongLong(r);
    });
}

template <typename R, typename... A>
PyObject *invoke(R (*fn)(A...), PyObject *const *args, Py_ssize_t nargs)
{
    return invoke(fn, args, nargs, std::index_sequence_for<A...>());
}

// NAME(arguments of the library's NAME) -> what it returns
#define ENTRIES(X) \
    X(fp8_rmsnorm) X(fp8_rmsnorm_t) X(fp8_rmsnorm_bwd) X(fp8_rmsnorm_bwd_workspace) X(fp8_gated_gemm) \
    X(fp8_gated_bwd) X(fp8fg_grad_clip) X(fp8fg_grad_clip_workspace)
#define DEFINE(NAME) \
    decltype(&::NAME) NAME##_fn; \
    PyObject *call_##NAME(PyObject *, PyObject *const *args, Py_ssize_t nargs) \
    { \
        return invoke(NAME##_fn, args, nargs); \
    }
ENTRIES(DEFINE)

// bind(handle): look the entry points up in the loaded library
PyObject *bind(PyObject *, PyObject *handle)
{
    void *lib = PyLong_AsVoidPtr(handle);
    if (PyErr_Occurred())
        return nullptr;
#define LOOKUP(NAME) \
    NAME##_fn = reinterpret_cast<decltype(&::NAME)>(dlsym(lib, #NAME)); \
    if (!NAME##_fn) \
        return refuse("the library lacks " #NAME);
    ENTRIES(LOOKUP)
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

PyMethodDef methods[] = {
    {"describe", fast(describe), METH_FASTCALL, "describe(grads, outs) -> bytes of fp8fg_grad rows"},
    {"matrix", fast(matrix), METH_FASTCALL, "matrix(t, dtype, rows, cols, name) -> row pitch"},
    {"vector", fast(vector), METH_FASTCALL, "vector(t, dtype, n, name)"},
    {"norm_weight", fast(norm_weight), METH_FASTCALL, "norm_weight(gamma, D) -> output kind of its type"},
    {"on_gpu", fast(on_gpu), METH_FASTCALL, "on_gpu(t, name, t, name, ...)"},
    {"empty", fast(empty), METH_FASTCALL, "empty(like, dtype, n) or (like, dtype, rows, cols) -> tensor"},
    {"bind", bind, METH_O, "bind(handle of libfp8fg.so)"},
#define METHOD(NAME) {#NAME, fast(call_##NAME), METH_FASTCALL, #NAME "(the library's arguments) -> what it returns"},
    ENTRIES(METHOD)
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
