// CPython helper of the binding: the table that fp8fg_grad_clip reads, from
// lists of torch tensors.
//
// A call that clips the gradients of a whole model passes hundreds of tensors.
// Looking at one from Python (type, size, contiguity, device, address) takes
// about a quarter of a microsecond, many times the library's own work on it;
// here it takes a few nanoseconds. This module only reads the tensors'
// metadata; it is compiled against the installed torch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "fp8fg.h"

namespace {

PyObject *refuse(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return nullptr;
}

// describe(grads, outs) -> bytes: one fp8fg_grad per tensor of the two lists
// (of the same length; outs may be grads itself). Raises ValueError for what
// the kernels cannot take; the device is looked at last.
PyObject *describe_checked(PyObject *grads, PyObject *outs)
{
    const Py_ssize_t n = PyList_GET_SIZE(grads);
    PyObject *table = PyBytes_FromStringAndSize(nullptr, n * (Py_ssize_t)sizeof(fp8fg_grad));
    if (!table)
        return nullptr;
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
    if (bad) {
        Py_DECREF(table);
        return refuse(bad);
    }
    return table;
}

PyObject *describe(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 2 || !PyList_Check(args[0]) || !PyList_Check(args[1]) ||
        PyList_GET_SIZE(args[0]) != PyList_GET_SIZE(args[1]))
        return refuse("describe takes two lists of the same length");
    try {
        return describe_checked(args[0], args[1]);
    } catch (const std::exception &e) {  // a tensor without storage, for example
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"describe", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(describe)), METH_FASTCALL,
     "describe(grads, outs) -> bytes of fp8fg_grad rows"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
