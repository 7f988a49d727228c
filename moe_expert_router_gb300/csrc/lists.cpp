// lists.cpp -- what the operators over lists of tensors read of each tensor (address,
// element count, type), gathered and checked in one native pass: through Python's own
// attributes it costs about 0.4 us a tensor, more than the kernels take on short lists.
//
// CPython module `_lists`:
//   gather(tensors, name, device, dtype, like, optional)
//       -> (addresses u64, counts i64, types i32) as bytes in the machine's order
//   tensors: list or tuple of torch tensors (with `optional`, or None: address 0)
//   dtype: a MOE_DTYPE_* code that all must have, or -1 for any of them
//   like: a list of tensors whose shapes and order in memory they must have, or None
// Raises TypeError / ValueError as the rest of the binding does.
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "moe.h"

namespace {

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return MOE_DTYPE_F32;
        case at::kBFloat16: return MOE_DTYPE_BF16;
        case at::kHalf: return MOE_DTYPE_F16;
        default: return -1;
    }
}

const char *const kNames[] = {"float32", "bfloat16", "float16"};

const at::Tensor *tensor_at(PyObject *seq, Py_ssize_t i, const char *name) {
    PyObject *o = PySequence_Fast_GET_ITEM(seq, i);
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    PyErr_Format(PyExc_TypeError, "%s must hold torch tensors", name);
    return nullptr;
}

PyObject *gather(PyObject *, PyObject *args) {
    PyObject *tensors = nullptr, *like = nullptr;
    const char *name = nullptr;
    int device = 0, dtype = -1, optional = 0;
    if (!PyArg_ParseTuple(args, "OsiiOp", &tensors, &name, &device, &dtype, &like, &optional)) return nullptr;
    if (!(PyList_Check(tensors) || PyTuple_Check(tensors)) ||
        !(like == Py_None || PyList_Check(like) || PyTuple_Check(like)))
        return PyErr_Format(PyExc_TypeError, "%s must be a list of tensors", name);
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(tensors);
    if (like != Py_None && PySequence_Fast_GET_SIZE(like) != n)
        return PyErr_Format(PyExc_ValueError, "%s must be as many as the parameters", name);
    std::vector<uint64_t> ptr(n);
    std::vector<int64_t> numel(n);
    std::vector<int32_t> type(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (optional && PySequence_Fast_GET_ITEM(tensors, i) == Py_None) continue;
        const at::Tensor *t = tensor_at(tensors, i, name);
        if (t == nullptr) return nullptr;
        if (!t->is_cuda() || t->get_device() != device)
            return PyErr_Format(PyExc_ValueError, "%s must be CUDA tensors on one device", name);
        const int code = code_of(t->scalar_type());
        if (code < 0) return PyErr_Format(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
        if (dtype >= 0 && code != dtype) return PyErr_Format(PyExc_TypeError, "%s must be %s", name, kNames[dtype]);
        if (t->layout() != at::kStrided || !(t->is_contiguous() || t->is_non_overlapping_and_dense()))
            return PyErr_Format(PyExc_ValueError, "%s must be dense", name);
        if (like != Py_None) {
            const at::Tensor *o = tensor_at(like, i, "params");
            if (o == nullptr) return nullptr;
            if (t->sizes() != o->sizes())
                return PyErr_Format(PyExc_ValueError, "%s must have the parameters' shapes", name);
            if (!(t->is_contiguous() && o->is_contiguous()) && t->strides() != o->strides())
                return PyErr_Format(PyExc_ValueError, "%s must have the parameters' order in memory", name);
        }
        ptr[i] = reinterpret_cast<uint64_t>(t->data_ptr());
        numel[i] = t->numel();
        type[i] = code;
    }
    // N takes the references over; a null among them (no memory) makes the tuple's error
    return Py_BuildValue("(NNN)", PyBytes_FromStringAndSize(reinterpret_cast<const char *>(ptr.data()), n * 8),
                         PyBytes_FromStringAndSize(reinterpret_cast<const char *>(numel.data()), n * 8),
                         PyBytes_FromStringAndSize(reinterpret_cast<const char *>(type.data()), n * 4));
}

// Exceptions of libtorch (a tensor without storage, for one) end as Python's.
PyObject *gather_guarded(PyObject *self, PyObject *args) {
    try {
        return gather(self, args);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef kMethods[] = {{"gather", gather_guarded, METH_VARARGS, "addresses, counts and types of a list of tensors"},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists(void) { return PyModule_Create(&kModule); }
