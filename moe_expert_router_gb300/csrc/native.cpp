// native.cpp -- the part of the Python binding whose cost on the host shows: the router's
// calls, short enough that a token waits for their argument checks (some 6 us through
// Python and ctypes), and lists of tensors, 0.4 us a tensor through Python's attributes.
// It reads and checks the tensors and calls libmoe's C entry points; nothing else.
//
// CPython module `_native`:
//   bind(moe_route, moe_route_backward, moe_bias_update): the entry points' addresses
//   route / route_backward / bias_update: the calls, from tensors (None where the C call
//       takes NULL), with the address of a moe_router_cfg_t and a stream; their status
//   gather(tensors, name, device, dtype, like, optional, apart)
//       -> (addresses u64, counts i64, types i32) as bytes in the machine's order
//     tensors: list or tuple of torch tensors (with `optional`, or None: address 0)
//     dtype: a MOE_DTYPE_* code that all must have, or -1 for any of them
//     like: a list of tensors whose shapes and order in memory they must have, or None
//     apart: they must not overlap (they are written)
// Raises TypeError / ValueError as the rest of the binding does.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "moe.h"

namespace {

struct Refused {};                          // a Python error is set

decltype(&moe_route) g_route = nullptr;
decltype(&moe_route_backward) g_route_backward = nullptr;
decltype(&moe_bias_update) g_bias_update = nullptr;

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return MOE_DTYPE_F32;
        case at::kBFloat16: return MOE_DTYPE_BF16;
        case at::kHalf: return MOE_DTYPE_F16;
        default: return -1;
    }
}

const char *const kNames[] = {"float32", "bfloat16", "float16"};

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... a) {
    PyErr_Format(type, format, a...);
    throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}

// The address of a dense CUDA tensor of the given type and shape; NULL for None.
void *address(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.sizes() != shape) {
        std::string want, is;
        for (int64_t d : shape) want += std::to_string(d) + ", ";
        for (int64_t d : t.sizes()) is += std::to_string(d) + ", ";
        refuse(PyExc_ValueError, "%s must have shape (%s), not (%s)", name, want.c_str(), is.c_str());
    }
    if (!t.is_cuda()) refuse(PyExc_ValueError, "libmoe takes CUDA tensors only");
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

template <typename T>
T *as(void *p) {
    return static_cast<T *>(p);
}

struct Logits {
    moe_route_shape_t shape;
    const void *ptr;
    at::ScalarType type;
};

Logits logits_of(PyObject *lo, PyObject *io, PyObject *oo) {
    const at::Tensor &l = tensor(lo, "logits");
    const at::Tensor &i = tensor(io, "topk_idx");
    if (l.dim() != 2 || i.dim() != 2) refuse(PyExc_ValueError, "logits must be [T, E] and topk_idx [T, k]");
    const int code = code_of(l.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "logits must be float32, bfloat16 or float16, not %s", c10::toString(l.scalar_type()));
    if (!l.is_cuda()) refuse(PyExc_ValueError, "libmoe takes CUDA tensors only");
    const int64_t T = l.size(0), E = l.size(1);
    if (E > 1 && l.stride(1) != 1) refuse(PyExc_ValueError, "the experts of a row of logits must be consecutive");
    const int64_t ld = T > 1 ? l.stride(0) : E;
    if (ld < E) refuse(PyExc_ValueError, "the rows of logits overlap");
    int64_t S = 1;
    if (oo != Py_None) {
        const at::Tensor &o = tensor(oo, "seq_offsets");
        if (o.dim() != 1 || o.size(0) < 2) refuse(PyExc_ValueError, "seq_offsets must be [S + 1] with S >= 1");
        S = o.size(0) - 1;
    }
    return {{T, E, S, ld, static_cast<int32_t>(i.size(1)), code}, l.data_ptr(), l.scalar_type()};
}

const uint8_t *mask_of(PyObject *o, int64_t T) {
    if (o == Py_None) return nullptr;
    const bool bytes = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kByte;
    return as<const uint8_t>(address(o, "token_mask", bytes ? at::kByte : at::kBool, {T}));
}

void *handle(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Refused();
    return p;
}

// logits, cfg, topk_idx, topk_w, sel_bias, token_mask, seq_offsets, counts, seq_tokens, losses, ws, stream
PyObject *route(PyObject *const *a) {
    const Logits l = logits_of(a[0], a[2], a[6]);
    const moe_route_shape_t &s = l.shape;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (a[10] != Py_None) {
        const at::Tensor &t = tensor(a[10], "ws");
        if (!t.is_cuda() || !t.is_contiguous()) refuse(PyExc_ValueError, "ws must be a contiguous CUDA tensor");
        ws = t.data_ptr();
        ws_bytes = t.nbytes();
    }
    return PyLong_FromLong(g_route(
        l.ptr, as<float>(address(a[4], "sel_bias", at::kFloat, {s.E})), mask_of(a[5], s.T),
        as<int32_t>(address(a[6], "seq_offsets", at::kInt, {s.S + 1})), &s, as<const moe_router_cfg_t>(handle(a[1])),
        as<int32_t>(address(a[2], "topk_idx", at::kInt, {s.T, s.k})),
        as<float>(address(a[3], "topk_w", at::kFloat, {s.T, s.k})),
        as<int32_t>(address(a[7], "counts", at::kInt, {s.S, s.E})),
        as<int32_t>(address(a[8], "seq_tokens", at::kInt, {s.S + 2})),
        as<float>(address(a[9], "losses", at::kFloat, {2})), ws, ws_bytes, handle(a[11])));
}

// logits, cfg, topk_idx, dtopk_w, dlogits, token_mask, seq_offsets, counts, seq_tokens, dlosses, stream
PyObject *route_backward(PyObject *const *a) {
    const Logits l = logits_of(a[0], a[2], a[6]);
    const moe_route_shape_t &s = l.shape;
    return PyLong_FromLong(g_route_backward(
        l.ptr, mask_of(a[5], s.T), as<int32_t>(address(a[6], "seq_offsets", at::kInt, {s.S + 1})), &s,
        as<const moe_router_cfg_t>(handle(a[1])), as<int32_t>(address(a[2], "topk_idx", at::kInt, {s.T, s.k})),
        as<float>(address(a[3], "dtopk_w", at::kFloat, {s.T, s.k})),
        as<int32_t>(address(a[7], "counts", at::kInt, {s.S, s.E})),
        as<int32_t>(address(a[8], "seq_tokens", at::kInt, {s.S + 2})),
        as<float>(address(a[9], "dlosses", at::kFloat, {2})), address(a[4], "dlogits", l.type, {s.T, s.E}),
        handle(a[10])));
}

// bias, counts, rate, stream
PyObject *bias_update(PyObject *const *a) {
    const at::Tensor &b = tensor(a[0], "bias"), &c = tensor(a[1], "counts");
    if (b.dim() < 1 || b.dim() > 2 || c.dim() != b.dim() + 1)
        refuse(PyExc_ValueError, "bias must be [E] and counts [S, E], or [L, E] and [L, S, E]");
    const int64_t L = b.dim() == 1 ? 1 : b.size(0), E = b.size(-1), S = c.size(-2);
    if (c.size(-1) != E || (b.dim() == 2 && c.size(0) != L))
        refuse(PyExc_ValueError, "bias and counts differ in layers or experts");
    const double rate = PyFloat_AsDouble(a[2]);
    if (rate == -1.0 && PyErr_Occurred()) throw Refused();
    return PyLong_FromLong(g_bias_update(as<float>(address(a[0], "bias", at::kFloat, b.sizes())),
                                         as<int32_t>(address(a[1], "counts", at::kInt, c.sizes())), L, S, E,
                                         static_cast<float>(rate), handle(a[3])));
}

PyObject *bind(PyObject *const *a) {
    g_route = reinterpret_cast<decltype(g_route)>(handle(a[0]));
    g_route_backward = reinterpret_cast<decltype(g_route_backward)>(handle(a[1]));
    g_bias_update = reinterpret_cast<decltype(g_bias_update)>(handle(a[2]));
    Py_RETURN_NONE;
}

// tensors, name, device, dtype, like, optional, apart
PyObject *gather(PyObject *const *a) {
    PyObject *list = a[0], *like = a[4];
    const char *name = PyUnicode_AsUTF8(a[1]);
    if (name == nullptr) throw Refused();
    const long device = PyLong_AsLong(a[2]), dtype = PyLong_AsLong(a[3]);
    const bool optional = PyObject_IsTrue(a[5]), apart = PyObject_IsTrue(a[6]);
    if (PyErr_Occurred()) throw Refused();
    if (!(PyList_Check(list) || PyTuple_Check(list)) || !(like == Py_None || PyList_Check(like) || PyTuple_Check(like)))
        refuse(PyExc_TypeError, "%s must be a list of tensors", name);
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
    if (like != Py_None && PySequence_Fast_GET_SIZE(like) != n)
        refuse(PyExc_ValueError, "%s must be as many as the parameters", name);
    std::vector<uint64_t> ptr(n);
    std::vector<int64_t> numel(n);
    std::vector<int32_t> type(n);
    std::vector<std::pair<uint64_t, uint64_t>> range;
    bool sorted = true;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *o = PySequence_Fast_GET_ITEM(list, i);
        if (optional && o == Py_None) continue;
        const at::Tensor &t = tensor(o, name);
        if (!t.is_cuda() || t.get_device() != device) refuse(PyExc_ValueError, "%s must be CUDA tensors on one device", name);
        const int code = code_of(t.scalar_type());
        if (code < 0) refuse(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
        if (dtype >= 0 && code != dtype) refuse(PyExc_TypeError, "%s must be %s", name, kNames[dtype]);
        if (t.layout() != at::kStrided || !(t.is_contiguous() || t.is_non_overlapping_and_dense()))
            refuse(PyExc_ValueError, "%s must be dense", name);
        if (like != Py_None) {
            const at::Tensor &p = tensor(PySequence_Fast_GET_ITEM(like, i), "params");
            if (t.sizes() != p.sizes()) refuse(PyExc_ValueError, "%s must have the parameters' shapes", name);
            if (!(t.is_contiguous() && p.is_contiguous()) && t.strides() != p.strides())
                refuse(PyExc_ValueError, "%s must have the parameters' order in memory", name);
        }
        ptr[i] = reinterpret_cast<uint64_t>(t.data_ptr());
        numel[i] = t.numel();
        type[i] = code;
        if (apart && numel[i] > 0) {
            const uint64_t end = ptr[i] + static_cast<uint64_t>(numel[i]) * (code == MOE_DTYPE_F32 ? 4 : 2);
            sorted = sorted && (range.empty() || range.back().first <= ptr[i]);
            range.emplace_back(ptr[i], end);
        }
    }
    if (!sorted) std::sort(range.begin(), range.end());
    for (size_t i = 1; i < range.size(); ++i)
        if (range[i].first < range[i - 1].second) refuse(PyExc_ValueError, "%s hold the same memory twice", name);
    // N takes the references over; a null among them (no memory) makes the tuple's error
    return Py_BuildValue("(NNN)", PyBytes_FromStringAndSize(reinterpret_cast<const char *>(ptr.data()), n * 8),
                         PyBytes_FromStringAndSize(reinterpret_cast<const char *>(numel.data()), n * 8),
                         PyBytes_FromStringAndSize(reinterpret_cast<const char *>(type.data()), n * 4));
}

// No C++ exception leaves the module: libtorch's (a tensor without storage, for one) end as Python's.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    try {
        return F(args);
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<bind, 3>("bind"),
                          method<route, 12>("route"),
                          method<route_backward, 11>("route_backward"),
                          method<bias_update, 4>("bias_update"),
                          method<gather, 7>("gather"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&kModule); }
