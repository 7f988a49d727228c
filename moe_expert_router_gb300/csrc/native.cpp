// native.cpp -- the part of the Python binding whose cost on the host shows: the router's
// calls, the norm and the grouped products, short enough that a token waits for their argument
// checks (some 6 us through Python and ctypes), and lists of tensors, 0.4 us a tensor through
// Python's attributes.
// It reads and checks the tensors and calls libmoe's C entry points; nothing else.
//
// CPython module `_native`: bind(addresses of the entry points), then the calls of the same
// names, from tensors and lists of tensors (None where the C call takes NULL), the address of
// a configuration, and a stream; they return the call's status. Raises TypeError / ValueError
// as the rest of the binding does.
#define PY_SSIZE_T_CLEAN
#include <ATen/ops/empty.h>
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
decltype(&moe_grad_norm) g_grad_norm = nullptr;
decltype(&moe_clip_grads) g_clip_grads = nullptr;
decltype(&moe_adamw) g_adamw = nullptr;
decltype(&moe_grouped_mm) g_grouped_mm = nullptr;
decltype(&moe_grouped_wgrad) g_grouped_wgrad = nullptr;
decltype(&moe_grouped_mm_mx) g_grouped_mm_mx = nullptr;
decltype(&moe_rms_norm) g_rms_norm = nullptr;
decltype(&moe_rms_norm_backward) g_rms_norm_backward = nullptr;

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

// The operands of a call lie on one device, that of a CUDA tensor `like`.
void together(const at::Tensor &like, const at::Tensor &t) {
    if (t.device() != like.device())
        refuse(PyExc_ValueError, t.is_cuda() ? "tensors must be on one device" : "libmoe takes CUDA tensors only");
}

// The address of a dense tensor of the given type and shape on the device of `like`; NULL for None.
void *address(PyObject *o, const char *name, const at::Tensor &like, at::ScalarType type, at::IntArrayRef shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.sizes() != shape) {
        std::string want, is;
        for (int64_t d : shape) want += std::to_string(d) + ", ";
        for (int64_t d : t.sizes()) is += std::to_string(d) + ", ";
        refuse(PyExc_ValueError, "%s must have shape (%s), not (%s)", name, want.c_str(), is.c_str());
    }
    together(like, t);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

template <typename T>
T *as(void *p) {
    return static_cast<T *>(p);
}

struct Logits {
    moe_route_shape_t shape;
    const at::Tensor &tensor;
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
    return {{T, E, S, ld, static_cast<int32_t>(i.size(1)), code}, l};
}

const uint8_t *mask_of(PyObject *o, const at::Tensor &like, int64_t T) {
    if (o == Py_None) return nullptr;
    const bool bytes = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kByte;
    return as<const uint8_t>(address(o, "token_mask", like, bytes ? at::kByte : at::kBool, {T}));
}

void *handle(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Refused();
    return p;
}

// A call's status for Python; where it succeeded, `bump` moves the version counters of what the
// caller holds and the call has changed in place, as torch's own in-place operations do: a saved
// tensor or a cached copy is seen to be old.
template <typename F>
PyObject *changed(moe_status_t status, F bump) {
    if (status == MOE_OK) bump();
    return PyLong_FromLong(status);
}
void bump(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();     // those have no counter
}

// logits, cfg, topk_idx, topk_w, sel_bias, token_mask, seq_offsets, counts, seq_tokens, losses, ws, stream
PyObject *route(PyObject *const *a) {
    const Logits l = logits_of(a[0], a[2], a[6]);
    const moe_route_shape_t &s = l.shape;
    const at::Tensor &on = l.tensor;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (a[10] != Py_None) {
        const at::Tensor &t = tensor(a[10], "ws");
        together(on, t);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "ws must be contiguous");
        ws = t.data_ptr();
        ws_bytes = t.nbytes();
    }
    return PyLong_FromLong(g_route(
        on.data_ptr(), as<float>(address(a[4], "sel_bias", on, at::kFloat, {s.E})), mask_of(a[5], on, s.T),
        as<int32_t>(address(a[6], "seq_offsets", on, at::kInt, {s.S + 1})), &s, as<const moe_router_cfg_t>(handle(a[1])),
        as<int32_t>(address(a[2], "topk_idx", on, at::kInt, {s.T, s.k})),
        as<float>(address(a[3], "topk_w", on, at::kFloat, {s.T, s.k})),
        as<int32_t>(address(a[7], "counts", on, at::kInt, {s.S, s.E})),
        as<int32_t>(address(a[8], "seq_tokens", on, at::kInt, {s.S + 2})),
        as<float>(address(a[9], "losses", on, at::kFloat, {2})), ws, ws_bytes, handle(a[11])));
}

// logits, cfg, topk_idx, dtopk_w, dlogits, token_mask, seq_offsets, counts, seq_tokens, dlosses, stream
PyObject *route_backward(PyObject *const *a) {
    const Logits l = logits_of(a[0], a[2], a[6]);
    const moe_route_shape_t &s = l.shape;
    const at::Tensor &on = l.tensor;
    return PyLong_FromLong(g_route_backward(
        on.data_ptr(), mask_of(a[5], on, s.T), as<int32_t>(address(a[6], "seq_offsets", on, at::kInt, {s.S + 1})), &s,
        as<const moe_router_cfg_t>(handle(a[1])), as<int32_t>(address(a[2], "topk_idx", on, at::kInt, {s.T, s.k})),
        as<float>(address(a[3], "dtopk_w", on, at::kFloat, {s.T, s.k})),
        as<int32_t>(address(a[7], "counts", on, at::kInt, {s.S, s.E})),
        as<int32_t>(address(a[8], "seq_tokens", on, at::kInt, {s.S + 2})),
        as<float>(address(a[9], "dlosses", on, at::kFloat, {2})), address(a[4], "dlogits", on, on.scalar_type(), {s.T, s.E}),
        handle(a[10])));
}

// bias, counts, rate, stream
PyObject *bias_update(PyObject *const *a) {
    const at::Tensor &b = tensor(a[0], "bias"), &c = tensor(a[1], "counts");
    if (!b.is_cuda()) refuse(PyExc_ValueError, "libmoe takes CUDA tensors only");
    if (b.dim() < 1 || b.dim() > 2 || c.dim() != b.dim() + 1)
        refuse(PyExc_ValueError, "bias must be [E] and counts [S, E], or [L, E] and [L, S, E]");
    const int64_t L = b.dim() == 1 ? 1 : b.size(0), E = b.size(-1), S = c.size(-2);
    if (c.size(-1) != E || (b.dim() == 2 && c.size(0) != L))
        refuse(PyExc_ValueError, "bias and counts differ in layers or experts");
    const double rate = PyFloat_AsDouble(a[2]);
    if (rate == -1.0 && PyErr_Occurred()) throw Refused();
    return changed(g_bias_update(as<float>(address(a[0], "bias", b, at::kFloat, b.sizes())),
                                 as<int32_t>(address(a[1], "counts", b, at::kInt, c.sizes())), L, S, E,
                                 static_cast<float>(rate), handle(a[3])),
                   [&] { bump(b); });
}

// A list's addresses, element counts and types, checked: dense CUDA tensors on one device,
// of the type `dtype` (-1: any of the three); like those of `like` in shape and order in
// memory, where that is not null; with `optional` or None (address 0); not overlapping,
// where they are written.
using Range = std::pair<uint64_t, uint64_t>;  // of addresses, the end not among them
struct List {
    const char *name;
    bool written;
    std::vector<const at::Tensor *> tensor;   // borrowed from the caller's list
    std::vector<void *> ptr;
    std::vector<int64_t> numel;
    std::vector<int32_t> type;
    std::vector<Range> range;                 // of the tensors that are not empty, in order
    uint64_t end;                             // the largest of theirs
};
// A thread's lists keep their memory from call to call, nothing of what is in them.
thread_local List t_lists[5];

bool is_list(PyObject *o) { return PyList_Check(o) || PyTuple_Check(o); }

const List &list_of(List &l, PyObject *o, const char *name, int device, int dtype, const List *like, bool optional,
                    bool written) {
    if (!is_list(o)) refuse(PyExc_TypeError, "%s must be a list of tensors", name);
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    if (like != nullptr && static_cast<Py_ssize_t>(like->tensor.size()) != n)
        refuse(PyExc_ValueError, "%s must be as many as the parameters", name);
    l.name = name;
    l.written = written;
    l.tensor.assign(n, nullptr);
    l.ptr.assign(n, nullptr);
    l.numel.assign(n, 0);
    l.type.assign(n, MOE_DTYPE_F32);
    const at::Device on(at::kCUDA, static_cast<at::DeviceIndex>(device));
    std::vector<Range> &range = l.range;
    range.clear();
    l.end = 0;
    bool sorted = true;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *item = PySequence_Fast_GET_ITEM(o, i);
        if (optional && item == Py_None) continue;
        const at::Tensor &t = tensor(item, name);
        if (t.device() != on) refuse(PyExc_ValueError, "%s must be CUDA tensors on one device", name);
        const int code = code_of(t.scalar_type());
        if (code < 0) refuse(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
        if (dtype >= 0 && code != dtype) refuse(PyExc_TypeError, "%s must be %s", name, kNames[dtype]);
        if (t.layout() != at::kStrided) refuse(PyExc_ValueError, "%s must be dense", name);
        const bool plain = t.is_contiguous();
        if (!plain && !t.is_non_overlapping_and_dense()) refuse(PyExc_ValueError, "%s must be dense", name);
        if (like != nullptr) {
            const at::Tensor &p = *like->tensor[i];
            if (t.sizes() != p.sizes()) refuse(PyExc_ValueError, "%s must have the parameters' shapes", name);
            if (!(plain && p.is_contiguous()) && t.strides() != p.strides())
                refuse(PyExc_ValueError, "%s must have the parameters' order in memory", name);
        }
        l.tensor[i] = &t;
        l.ptr[i] = t.data_ptr();
        l.numel[i] = t.numel();
        l.type[i] = code;
        if (l.numel[i] > 0) {
            const uint64_t at = reinterpret_cast<uint64_t>(l.ptr[i]);
            sorted = sorted && (range.empty() || range.back().first <= at);
            range.emplace_back(at, at + static_cast<uint64_t>(l.numel[i]) * (code == MOE_DTYPE_F32 ? 4 : 2));
            l.end = std::max(l.end, range.back().second);
        }
    }
    if (!sorted) std::sort(range.begin(), range.end());
    for (size_t i = 1; written && i < range.size(); ++i)
        if (range[i].first < range[i - 1].second) refuse(PyExc_ValueError, "%s hold the same memory twice", name);
    return l;
}

// What a call writes lies in none of its other operands: blocks would read it while others write.
void apart(const List &a, const List &b) {
    if (!a.written && !b.written) return;
    if (a.range.empty() || b.range.empty() || a.end <= b.range.front().first || b.end <= a.range.front().first) return;
    uint64_t a_end = 0, b_end = 0;            // as far as they have been walked
    for (size_t i = 0, j = 0; i < a.range.size() || j < b.range.size();) {
        const bool first = j == b.range.size() || (i < a.range.size() && a.range[i].first < b.range[j].first);
        const Range &r = first ? a.range[i++] : b.range[j++];
        if (r.first < (first ? b_end : a_end)) refuse(PyExc_ValueError, "%s and %s hold the same memory", a.name, b.name);
        uint64_t &end = first ? a_end : b_end;
        end = std::max(end, r.second);
    }
}
void apart(const List &l, const void *ptr, size_t bytes, const char *name, bool written) {
    const uint64_t at = reinterpret_cast<uint64_t>(ptr), end = at + bytes;
    if (ptr == nullptr || !(written || l.written) || l.range.empty() || l.end <= at || end <= l.range.front().first) return;
    for (const Range &r : l.range)
        if (r.first < end && at < r.second) refuse(PyExc_ValueError, "%s and %s hold the same memory", l.name, name);
}

void bump(const List &l) {
    for (const at::Tensor *t : l.tensor)
        if (t != nullptr) bump(*t);
}

struct Scratch {
    void *ptr;
    size_t bytes;
};
Scratch scratch(PyObject *o, const at::Tensor &like) {
    const at::Tensor &t = tensor(o, "ws");
    together(like, t);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "ws must be contiguous");
    return {t.data_ptr(), t.nbytes()};
}

// The address of the fp32 number that a norm goes to (any shape of one element); NULL for None.
float *number(PyObject *o, const char *name, const at::Tensor &like) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "%s must be Float, not %s", name, c10::toString(t.scalar_type()));
    if (t.numel() != 1) refuse(PyExc_ValueError, "%s must have one element", name);
    together(like, t);
    return static_cast<float *>(t.data_ptr());
}

int device_of(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) refuse(PyExc_ValueError, "libmoe takes CUDA tensors only");
    return t.get_device();
}

long whole(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

// grads, norm_type, norm, ws, stream
PyObject *grad_norm(PyObject *const *a) {
    const List &g = list_of(t_lists[0], a[0], "grads", device_of(a[2], "norm"), -1, nullptr, false, false);
    const at::Tensor &on = tensor(a[2], "norm");
    const Scratch ws = scratch(a[3], on);
    float *norm = number(a[2], "norm", on);
    apart(g, norm, 4, "norm", true);
    apart(g, ws.ptr, ws.bytes, "ws", true);
    return PyLong_FromLong(g_grad_norm(g.ptr.data(), g.numel.data(), g.type.data(), static_cast<int32_t>(g.ptr.size()),
                                       static_cast<int32_t>(whole(a[1])), norm, ws.ptr, ws.bytes, handle(a[4])));
}

// grads, norm_type, max_norm, norm, ws, stream
PyObject *clip_grads(PyObject *const *a) {
    const List &g = list_of(t_lists[0], a[0], "grads", device_of(a[3], "norm"), -1, nullptr, false, true);
    const at::Tensor &on = tensor(a[3], "norm");
    const Scratch ws = scratch(a[4], on);
    float *norm = number(a[3], "norm", on);
    apart(g, norm, 4, "norm", true);
    apart(g, ws.ptr, ws.bytes, "ws", true);
    const double most = PyFloat_AsDouble(a[2]);
    if (most == -1.0 && PyErr_Occurred()) throw Refused();
    return changed(g_clip_grads(g.ptr.data(), g.numel.data(), g.type.data(), static_cast<int32_t>(g.ptr.size()),
                                static_cast<int32_t>(whole(a[1])), static_cast<float>(most),
                                norm, ws.ptr, ws.bytes, handle(a[5])),
                   [&] { bump(g); });
}

// params, grads, exp_avg, exp_avg_sq, masters, cfg, lr, step, norm, ws, missed, stream
PyObject *adamw(PyObject *const *a) {
    const int device = device_of(a[6], "lr");
    const List &p = list_of(t_lists[0], a[0], "params", device, -1, nullptr, false, true);
    const List &g = list_of(t_lists[1], a[1], "grads", device, -1, &p, false, false);
    const List &m = list_of(t_lists[2], a[2], "exp_avg", device, MOE_DTYPE_F32, &p, false, true);
    const List &v = list_of(t_lists[3], a[3], "exp_avg_sq", device, MOE_DTYPE_F32, &p, false, true);
    const List *x = a[4] != Py_None ? &list_of(t_lists[4], a[4], "masters", device, MOE_DTYPE_F32, &p, true, true) : nullptr;
    const at::Tensor &on = tensor(a[6], "lr");
    const Scratch ws = scratch(a[9], on);
    const int64_t n = static_cast<int64_t>(p.ptr.size());
    float *lr = as<float>(address(a[6], "lr", on, at::kFloat, {1})), *norm = number(a[8], "norm", on);
    int32_t *step = as<int32_t>(address(a[7], "step", on, at::kInt, {1}));
    moe_adamw_cfg_t cfg = *as<const moe_adamw_cfg_t>(handle(a[5]));
    cfg.missed = as<const int32_t>(address(a[10], "missed", on, at::kInt, {n}));
    const List *const lists[] = {&p, &g, &m, &v, x};
    for (int i = 0; i < 5 && lists[i] != nullptr; ++i) {
        for (int j = 0; j < i; ++j) apart(*lists[j], *lists[i]);
        apart(*lists[i], lr, 4, "lr", false);
        apart(*lists[i], step, 4, "step", true);
        apart(*lists[i], norm, 4, "norm", true);
        apart(*lists[i], ws.ptr, ws.bytes, "ws", true);
        apart(*lists[i], cfg.missed, 4 * static_cast<size_t>(n), "missed", false);
    }
    auto floats = [](const List &l) { return reinterpret_cast<float *const *>(l.ptr.data()); };
    return changed(g_adamw(p.ptr.data(), p.type.data(), g.ptr.data(), g.type.data(), floats(m), floats(v),
                           x != nullptr ? floats(*x) : nullptr, p.numel.data(), static_cast<int32_t>(p.ptr.size()),
                           &cfg, lr, step, norm, ws.ptr, ws.bytes, handle(a[11])),
                   // not the optimizer's own state, which no graph saves: 10 ns each, 3 us of a call's 32 for 120 parameters
                   [&] { bump(p); });
}

// bytes, like: a workspace on that tensor's device, and an fp32 number at its end
PyObject *scratch_with_norm(PyObject *const *a) {
    const at::Tensor &like = tensor(a[1], "tensors");
    at::Tensor ws = at::empty({whole(a[0]) / 4 + 4}, at::TensorOptions().device(like.device()).dtype(at::kFloat));
    at::Tensor norm = ws.select(0, -1);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(ws)), THPVariable_Wrap(std::move(norm)));
}

// A matrix of `rows` x `cols` whose columns are consecutive: rows may lie apart.
struct Rows {
    const at::Tensor &tensor;
    const char *name;
    void *ptr;
    int64_t rows, cols, ld;
};
Rows rows_of(PyObject *o, const char *name, const at::Tensor *like, int64_t rows, int64_t cols) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2) refuse(PyExc_ValueError, "%s must have two dimensions", name);
    if (!t.is_cuda()) refuse(PyExc_ValueError, "libmoe takes CUDA tensors only");
    if (like != nullptr) {
        together(*like, t);
        if (t.scalar_type() != like->scalar_type())
            refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(like->scalar_type()), c10::toString(t.scalar_type()));
    }
    const int64_t r = t.size(0), c = t.size(1);
    if ((rows >= 0 && r != rows) || (cols >= 0 && c != cols))
        refuse(PyExc_ValueError, "%s must have shape (%lld, %lld), not (%lld, %lld)", name, static_cast<long long>(rows >= 0 ? rows : r),
               static_cast<long long>(cols >= 0 ? cols : c), static_cast<long long>(r), static_cast<long long>(c));
    if (c > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "the columns of %s must be consecutive", name);
    const int64_t ld = r > 1 ? t.stride(0) : c;
    if (ld < c) refuse(PyExc_ValueError, "the rows of %s overlap", name);
    return {t, name, t.data_ptr(), r, c, ld};
}

// What a call writes lies in none of its other operands. Rows of one wide tensor's columns, as far
// apart as the other's, interleave without meeting.
bool meet(const void *a, int64_t rows_a, int64_t run_a, int64_t ld_a, const void *b, int64_t rows_b, int64_t run_b, int64_t ld_b) {
    if (a == nullptr || b == nullptr || rows_a <= 0 || rows_b <= 0 || run_a <= 0 || run_b <= 0) return false;
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    if (d >= (rows_a - 1) * ld_a + run_a || -d >= (rows_b - 1) * ld_b + run_b) return false;
    if (rows_a > 1 && rows_b > 1 && ld_a != ld_b) return true;
    const int64_t ld = rows_a > 1 ? ld_a : rows_b > 1 ? ld_b : 0;
    if (ld == 0) return true;
    const int64_t at = ((d % ld) + ld) % ld;                            // of b's run in a's row
    return at < run_a || at + run_b > ld;
}
void apart(const Rows &w, const Rows &r) {
    const int64_t size = w.tensor.element_size(), other = r.tensor.element_size();
    if (meet(w.ptr, w.rows, w.cols * size, w.ld * size, r.ptr, r.rows, r.cols * other, r.ld * other))
        refuse(PyExc_ValueError, "%s and %s hold the same memory", w.name, r.name);
}
void apart(const Rows &w, const at::Tensor &t, const char *name) {
    const int64_t size = w.tensor.element_size(), bytes = static_cast<int64_t>(t.nbytes());
    if (t.numel() > 0 && meet(w.ptr, w.rows, w.cols * size, w.ld * size, t.data_ptr(), 1, bytes, bytes))
        refuse(PyExc_ValueError, "%s and %s hold the same memory", w.name, name);
}
void apart(const at::Tensor &w, const char *name, const Rows &r) {
    const int64_t size = r.tensor.element_size(), bytes = static_cast<int64_t>(w.nbytes());
    if (w.numel() > 0 && meet(w.data_ptr(), 1, bytes, bytes, r.ptr, r.rows, r.cols * size, r.ld * size))
        refuse(PyExc_ValueError, "%s and %s hold the same memory", name, r.name);
}
void apart(const at::Tensor &w, const char *name, const at::Tensor &t, const char *other) {
    const int64_t bytes = static_cast<int64_t>(w.nbytes()), more = static_cast<int64_t>(t.nbytes());
    if (bytes > 0 && more > 0 && meet(w.data_ptr(), 1, bytes, bytes, t.data_ptr(), 1, more, more))
        refuse(PyExc_ValueError, "%s and %s hold the same memory", name, other);
}

// A dense tensor with group matrices [G, rows, cols] (-1: any).
const at::Tensor &matrices_of(PyObject *o, const char *name, const at::Tensor &like, at::ScalarType type, int64_t rows, int64_t cols) {
    const at::Tensor &t = tensor(o, name);
    together(like, t);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.dim() != 3 || (rows >= 0 && t.size(1) != rows) || (cols >= 0 && t.size(2) != cols))
        refuse(PyExc_ValueError, "%s must be a matrix for each group that fits the other operands", name);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

const int32_t *offsets_of(PyObject *o, const at::Tensor &like, int64_t G) {
    return as<const int32_t>(address(o, "offsets", like, at::kInt, {G + 1}));
}

int grouped_type(const at::Tensor &t, const char *name) {
    const int code = code_of(t.scalar_type());
    if (code != MOE_DTYPE_BF16 && code != MOE_DTYPE_F16)
        refuse(PyExc_TypeError, "%s must be bfloat16 or float16, not %s", name, c10::toString(t.scalar_type()));
    return code;
}

// x, w, offsets, out, ws, transposed, nan_on_bad, stream
PyObject *grouped_mm(PyObject *const *a) {
    const Rows x = rows_of(a[0], "x", nullptr, -1, -1);
    const at::Tensor &on = x.tensor;
    const int code = grouped_type(on, "x");
    const bool kn = whole(a[5]) != 0;
    const at::Tensor &w = matrices_of(a[1], "w", on, on.scalar_type(), kn ? x.cols : -1, kn ? -1 : x.cols);
    const int64_t G = w.size(0), N = w.size(kn ? 2 : 1);
    const Rows out = rows_of(a[3], "out", &on, x.rows, N);
    const int32_t *offsets = offsets_of(a[2], on, G);
    const Scratch ws = scratch(a[4], on);
    apart(out, x);
    apart(out, w, "w");
    apart(out, THPVariable_Unpack(a[2]), "offsets");
    apart(out, THPVariable_Unpack(a[4]), "ws");
    const moe_grouped_shape_t s{x.rows, G, x.cols, N, x.ld, out.ld, code,
                                (kn ? MOE_GROUPED_W_KN : 0) | (whole(a[6]) != 0 ? MOE_GROUPED_NAN_ON_BAD : 0)};
    return changed(g_grouped_mm(x.ptr, w.data_ptr(), offsets, &s, out.ptr, ws.ptr, ws.bytes, handle(a[7])),
                   [&] { bump(out.tensor); });
}

// a, b, offsets, dw, ws, nan_on_bad, stream
PyObject *grouped_wgrad(PyObject *const *a) {
    const Rows l = rows_of(a[0], "a", nullptr, -1, -1);
    const at::Tensor &on = l.tensor;
    const int code = grouped_type(on, "a");
    const Rows r = rows_of(a[1], "b", &on, l.rows, -1);
    const at::Tensor &dw = matrices_of(a[3], "dw", on, on.scalar_type(), l.cols, r.cols);
    const int64_t G = dw.size(0);
    const int32_t *offsets = offsets_of(a[2], on, G);
    const Scratch ws = scratch(a[4], on);
    apart(dw, "dw", l);
    apart(dw, "dw", r);
    apart(dw, "dw", THPVariable_Unpack(a[2]), "offsets");
    apart(dw, "dw", THPVariable_Unpack(a[4]), "ws");
    const moe_grouped_shape_t s{l.rows, G, r.cols, l.cols, r.ld, l.ld, code, whole(a[5]) != 0 ? MOE_GROUPED_NAN_ON_BAD : 0};
    return changed(g_grouped_wgrad(l.ptr, r.ptr, offsets, &s, dw.data_ptr(), ws.ptr, ws.bytes, handle(a[6])), [&] { bump(dw); });
}

// x_codes, x_scales, w_codes, w_scales, offsets, out, ws, stream
PyObject *grouped_mm_mx(PyObject *const *a) {
    const Rows x = rows_of(a[0], "x_codes", nullptr, -1, -1);
    const at::Tensor &on = x.tensor;
    if (on.scalar_type() != at::kByte) refuse(PyExc_TypeError, "x_codes must be Byte, not %s", c10::toString(on.scalar_type()));
    if (!on.is_contiguous()) refuse(PyExc_ValueError, "x_codes must be contiguous");
    const at::Tensor &w = matrices_of(a[2], "w_codes", on, at::kByte, -1, x.cols);
    const int64_t G = w.size(0), N = w.size(1);
    auto words = [&](PyObject *o, const char *name, int64_t rows) {
        const at::Tensor &t = tensor(o, name);
        together(on, t);
        if (t.scalar_type() != at::kByte) refuse(PyExc_TypeError, "%s must be Byte, not %s", name, c10::toString(t.scalar_type()));
        if (!t.is_contiguous() || t.numel() != (rows + 3) / 4 * 4 * (x.cols / 32))
            refuse(PyExc_ValueError, "%s must hold the k-block-major words of its rows rounded up to 4", name);
        return t.data_ptr();
    };
    const void *xs = words(a[1], "x_scales", x.rows), *ws_w = words(a[3], "w_scales", G * N);
    const at::Tensor &o = tensor(a[5], "out");
    if (o.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "out must be BFloat16, not %s", c10::toString(o.scalar_type()));
    together(on, o);
    const Rows out = rows_of(a[5], "out", nullptr, x.rows, N);
    const int32_t *offsets = offsets_of(a[4], on, G);
    const Scratch ws = scratch(a[6], on);
    for (int i = 0; i < 5; ++i) apart(out, THPVariable_Unpack(a[i]), i == 4 ? "offsets" : i < 2 ? "x" : "w");
    apart(out, THPVariable_Unpack(a[6]), "ws");
    const moe_grouped_shape_t s{x.rows, G, x.cols, N, x.ld, out.ld, MOE_DTYPE_BF16, 0};
    return changed(g_grouped_mm_mx(x.ptr, xs, w.data_ptr(), ws_w, offsets, &s, out.ptr, ws.ptr, ws.bytes, handle(a[7])),
                   [&] { bump(out.tensor); });
}

// The weight of a norm over H columns, of the rows' type or fp32; its MOE_DTYPE_*.
int norm_weight(PyObject *o, const char *name, const at::Tensor &on, int64_t H, void **ptr) {
    const at::Tensor &w = tensor(o, name);
    const at::ScalarType type = w.scalar_type() == at::kFloat ? at::kFloat : on.scalar_type();
    *ptr = address(o, name, on, type, {H});
    return code_of(type);
}
double number_of(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
// A dense [T, H] operand of the type of `on`; none where it is None.
Rows dense(PyObject *o, const char *name, const at::Tensor &on, int64_t T, int64_t H) {
    if (o == Py_None) return {on, name, nullptr, 0, 0, 0};
    Rows r = rows_of(o, name, &on, T, H);
    if (r.rows > 1 && r.ld != H) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return r;
}
// A written operand is apart from a read one or in its very place.
void apart_or_same(const Rows &w, const Rows &r) {
    if (w.ptr == nullptr || r.ptr == nullptr || (w.ptr == r.ptr && w.ld == r.ld)) return;
    apart(w, r);
}
void apart_if(const Rows &w, PyObject *o, const char *name) {
    if (w.ptr != nullptr && o != Py_None) apart(w, THPVariable_Unpack(o), name);
}

// x, weight, y, eps, residual, h, rstd, codes, scales, stream
PyObject *rms_norm(PyObject *const *a) {
    const Rows x = rows_of(a[0], "x", nullptr, -1, -1);
    const at::Tensor &on = x.tensor;
    const int code = code_of(on.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "x must be float32, bfloat16 or float16, not %s", c10::toString(on.scalar_type()));
    const int64_t T = x.rows, H = x.cols;
    void *weight;
    const int w_code = norm_weight(a[1], "weight", on, H, &weight);
    const Rows residual = a[4] == Py_None ? Rows{on, "residual", nullptr, 0, 0, 0} : rows_of(a[4], "residual", &on, T, H);
    const Rows y = dense(a[2], "y", on, T, H), h = dense(a[5], "h", on, T, H);
    float *rstd = as<float>(address(a[6], "rstd", on, at::kFloat, {T}));
    void *codes = address(a[7], "codes", on, at::kByte, {T, H}), *scales = nullptr;
    if (a[8] != Py_None) {
        const at::Tensor &s = tensor(a[8], "scales");
        together(on, s);
        if (s.scalar_type() != at::kByte) refuse(PyExc_TypeError, "scales must be Byte, not %s", c10::toString(s.scalar_type()));
        if (!s.is_contiguous() || s.numel() != (T + 3) / 4 * 4 * (H / 32))
            refuse(PyExc_ValueError, "scales must hold the k-block-major words of T rounded up to 4");
        scales = s.data_ptr();
    }
    for (const Rows *w : {&y, &h}) {
        apart_or_same(*w, x);
        apart_or_same(*w, residual);
        for (int i : {1, 6, 7, 8}) apart_if(*w, a[i], i == 1 ? "weight" : i == 6 ? "rstd" : i == 7 ? "codes" : "scales");
    }
    if (y.ptr != nullptr && h.ptr != nullptr) apart(y, h);
    static const char *const names[] = {"rstd", "codes", "scales"};
    for (int i : {6, 7, 8}) {
        if (a[i] == Py_None) continue;
        const at::Tensor &w = THPVariable_Unpack(a[i]);
        apart(w, names[i - 6], x);
        if (residual.ptr != nullptr) apart(w, names[i - 6], residual);
        apart(w, names[i - 6], THPVariable_Unpack(a[1]), "weight");
        for (int j = 6; j < i; ++j)
            if (a[j] != Py_None) apart(w, names[i - 6], THPVariable_Unpack(a[j]), names[j - 6]);
    }
    const moe_norm_shape_t s{T, H, x.ld, residual.ptr != nullptr ? residual.ld : H, number_of(a[3]), code, w_code};
    return changed(g_rms_norm(x.ptr, residual.ptr, weight, &s, h.ptr, y.ptr, rstd, codes, scales, handle(a[9])), [&] {
        for (int i : {2, 5, 6, 7, 8})
            if (a[i] != Py_None) bump(THPVariable_Unpack(a[i]));
    });
}

// dy, h, weight, rstd, dx, dweight, ws, dh, stream
PyObject *rms_norm_backward(PyObject *const *a) {
    const Rows h = rows_of(a[1], "h", nullptr, -1, -1);
    const at::Tensor &on = h.tensor;
    const int code = code_of(on.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "h must be float32, bfloat16 or float16, not %s", c10::toString(on.scalar_type()));
    const int64_t T = h.rows, H = h.cols;
    void *weight;
    const int w_code = norm_weight(a[2], "weight", on, H, &weight);
    const Rows dy = dense(a[0], "dy", on, T, H), dh = dense(a[7], "dh", on, T, H), dx = dense(a[4], "dx", on, T, H);
    const float *rstd = as<const float>(address(a[3], "rstd", on, at::kFloat, {T}));
    void *dweight = address(a[5], "dweight", on, w_code == MOE_DTYPE_F32 ? at::kFloat : on.scalar_type(), {H});
    const Scratch ws = scratch(a[6], on);
    apart_or_same(dx, dy);
    apart_or_same(dx, dh);
    if (dx.ptr != nullptr) apart(dx, h);
    for (int i : {2, 3, 5, 6}) apart_if(dx, a[i], i == 2 ? "weight" : i == 3 ? "rstd" : i == 5 ? "dweight" : "ws");
    for (int i : {5, 6}) {
        if (a[i] == Py_None) continue;
        const at::Tensor &w = THPVariable_Unpack(a[i]);
        const char *name = i == 5 ? "dweight" : "ws";
        apart(w, name, h);
        if (dy.ptr != nullptr) apart(w, name, dy);
        if (dh.ptr != nullptr) apart(w, name, dh);
        apart(w, name, THPVariable_Unpack(a[2]), "weight");
        if (a[3] != Py_None) apart(w, name, THPVariable_Unpack(a[3]), "rstd");
        if (i == 6 && a[5] != Py_None) apart(w, name, THPVariable_Unpack(a[5]), "dweight");
    }
    const moe_norm_shape_t s{T, H, h.ld, H, 1.0, code, w_code};
    return changed(g_rms_norm_backward(dy.ptr, dh.ptr, h.ptr, weight, rstd, &s, dx.ptr, dweight, ws.ptr, ws.bytes, handle(a[8])),
                   [&] {
                       for (int i : {4, 5})
                           if (a[i] != Py_None) bump(THPVariable_Unpack(a[i]));
                   });
}

PyObject *bind(PyObject *const *a) {
    g_route = reinterpret_cast<decltype(g_route)>(handle(a[0]));
    g_route_backward = reinterpret_cast<decltype(g_route_backward)>(handle(a[1]));
    g_bias_update = reinterpret_cast<decltype(g_bias_update)>(handle(a[2]));
    g_grad_norm = reinterpret_cast<decltype(g_grad_norm)>(handle(a[3]));
    g_clip_grads = reinterpret_cast<decltype(g_clip_grads)>(handle(a[4]));
    g_adamw = reinterpret_cast<decltype(g_adamw)>(handle(a[5]));
    g_grouped_mm = reinterpret_cast<decltype(g_grouped_mm)>(handle(a[6]));
    g_grouped_wgrad = reinterpret_cast<decltype(g_grouped_wgrad)>(handle(a[7]));
    g_grouped_mm_mx = reinterpret_cast<decltype(g_grouped_mm_mx)>(handle(a[8]));
    g_rms_norm = reinterpret_cast<decltype(g_rms_norm)>(handle(a[9]));
    g_rms_norm_backward = reinterpret_cast<decltype(g_rms_norm_backward)>(handle(a[10]));
    Py_RETURN_NONE;
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

PyMethodDef kMethods[] = {method<bind, 11>("bind"),
                          method<route, 12>("route"),
                          method<route_backward, 11>("route_backward"),
                          method<bias_update, 4>("bias_update"),
                          method<grad_norm, 5>("grad_norm"),
                          method<clip_grads, 6>("clip_grads"),
                          method<adamw, 12>("adamw"),
                          method<scratch_with_norm, 2>("scratch"),
                          method<grouped_mm, 8>("grouped_mm"),
                          method<grouped_wgrad, 7>("grouped_wgrad"),
                          method<grouped_mm_mx, 8>("grouped_mm_mx"),
                          method<rms_norm, 10>("rms_norm"),
                          method<rms_norm_backward, 9>("rms_norm_backward"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&kModule); }
