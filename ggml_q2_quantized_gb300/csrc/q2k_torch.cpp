// The quick way from PyTorch tensors to the feed-forward calls of libq2k.
//
// A call of a few microseconds on the GPU is bound by the host: through ctypes a
// gated block takes 12 us to issue and a projection with adapters 22, of which the
// library's own launches are 3 and 7.  This module reads the tensors and allocates
// the outputs and the workspace (from PyTorch's allocator) in C++.  It handles the
// ordinary call only - contiguous tensors of the right types and shapes on the
// current device - and returns None for any other, which the Python layer then
// checks and refuses, or runs, itself.
//
// Each function returns None (not handled), an int (the library's status, not 0)
// or its outputs.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "q2k.h"

namespace {

using at::Tensor;

// libq2k's functions, from the library that Python loaded.
struct Calls {
    decltype(&q2k_gated_ffn) gated;
    decltype(&q2k_gated_ffn_workspace_bytes) gated_bytes;
    decltype(&q2k_gated_ffn_backward) backward;
    decltype(&q2k_gated_ffn_backward_workspace_bytes) backward_bytes;
    decltype(&q2k_matmul_lora) lora;
    decltype(&q2k_matmul_lora_workspace_bytes) lora_bytes;
    decltype(&q2k_linear) linear;
    decltype(&q2k_linear_workspace_bytes) linear_bytes;
    decltype(&q2k_linear_backward) linear_backward;
    decltype(&q2k_linear_backward_workspace_bytes) linear_backward_bytes;
    decltype(&q2k_gated_ffn_experts) gated_experts;
    decltype(&q2k_gated_ffn_experts_workspace_bytes) gated_experts_bytes;
    decltype(&q2k_gated_ffn_experts_backward) experts_backward;
    decltype(&q2k_gated_ffn_experts_backward_workspace_bytes) experts_backward_bytes;
    decltype(&q2k_moe_route) route;
    decltype(&q2k_moe_sort) sort;
    decltype(&q2k_moe_sort_backward) sort_backward;
    decltype(&q2k_moe_combine) combine;
    decltype(&q2k_moe_combine_backward) combine_backward;
} calls;

// A contiguous tensor of a type and number of dimensions on `device` (-1: any), or
// nullptr.
const Tensor* take(PyObject* o, c10::ScalarType type, int dims, int device) {
    if (!THPVariable_Check(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || !t.is_contiguous()) return nullptr;
    if ((dims >= 0 && t.dim() != dims) || (device >= 0 && t.get_device() != device)) return nullptr;
    return &t;
}

// Activations: f32 or bf16 [rows, columns] on the current device.
const Tensor* take_activations(PyObject* o) {
    if (!THPVariable_Check(o)) return nullptr;
    const c10::ScalarType type = THPVariable_Unpack(o).scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) return nullptr;
    const Tensor* t = take(o, type, 2, -1);
    if (t == nullptr || t->get_device() != c10::cuda::current_device()) return nullptr;
    return t->size(0) <= INT_MAX && t->size(1) <= INT_MAX ? t : nullptr;
}

bool take_size(PyObject* o, uint32_t& out) {
    if (!PyLong_Check(o)) return false;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    if (v < 0 || v > INT_MAX) return false;
    out = static_cast<uint32_t>(v);
    return true;
}

bool take_name(PyObject* o, std::initializer_list<const char*> names, int& out) {
    if (!PyUnicode_Check(o)) return false;
    out = 0;
    for (const char* name : names) {
        if (PyUnicode_CompareWithASCIIString(o, name) == 0) return true;
        ++out;
    }
    return false;
}
bool take_path(PyObject* o, q2k_path& path) {
    int i = 0;
    if (!take_name(o, {"auto", "gemv", "tensor"}, i)) return false;
    path = i == 0 ? Q2K_PATH_AUTO : i == 1 ? Q2K_PATH_GEMV : Q2K_PATH_TENSOR;
    return true;
}
bool take_act(PyObject* o, uint32_t& act) {
    int i = 0;
    if (!take_name(o, {"silu", "gelu"}, i)) return false;
    act = i == 0 ? Q2K_ACT_SILU : Q2K_ACT_GELU;
    return true;
}

// An activation's name, or None.
bool take_linear_act(PyObject* o, uint32_t& act) {
    act = Q2K_ACT_NONE;
    return o == Py_None || take_act(o, act);
}

// A tensor or None (then `out` is null); false for anything else.
bool take_optional(PyObject* o, c10::ScalarType type, int dims, int device, const Tensor*& out) {
    out = o == Py_None ? nullptr : take(o, type, dims, device);
    return o == Py_None || out != nullptr;
}

// The offsets of a call's segments, or None: their address and how many segments.
bool take_offsets(PyObject* o, int device, const int32_t*& offsets, uint32_t& experts) {
    const Tensor* t;
    if (!take_optional(o, at::kInt, 1, device, t)) return false;
    offsets = nullptr;
    experts = 0;
    if (t == nullptr) return true;
    if (t->size(0) < 2 || t->size(0) > INT_MAX) return false;
    offsets = t->const_data_ptr<int32_t>();
    experts = static_cast<uint32_t>(t->size(0) - 1);
    return true;
}

void* at_or_null(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const void* at_or_null(const Tensor* t) { return t != nullptr ? t->const_data_ptr() : nullptr; }

uint32_t code(const Tensor& t) { return t.scalar_type() == at::kFloat ? Q2K_DTYPE_F32 : Q2K_DTYPE_BF16; }

struct Workspace {
    Tensor hold;
    void* at = nullptr;
    size_t bytes;
    Workspace(size_t need, const Tensor& like) : bytes(need) {
        if (need == 0) return;
        hold = at::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
        at = hold.data_ptr();
    }
};

// The interpreter's lock is free while this lives, also where an exception ends it.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename Call>
PyObject* finish(Call&& call, const Tensor& like, std::initializer_list<Tensor> outs) {
    const q2k_stream_t stream =
        reinterpret_cast<q2k_stream_t>(c10::cuda::getCurrentCUDAStream(like.get_device()).stream());
    int status;
    {
        const Unlocked unlocked;
        status = static_cast<int>(call(stream));
    }
    if (status != 0) return PyLong_FromLong(status);
    if (outs.size() == 1) return THPVariable_Wrap(*outs.begin());
    PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
    if (all == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : outs) {
        PyObject* o = THPVariable_Wrap(t);
        if (o == nullptr) {
            Py_DECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, i++, o);
    }
    return all;
}

// C++ exceptions (the allocator's) become Python's.
template <typename Body>
PyObject* guarded(Body&& body) {
    try {
        return body();
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type != nullptr ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// gated(x, w_gate, w_up, n, act, save, path, const_weights[, offsets])
PyObject* gated(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 8 && count != 9) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_gated_ffn_params p = {};
        q2k_path path;
        const Tensor* x = take_activations(v[0]);
        if (x == nullptr) Py_RETURN_NONE;
        const int device = x->get_device();
        const Tensor *wg = take(v[1], at::kByte, -1, device), *wu = take(v[2], at::kByte, -1, device);
        const int save = PyObject_IsTrue(v[5]), constant = PyObject_IsTrue(v[7]);
        const int32_t* offsets = nullptr;
        uint32_t experts = 0;
        if (wg == nullptr || wu == nullptr || !take_size(v[3], p.n) || !take_act(v[4], p.act) ||
            !take_path(v[6], path) || save < 0 || constant < 0 ||
            (count == 9 && !take_offsets(v[8], device, offsets, experts))) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        p.m = static_cast<uint32_t>(x->size(0));
        p.k = static_cast<uint32_t>(x->size(1));
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = code(*x);
        const int64_t m = p.m, n = p.n;
        Tensor h = at::empty({m, n}, x->options()), g, u;
        if (save) {
            g = at::empty({m, n}, x->options());
            u = at::empty({m, n}, x->options());
        }
        const Workspace ws(offsets != nullptr ? calls.gated_experts_bytes(path, &p, experts)
                                              : calls.gated_bytes(path, &p), *x);
        auto call = [&](q2k_stream_t stream) {
            const uint32_t flags = constant ? Q2K_FLAG_CONST_WEIGHTS : 0u;
            return offsets != nullptr
                       ? calls.gated_experts(path, flags, x->const_data_ptr(), x->numel(), wg->const_data_ptr(),
                                             wg->numel(), wu->const_data_ptr(), wu->numel(), h.data_ptr(),
                                             h.numel(), at_or_null(g), at_or_null(u), offsets, experts, &p,
                                             ws.at, ws.bytes, stream)
                       : calls.gated(path, flags, x->const_data_ptr(), x->numel(), wg->const_data_ptr(),
                                     wg->numel(), wu->const_data_ptr(), wu->numel(), h.data_ptr(), h.numel(),
                                     at_or_null(g), at_or_null(u), &p, ws.at, ws.bytes, stream);
        };
        return save ? finish(call, *x, {h, g, u}) : finish(call, *x, {h});
    });
}

// backward(dh, gate, up, w_gate, w_up, k, act[, offsets])
PyObject* backward(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 7 && count != 8) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_gated_ffn_params p = {};
        const Tensor* dh = take_activations(v[0]);
        if (dh == nullptr || dh->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
        const int device = dh->get_device();
        const Tensor *g = take(v[1], at::kBFloat16, 2, device), *u = take(v[2], at::kBFloat16, 2, device);
        const Tensor *wg = take(v[3], at::kByte, -1, device), *wu = take(v[4], at::kByte, -1, device);
        const int32_t* offsets = nullptr;
        uint32_t experts = 0;
        if (g == nullptr || u == nullptr || wg == nullptr || wu == nullptr || !take_size(v[5], p.k) ||
            !take_act(v[6], p.act) || g->sizes() != dh->sizes() || u->sizes() != dh->sizes() ||
            (count == 8 && !take_offsets(v[7], device, offsets, experts)))
            Py_RETURN_NONE;
        p.m = static_cast<uint32_t>(dh->size(0));
        p.n = static_cast<uint32_t>(dh->size(1));
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = Q2K_DTYPE_BF16;
        const int64_t m = p.m, n = p.n, k = p.k;
        Tensor dx = at::empty({m, k}, dh->options()), dg = at::empty({m, n}, dh->options()),
               du = at::empty({m, n}, dh->options());
        const Workspace ws(offsets != nullptr ? calls.experts_backward_bytes(&p, experts)
                                              : calls.backward_bytes(&p), *dh);
        return finish(
            [&](q2k_stream_t stream) {
                return offsets != nullptr
                           ? calls.experts_backward(dh->const_data_ptr(), g->const_data_ptr(), u->const_data_ptr(),
                                                    dh->numel(), wg->const_data_ptr(), wg->numel(),
                                                    wu->const_data_ptr(), wu->numel(), dx.data_ptr(), dx.numel(),
                                                    dg.data_ptr(), du.data_ptr(), offsets, experts, &p, ws.at,
                                                    ws.bytes, stream)
                           : calls.backward(dh->const_data_ptr(), g->const_data_ptr(), u->const_data_ptr(),
                                            dh->numel(), wg->const_data_ptr(), wg->numel(), wu->const_data_ptr(),
                                            wu->numel(), dx.data_ptr(), dx.numel(), dg.data_ptr(), du.data_ptr(),
                                            &p, ws.at, ws.bytes, stream);
            },
            *dh, {dx, dg, du});
    });
}

// linear(x, w, n, bias, act, residual, save, path, const_weights, offsets)
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 10) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_linear_params p = {};
        q2k_path path;
        const Tensor* x = take_activations(v[0]);
        if (x == nullptr) Py_RETURN_NONE;
        const int device = x->get_device();
        const Tensor *w = take(v[1], at::kByte, -1, device), *bias = nullptr, *residual = nullptr;
        const int save = PyObject_IsTrue(v[6]), constant = PyObject_IsTrue(v[8]);
        const int32_t* offsets = nullptr;
        if (w == nullptr || !take_size(v[2], p.n) || !take_linear_act(v[4], p.act) || !take_path(v[7], path) ||
            save < 0 || constant < 0 || !take_offsets(v[9], device, offsets, p.n_experts) ||
            !take_optional(v[3], at::kFloat, offsets != nullptr ? 2 : 1, device, bias) ||
            !take_optional(v[5], x->scalar_type(), 2, device, residual)) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        p.m = static_cast<uint32_t>(x->size(0));
        p.k = static_cast<uint32_t>(x->size(1));
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = code(*x);
        const int64_t m = p.m, n = p.n;
        if ((bias != nullptr && (bias->size(-1) != n || (offsets != nullptr && bias->size(0) != p.n_experts))) ||
            (residual != nullptr && (residual->size(0) != m || residual->size(1) != n)))
            Py_RETURN_NONE;
        Tensor y = at::empty({m, n}, x->options()), z;
        if (save) z = at::empty({m, n}, x->options());
        const Workspace ws(calls.linear_bytes(path, &p), *x);
        auto call = [&](q2k_stream_t stream) {
            return calls.linear(path, constant ? Q2K_FLAG_CONST_WEIGHTS : 0u, x->const_data_ptr(), x->numel(),
                                w->const_data_ptr(), w->numel(), static_cast<const float*>(at_or_null(bias)),
                                at_or_null(residual), y.data_ptr(), y.numel(), at_or_null(z), offsets, &p,
                                ws.at, ws.bytes, stream);
        };
        return save ? finish(call, *x, {y, z}) : finish(call, *x, {y});
    });
}

// linear_backward(dy, w, k, z, act, bias, offsets): (dx, dz, dbias), without dz where
// there is no activation and without dbias unless it is asked for
PyObject* linear_backward(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 7) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_linear_params p = {};
        const Tensor* dy = take_activations(v[0]);
        if (dy == nullptr || dy->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
        const int device = dy->get_device();
        const Tensor *w = take(v[1], at::kByte, -1, device), *z = nullptr;
        const int bias = PyObject_IsTrue(v[5]);
        const int32_t* offsets = nullptr;
        if (w == nullptr || bias < 0 || !take_size(v[2], p.k) || !take_linear_act(v[4], p.act) ||
            !take_offsets(v[6], device, offsets, p.n_experts)) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        if (p.act != Q2K_ACT_NONE) {
            z = take(v[3], at::kBFloat16, 2, device);
            if (z == nullptr || z->sizes() != dy->sizes()) Py_RETURN_NONE;
        }
        p.m = static_cast<uint32_t>(dy->size(0));
        p.n = static_cast<uint32_t>(dy->size(1));
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = Q2K_DTYPE_BF16;
        const int64_t m = p.m, n = p.n, k = p.k, experts = p.n_experts;
        Tensor dx = at::empty({m, k}, dy->options()), dz, dbias;
        if (z != nullptr) dz = at::empty({m, n}, dy->options());
        if (bias) {
            const auto f32 = dy->options().dtype(at::kFloat);
            dbias = offsets != nullptr ? at::empty({experts, n}, f32) : at::empty({n}, f32);
        }
        const Workspace ws(calls.linear_backward_bytes(&p), *dy);
        auto call = [&](q2k_stream_t stream) {
            return calls.linear_backward(dy->const_data_ptr(), dy->numel(), at_or_null(z), w->const_data_ptr(),
                                         w->numel(), dx.data_ptr(), dx.numel(), at_or_null(dz),
                                         static_cast<float*>(at_or_null(dbias)), offsets, &p, ws.at, ws.bytes,
                                         stream);
        };
        if (z != nullptr) return bias ? finish(call, *dy, {dx, dz, dbias}) : finish(call, *dy, {dx, dz});
        return bias ? finish(call, *dy, {dx, dbias}) : finish(call, *dy, {dx});
    });
}

// route(ids, n_experts): (rows, order, offsets, bad)
PyObject* route(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 2) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_moe_params p = {};
        const Tensor* ids = take(v[0], at::kInt, 2, -1);
        if (ids == nullptr || ids->get_device() != c10::cuda::current_device() || !take_size(v[1], p.n_experts) ||
            p.n_experts > Q2K_MOE_MAX_EXPERTS || ids->size(0) > INT_MAX || ids->size(1) > Q2K_MOE_MAX_TOP_K)
            Py_RETURN_NONE;
        const int64_t tokens = ids->size(0), top_k = ids->size(1);
        p.n_tokens = static_cast<uint32_t>(tokens);
        p.top_k = static_cast<uint32_t>(top_k);
        Tensor rows = at::empty({tokens, top_k}, ids->options()), order = at::empty({tokens * top_k}, ids->options()),
               offsets = at::empty({int64_t(p.n_experts) + 1}, ids->options()), bad = at::empty({1}, ids->options());
        return finish(
            [&](q2k_stream_t stream) {
                return calls.route(ids->const_data_ptr<int32_t>(), ids->numel(), rows.data_ptr<int32_t>(),
                                   order.data_ptr<int32_t>(), offsets.data_ptr<int32_t>(), &p,
                                   static_cast<uint32_t*>(bad.data_ptr()), stream);
            },
            *ids, {rows, order, offsets, bad});
    });
}

// The activations of a move (one row for each token, or `wide` for each choice) and its
// rows and offsets; false if they are not ordinary.
struct Move {
    q2k_moe_params p = {};
    const Tensor *t, *rows, *offsets;
    bool take_all(PyObject* o, PyObject* r, PyObject* f, bool wide) {
        t = take_activations(o);
        if (t == nullptr) return false;
        rows = take(r, at::kInt, 2, t->get_device());
        offsets = take(f, at::kInt, 1, t->get_device());
        if (rows == nullptr || offsets == nullptr || offsets->size(0) < 2 || offsets->size(0) > INT_MAX ||
            rows->size(0) > INT_MAX || rows->size(1) > INT_MAX ||
            t->size(0) != (wide ? rows->numel() : rows->size(0)))
            return false;
        p.n_tokens = static_cast<uint32_t>(rows->size(0));
        p.top_k = static_cast<uint32_t>(rows->size(1));
        p.n_experts = static_cast<uint32_t>(offsets->size(0) - 1);
        p.width = static_cast<uint32_t>(t->size(1));
        p.dtype = code(*t);
        return true;
    }
    Tensor out(bool wide) const {
        return at::empty({wide ? rows->numel() : rows->size(0), t->size(1)}, t->options());
    }
    const int32_t* rows_at() const { return rows->const_data_ptr<int32_t>(); }
    const int32_t* offsets_at() const { return offsets->const_data_ptr<int32_t>(); }
};

// sort(x, rows, offsets), sort_backward(dxs, rows, offsets)
template <bool kBack>
PyObject* sort(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Move m;
        if (!m.take_all(v[0], v[1], v[2], kBack)) Py_RETURN_NONE;
        Tensor out = m.out(!kBack);
        return finish(
            [&](q2k_stream_t stream) {
                return (kBack ? calls.sort_backward : calls.sort)(m.t->const_data_ptr(), m.t->numel(), m.rows_at(),
                                                                  m.offsets_at(), out.data_ptr(), out.numel(),
                                                                  &m.p, stream);
            },
            *m.t, {out});
    });
}

bool same_shape(const Tensor* t, int64_t rows, int64_t columns) {
    return t->size(0) == rows && t->size(1) == columns;
}

// combine(ys, rows, offsets, weights or None, residual or None)
PyObject* combine(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 5) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Move m;
        if (!m.take_all(v[0], v[1], v[2], true)) Py_RETURN_NONE;
        const int device = m.t->get_device();
        const Tensor *weights, *residual;
        if (!take_optional(v[3], at::kFloat, 2, device, weights) ||
            !take_optional(v[4], m.t->scalar_type(), 2, device, residual) ||
            (weights != nullptr && weights->sizes() != m.rows->sizes()) ||
            (residual != nullptr && !same_shape(residual, m.rows->size(0), m.t->size(1))))
            Py_RETURN_NONE;
        Tensor out = m.out(false);
        return finish(
            [&](q2k_stream_t stream) {
                return calls.combine(m.t->const_data_ptr(), m.t->numel(), m.rows_at(), m.offsets_at(),
                                     static_cast<const float*>(at_or_null(weights)), at_or_null(residual),
                                     out.data_ptr(), out.numel(), &m.p, stream);
            },
            *m.t, {out});
    });
}

// combine_backward(dy, ys, rows, offsets, weights)
PyObject* combine_backward(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 5) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Move m;
        if (!m.take_all(v[1], v[2], v[3], true)) Py_RETURN_NONE;
        const int device = m.t->get_device();
        const Tensor *dy = take(v[0], m.t->scalar_type(), 2, device), *weights = take(v[4], at::kFloat, 2, device);
        if (dy == nullptr || weights == nullptr || weights->sizes() != m.rows->sizes() ||
            !same_shape(dy, m.rows->size(0), m.t->size(1)))
            Py_RETURN_NONE;
        Tensor dys = m.out(true), dweights = at::empty(weights->sizes(), weights->options());
        return finish(
            [&](q2k_stream_t stream) {
                return calls.combine_backward(dy->const_data_ptr(), dy->numel(), m.t->const_data_ptr(),
                                              m.t->numel(), m.rows_at(), m.offsets_at(),
                                              weights->const_data_ptr<float>(), dys.data_ptr(),
                                              dweights.data_ptr<float>(), &m.p, stream);
            },
            *m.t, {dys, dweights});
    });
}

// lora(x, w, n, lora_a, lora_b, ids, scales or None, path, const_weights): (y, bad)
PyObject* lora(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 9) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_lora_params p = {};
        q2k_path path;
        const Tensor* x = take_activations(v[0]);
        if (x == nullptr) Py_RETURN_NONE;
        const int device = x->get_device();
        const Tensor* w = take(v[1], at::kByte, -1, device);
        const Tensor *a = take(v[3], at::kBFloat16, 3, device), *b = take(v[4], at::kBFloat16, 3, device);
        const Tensor* ids = take(v[5], at::kInt, 1, device);
        const Tensor* scales = v[6] == Py_None ? nullptr : take(v[6], at::kFloat, 1, device);
        const int constant = PyObject_IsTrue(v[8]);
        if (w == nullptr || a == nullptr || b == nullptr || ids == nullptr || !take_size(v[2], p.n) ||
            (v[6] != Py_None && scales == nullptr) || !take_path(v[7], path) || constant < 0) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        const int64_t m = x->size(0), k = x->size(1), n = p.n, adapters = a->size(0), rank = a->size(1);
        if (adapters > INT_MAX || rank > INT_MAX || a->size(2) != k || b->size(0) != adapters ||
            b->size(1) != n || b->size(2) != rank || ids->size(0) != m ||
            (scales != nullptr && scales->size(0) != adapters))
            Py_RETURN_NONE;
        p.m = static_cast<uint32_t>(m);
        p.k = static_cast<uint32_t>(k);
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = code(*x);
        p.rank = static_cast<uint32_t>(rank);
        p.n_adapters = static_cast<uint32_t>(adapters);
        Tensor y = at::empty({m, n}, x->options());
        Tensor bad = at::empty({1}, ids->options());
        const Workspace ws(calls.lora_bytes(path, &p), *x);
        return finish(
            [&](q2k_stream_t stream) {
                return calls.lora(path, constant ? Q2K_FLAG_CONST_WEIGHTS : 0u, x->const_data_ptr(), x->numel(),
                                  w->const_data_ptr(), w->numel(), a->const_data_ptr(), a->numel(), b->const_data_ptr(),
                                  b->numel(), scales != nullptr ? scales->const_data_ptr<float>() : nullptr,
                                  ids->const_data_ptr<int32_t>(), y.data_ptr(), y.numel(), &p,
                                  static_cast<uint32_t*>(bad.data_ptr()), ws.at, ws.bytes, stream);
            },
            *x, {y, bad});
    });
}

template <typename F>
void set_call(F& f, void* at) { f = reinterpret_cast<F>(at); }

// `want` addresses, none of them null, into `at`.
bool take_addresses(PyObject* const* v, Py_ssize_t count, Py_ssize_t want, const char* complaint, void** at) {
    if (count != want) {
        PyErr_SetString(PyExc_TypeError, complaint);
        return false;
    }
    for (Py_ssize_t i = 0; i < want; ++i) {
        at[i] = PyLong_AsVoidPtr(v[i]);
        if (at[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return false;
        }
    }
    return true;
}

// bind(addresses): the first six functions of Calls, in its order
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t count) {
    void* at[6];
    if (!take_addresses(v, count, 6, "bind takes six addresses", at)) return nullptr;
    set_call(calls.gated, at[0]);
    set_call(calls.gated_bytes, at[1]);
    set_call(calls.backward, at[2]);
    set_call(calls.backward_bytes, at[3]);
    set_call(calls.lora, at[4]);
    set_call(calls.lora_bytes, at[5]);
    Py_RETURN_NONE;
}

// bind_experts(addresses): the other thirteen
PyObject* bind_experts(PyObject*, PyObject* const* v, Py_ssize_t count) {
    void* at[13];
    if (!take_addresses(v, count, 13, "bind_experts takes thirteen addresses", at)) return nullptr;
    set_call(calls.linear, at[0]);
    set_call(calls.linear_bytes, at[1]);
    set_call(calls.linear_backward, at[2]);
    set_call(calls.linear_backward_bytes, at[3]);
    set_call(calls.gated_experts, at[4]);
    set_call(calls.gated_experts_bytes, at[5]);
    set_call(calls.experts_backward, at[6]);
    set_call(calls.experts_backward_bytes, at[7]);
    set_call(calls.route, at[8]);
    set_call(calls.sort, at[9]);
    set_call(calls.sort_backward, at[10]);
    set_call(calls.combine, at[11]);
    set_call(calls.combine_backward, at[12]);
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

}  // namespace

PyMODINIT_FUNC PyInit_q2k_torch() {
    static PyMethodDef methods[] = {
        {"bind", fast(bind), METH_FASTCALL, "bind(addresses)"},
        {"bind_experts", fast(bind_experts), METH_FASTCALL, "bind_experts(addresses)"},
        {"gated", fast(gated), METH_FASTCALL,
         "gated(x, w_gate, w_up, n, act, save, path, const_weights[, offsets])"},
        {"backward", fast(backward), METH_FASTCALL, "backward(dh, gate, up, w_gate, w_up, k, act[, offsets])"},
        {"lora", fast(lora), METH_FASTCALL,
         "lora(x, w, n, lora_a, lora_b, ids, scales, path, const_weights)"},
        {"linear", fast(linear), METH_FASTCALL,
         "linear(x, w, n, bias, act, residual, save, path, const_weights, offsets)"},
        {"linear_backward", fast(linear_backward), METH_FASTCALL,
         "linear_backward(dy, w, k, z, act, bias, offsets)"},
        {"route", fast(route), METH_FASTCALL, "route(ids, n_experts)"},
        {"sort", fast(sort<false>), METH_FASTCALL, "sort(x, rows, offsets)"},
        {"sort_backward", fast(sort<true>), METH_FASTCALL, "sort_backward(dxs, rows, offsets)"},
        {"combine", fast(combine), METH_FASTCALL, "combine(ys, rows, offsets, weights, residual)"},
        {"combine_backward", fast(combine_backward), METH_FASTCALL,
         "combine_backward(dy, ys, rows, offsets, weights)"},
        {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "q2k_torch",
                                 "libq2k's feed-forward calls for PyTorch tensors.", -1, methods,
                                 nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&module);
}
