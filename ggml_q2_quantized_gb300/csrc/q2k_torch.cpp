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

// gated(x, w_gate, w_up, n, act, save, path, const_weights)
PyObject* gated(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 8) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_gated_ffn_params p = {};
        q2k_path path;
        const Tensor* x = take_activations(v[0]);
        if (x == nullptr) Py_RETURN_NONE;
        const int device = x->get_device();
        const Tensor *wg = take(v[1], at::kByte, -1, device), *wu = take(v[2], at::kByte, -1, device);
        const int save = PyObject_IsTrue(v[5]), constant = PyObject_IsTrue(v[7]);
        if (wg == nullptr || wu == nullptr || !take_size(v[3], p.n) || !take_act(v[4], p.act) ||
            !take_path(v[6], path) || save < 0 || constant < 0) {
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
        const Workspace ws(calls.gated_bytes(path, &p), *x);
        auto call = [&](q2k_stream_t stream) {
            return calls.gated(path, constant ? Q2K_FLAG_CONST_WEIGHTS : 0u, x->const_data_ptr(), x->numel(),
                               wg->const_data_ptr(), wg->numel(), wu->const_data_ptr(), wu->numel(), h.data_ptr(),
                               h.numel(), save ? g.data_ptr() : nullptr, save ? u.data_ptr() : nullptr,
                               &p, ws.at, ws.bytes, stream);
        };
        return save ? finish(call, *x, {h, g, u}) : finish(call, *x, {h});
    });
}

// backward(dh, gate, up, w_gate, w_up, k, act)
PyObject* backward(PyObject*, PyObject* const* v, Py_ssize_t count) {
    if (count != 7) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        q2k_gated_ffn_params p = {};
        const Tensor* dh = take_activations(v[0]);
        if (dh == nullptr || dh->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
        const int device = dh->get_device();
        const Tensor *g = take(v[1], at::kBFloat16, 2, device), *u = take(v[2], at::kBFloat16, 2, device);
        const Tensor *wg = take(v[3], at::kByte, -1, device), *wu = take(v[4], at::kByte, -1, device);
        if (g == nullptr || u == nullptr || wg == nullptr || wu == nullptr || !take_size(v[5], p.k) ||
            !take_act(v[6], p.act) || g->sizes() != dh->sizes() || u->sizes() != dh->sizes())
            Py_RETURN_NONE;
        p.m = static_cast<uint32_t>(dh->size(0));
        p.n = static_cast<uint32_t>(dh->size(1));
        p.ggml_type = Q2K_GGML_TYPE_Q2_K;
        p.dtype = Q2K_DTYPE_BF16;
        const int64_t m = p.m, n = p.n, k = p.k;
        Tensor dx = at::empty({m, k}, dh->options()), dg = at::empty({m, n}, dh->options()),
               du = at::empty({m, n}, dh->options());
        const Workspace ws(calls.backward_bytes(&p), *dh);
        return finish(
            [&](q2k_stream_t stream) {
                return calls.backward(dh->const_data_ptr(), g->const_data_ptr(), u->const_data_ptr(), dh->numel(),
                                      wg->const_data_ptr(), wg->numel(), wu->const_data_ptr(), wu->numel(),
                                      dx.data_ptr(), dx.numel(), dg.data_ptr(), du.data_ptr(), &p, ws.at,
                                      ws.bytes, stream);
            },
            *dh, {dx, dg, du});
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

// bind(addresses): the six functions of Calls, in its order
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t count) {
    void* at[6];
    if (count != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i) {
        at[i] = PyLong_AsVoidPtr(v[i]);
        if (at[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    calls.gated = reinterpret_cast<decltype(calls.gated)>(at[0]);
    calls.gated_bytes = reinterpret_cast<decltype(calls.gated_bytes)>(at[1]);
    calls.backward = reinterpret_cast<decltype(calls.backward)>(at[2]);
    calls.backward_bytes = reinterpret_cast<decltype(calls.backward_bytes)>(at[3]);
    calls.lora = reinterpret_cast<decltype(calls.lora)>(at[4]);
    calls.lora_bytes = reinterpret_cast<decltype(calls.lora_bytes)>(at[5]);
    Py_RETURN_NONE;
}

}  // namespace

PyMODINIT_FUNC PyInit_q2k_torch() {
    static PyMethodDef methods[] = {
        {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL,
         "bind(addresses)"},
        {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated)), METH_FASTCALL,
         "gated(x, w_gate, w_up, n, act, save, path, const_weights)"},
        {"backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(backward)), METH_FASTCALL,
         "backward(dh, gate, up, w_gate, w_up, k, act)"},
        {"lora", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(lora)), METH_FASTCALL,
         "lora(x, w, n, lora_a, lora_b, ids, scales, path, const_weights)"},
        {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "q2k_torch",
                                 "libq2k's feed-forward calls for PyTorch tensors.", -1, methods,
                                 nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&module);
}
