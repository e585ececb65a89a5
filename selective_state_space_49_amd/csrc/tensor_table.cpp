// tensor_table.cpp -- a CPython extension for the calls whose marshalling in Python would take
// longer than their kernels.
//
// A step over a stack of layers passes several hundred tensors. Asking each of them from
// Python for its address, size, type, device and layout takes 0.45 us a tensor (124 us for
// 281), longer than the step's kernels; here it takes 0.02 us. A single token's call has seven
// tensors and a kernel of 2.6 us.
//
// The entry points of the library come as addresses, from the binding that has loaded it. A call
// returns what it has made; the status where the library refuses; None where an argument is not
// as it should be. The tensors' GPU is the current one during the call: a default stream is
// that of the current GPU, whichever tensor it was asked for.
#include "ssm_scan.h"

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_cpp_function.h>
#include <torch/csrc/autograd/python_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <memory>
#include <unordered_map>
#include <unordered_set>
#include <vector>

namespace {

// The tensor's ssm_dtype, or -1 with a Python error: it must be a contiguous float32 or bfloat16
// tensor on the GPU `device` (-1: any, which is then taken).
int kind_of(const at::Tensor &t, int *device, const char *what, Py_ssize_t k) {
    const bool here = t.defined() && t.is_cuda() && t.is_contiguous() &&
                      (t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16);
    if (!here || (*device >= 0 && t.get_device() != *device)) {
        PyErr_Format(PyExc_ValueError, "%s %zd must be a contiguous float32 or bfloat16 tensor on one GPU", what, k);
        return -1;
    }
    *device = (int)t.get_device();
    return t.scalar_type() == at::kFloat ? SSM_F32 : SSM_BF16;
}

// The host arrays of ssm_adamw_step for lists of tensors.
struct Table {
    std::vector<void *> params;
    std::vector<const void *> grads;
    std::vector<int64_t> sizes;
    std::vector<int32_t> kinds, grad_kinds;
    int64_t blocks = 0;  // the sizes in blocks, each rounded up
    int device = -1;
    // False with a Python error.
    bool read(PyObject *p_list, PyObject *g_list, int64_t block) {
        if (!PyList_Check(p_list) || !PyList_Check(g_list)) {
            PyErr_SetString(PyExc_TypeError, "parameters and gradients must be lists");
            return false;
        }
        const Py_ssize_t n = PyList_GET_SIZE(p_list);
        if (PyList_GET_SIZE(g_list) != n) {
            PyErr_Format(PyExc_ValueError, "%zd parameters and %zd gradients", n, PyList_GET_SIZE(g_list));
            return false;
        }
        params.resize(n);
        grads.resize(n);
        sizes.resize(n);
        kinds.resize(n);
        grad_kinds.resize(n);
        for (Py_ssize_t k = 0; k < n; ++k) {
            PyObject *po = PyList_GET_ITEM(p_list, k), *go = PyList_GET_ITEM(g_list, k);
            if (!THPVariable_Check(po) || (go != Py_None && !THPVariable_Check(go))) {
                PyErr_Format(PyExc_TypeError, "parameter and gradient %zd must be tensors", k);
                return false;
            }
            const at::Tensor &p = THPVariable_Unpack(po);
            const int pk = kind_of(p, &device, "parameter", k);
            if (pk < 0) return false;
            params[k] = p.data_ptr();
            sizes[k] = p.numel();
            kinds[k] = pk;
            grads[k] = nullptr;
            grad_kinds[k] = SSM_F32;
            if (go != Py_None) {
                const at::Tensor &g = THPVariable_Unpack(go);
                const int gk = kind_of(g, &device, "gradient", k);
                if (gk < 0) return false;
                if (g.sizes() != p.sizes()) {
                    PyErr_Format(PyExc_ValueError, "gradient %zd must have its parameter's shape", k);
                    return false;
                }
                grads[k] = g.data_ptr();
                grad_kinds[k] = gk;
            }
            blocks += (sizes[k] + block - 1) / block;
        }
        return true;
    }
};

// The address of a contiguous tensor of this type and these sizes on the GPU, or ok = false.
void *address(PyObject *o, at::ScalarType type, at::IntArrayRef sizes, int device, bool *ok) {
    if (!THPVariable_Check(o)) {
        *ok = false;
        return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.get_device() != device || t.sizes() != sizes || !t.is_contiguous()) {
        *ok = false;
        return nullptr;
    }
    return t.data_ptr();
}
void *optional(PyObject *o, at::ScalarType type, at::IntArrayRef sizes, int device, bool *ok) {
    return o == Py_None ? nullptr : address(o, type, sizes, device, ok);
}

// Autograd is told that a tensor was written: what saved it for a backward must not use it.
void written(const at::Tensor &t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *o) {
    if (o != Py_None) written(THPVariable_Unpack(o));
}

template <typename F>
PyObject *no_exceptions(F fn) {
    try {
        return fn();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// gated_step(entry, stream, h, x_t, r_t, i_t, decay, c, y_t or None): y_t.
PyObject *gated_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 9) return PyErr_Format(PyExc_TypeError, "9 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_gated_step))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        const double c = PyFloat_AsDouble(args[7]);
        if (PyErr_Occurred()) return nullptr;
        if (!THPVariable_Check(args[3])) Py_RETURN_NONE;
        const at::Tensor &x = THPVariable_Unpack(args[3]);
        const at::ScalarType io = x.scalar_type();
        const at::IntArrayRef all = x.sizes();
        if (!x.is_cuda() || all.size() != 3 || (io != at::kFloat && io != at::kBFloat16)) Py_RETURN_NONE;
        const int device = (int)x.get_device();
        const int64_t layer[2] = {all[0], all[2]};
        bool ok = true;
        float *const h = (float *)address(args[2], at::kFloat, all, device, &ok);
        const void *const xp = address(args[3], io, all, device, &ok), *const r = address(args[4], io, all, device, &ok),
                   *const i = address(args[5], io, all, device, &ok);
        const float *const decay = (const float *)address(args[6], at::kFloat, layer, device, &ok);
        if (!ok) Py_RETURN_NONE;
        PyObject *out = args[8];
        if (out == Py_None) out = THPVariable_Wrap(at::empty_like(x));
        else Py_INCREF(out);
        if (!out) return nullptr;
        void *const y = address(out, io, all, device, &ok);
        if (!ok) {
            Py_DECREF(out);
            Py_RETURN_NONE;
        }
        const c10::DeviceGuard on(x.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(h, xp, r, i, decay, (float)c, y, all[0], all[1], all[2], io == at::kFloat ? SSM_F32 : SSM_BF16, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK) {
            written(args[2]);
            written(args[8]);
            return out;
        }
        Py_DECREF(out);
        return PyLong_FromLong(st);
    });
}

// adamw_step(entry, stream, block, params, grads, exp_avg, exp_avg_sq, avg_scale, avg_sq_scale,
// grad_scale, lr, beta1, beta2, eps, weight_decay, step): the status; a Python error where a
// parameter or a gradient is not as it should be.
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 16) return PyErr_Format(PyExc_TypeError, "16 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_adamw_step))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        const int64_t block = PyLong_AsLongLong(args[2]);
        double f[5];
        for (int k = 0; k < 5; ++k) f[k] = PyFloat_AsDouble(args[10 + k]);
        const int64_t step = PyLong_AsLongLong(args[15]);
        if (PyErr_Occurred()) return nullptr;
        Table t;
        if (!t.read(args[3], args[4], block)) return nullptr;
        const bool codes = args[7] != Py_None;
        const int64_t total = t.blocks * block;
        bool ok = true;
        void *const m = address(args[5], codes ? at::kChar : at::kFloat, total, t.device, &ok);
        void *const v = address(args[6], codes ? at::kByte : at::kFloat, total, t.device, &ok);
        float *const ms = (float *)optional(args[7], at::kFloat, t.blocks, t.device, &ok);
        float *const vs = (float *)optional(args[8], at::kFloat, t.blocks, t.device, &ok);
        const float *gs = nullptr;
        if (args[9] != Py_None) {
            if (!THPVariable_Check(args[9]) || THPVariable_Unpack(args[9]).numel() != 1) Py_RETURN_NONE;
            gs = (const float *)address(args[9], at::kFloat, THPVariable_Unpack(args[9]).sizes(), t.device, &ok);
        }
        if (!ok) Py_RETURN_NONE;
        const c10::OptionalDeviceGuard on(t.device < 0 ? c10::optional<c10::Device>() : c10::Device(c10::kCUDA, (c10::DeviceIndex)t.device));
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry((int32_t)t.params.size(), t.params.data(), t.grads.data(), t.sizes.data(), t.kinds.data(),
                   t.grad_kinds.data(), m, v, ms, vs, gs, f[0], f[1], f[2], f[3], f[4], step, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK) {
            for (size_t k = 0; k < t.params.size(); ++k)
                if (t.grads[k]) written(PyList_GET_ITEM(args[3], (Py_ssize_t)k));
            for (int k = 5; k < 9; ++k) written(args[k]);
        }
        return PyLong_FromLong(st);
    });
}

// What the larger calls share: the first tensor's device and type, what is read of the arguments,
// new tensors, and the workspace, which lives until the call is enqueued.
struct Call {
    const at::Tensor &first;
    const at::ScalarType io;
    const int device;
    bool ok;
    explicit Call(PyObject *o, size_t dims)
        : first(THPVariable_Unpack(o)), io(first.scalar_type()), device(first.is_cuda() ? (int)first.get_device() : -1),
          ok(device >= 0 && first.sizes().size() == dims && (io == at::kFloat || io == at::kBFloat16)) {}
    ssm_dtype kind() const { return io == at::kFloat ? SSM_F32 : SSM_BF16; }
    void *in(PyObject *o, at::ScalarType type, at::IntArrayRef sizes) { return optional(o, type, sizes, device, &ok); }
    void *need(PyObject *o, at::ScalarType type, at::IntArrayRef sizes) { return address(o, type, sizes, device, &ok); }
    // The caller's tensor or, for None, a new one.
    at::Tensor out(PyObject *o, at::ScalarType type, at::IntArrayRef sizes) {
        if (o == Py_None) return fresh(type, sizes);
        need(o, type, sizes);
        return ok ? THPVariable_Unpack(o) : at::Tensor();
    }
    at::Tensor fresh(at::ScalarType type, at::IntArrayRef sizes) const {
        return at::empty(sizes, first.options().dtype(type).requires_grad(false));
    }
};
void *at_of(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject *wrap(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
// The status, or the tensors where it is SSM_OK; an undefined one is None.
PyObject *result(ssm_status st, std::initializer_list<at::Tensor> outs) {
    if (st != SSM_OK) return PyLong_FromLong(st);
    PyObject *tuple = PyTuple_New((Py_ssize_t)outs.size());
    Py_ssize_t k = 0;
    for (const at::Tensor &t : outs) {
        PyObject *o = tuple ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, k++, o);
    }
    return tuple;
}
at::ScalarType byte_type(PyObject *o) {  // bool or uint8
    return THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kBool ? at::kBool : at::kByte;
}

// gated_fwd(entry, workspace size's entry, stream, x, r, i, decay, h0, reset, c, y, h_final, states,
// want_h_final, save): (y, h_final, states).
PyObject *gated_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 15) return PyErr_Format(PyExc_TypeError, "15 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_gated_fwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_gated_fwd_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        const float c = (float)PyFloat_AsDouble(args[9]);
        if (PyErr_Occurred()) return nullptr;
        if (!THPVariable_Check(args[3])) Py_RETURN_NONE;
        Call k(args[3], 3);
        if (!k.ok) Py_RETURN_NONE;
        const at::IntArrayRef all = k.first.sizes();
        const int64_t b = all[0], L = all[1], D = all[2], ends[2] = {b, D}, steps[2] = {b, L},
                      rows[3] = {b, (L + SSM_GATED_STATE_EVERY - 1) / SSM_GATED_STATE_EVERY, D};
        const void *const x = k.need(args[3], k.io, all), *const r = k.need(args[4], k.io, all), *const i = k.need(args[5], k.io, all);
        const float *const decay = (const float *)k.need(args[6], at::kFloat, D);
        const float *const h0 = (const float *)k.in(args[7], at::kFloat, ends);
        const uint8_t *const reset = (const uint8_t *)k.in(args[8], byte_type(args[8]), steps);
        if (!k.ok) Py_RETURN_NONE;
        const at::Tensor y = k.out(args[10], k.io, all);
        const at::Tensor h = args[11] != Py_None || args[13] == Py_True ? k.out(args[11], at::kFloat, ends) : at::Tensor();
        const at::Tensor states = args[12] != Py_None || args[14] == Py_True ? k.out(args[12], at::kFloat, rows) : at::Tensor();
        if (!k.ok) Py_RETURN_NONE;
        const size_t bytes = size(b, L, D);
        const at::Tensor ws = bytes ? k.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(k.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(x, r, i, decay, h0, reset, c, at_of(y), (float *)at_of(h), (float *)at_of(states), b, L, D, k.kind(),
                   at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int k = 10; k < 13; ++k) written(args[k]);
        return result(st, {y, h, states});
    });
}

// gated_bwd(entry, workspace size's entry, stream, x, r, i, decay, states, reset, dy, dh_final, c,
// want_dh0): (dx, dr, di, ddecay, dh0).
PyObject *gated_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 13) return PyErr_Format(PyExc_TypeError, "13 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_gated_bwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_gated_bwd_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        const float c = (float)PyFloat_AsDouble(args[11]);
        if (PyErr_Occurred()) return nullptr;
        if (!THPVariable_Check(args[3])) Py_RETURN_NONE;
        Call k(args[3], 3);
        if (!k.ok) Py_RETURN_NONE;
        const at::IntArrayRef all = k.first.sizes();
        const int64_t b = all[0], L = all[1], D = all[2], ends[2] = {b, D}, steps[2] = {b, L},
                      rows[3] = {b, (L + SSM_GATED_STATE_EVERY - 1) / SSM_GATED_STATE_EVERY, D};
        const void *const x = k.need(args[3], k.io, all), *const r = k.need(args[4], k.io, all), *const i = k.need(args[5], k.io, all);
        const float *const decay = (const float *)k.need(args[6], at::kFloat, D);
        const float *const states = (const float *)k.need(args[7], at::kFloat, rows);
        const uint8_t *const reset = (const uint8_t *)k.in(args[8], byte_type(args[8]), steps);
        const void *const dy = k.need(args[9], k.io, all);
        const float *const dh = (const float *)k.in(args[10], at::kFloat, ends);
        if (!k.ok) Py_RETURN_NONE;
        const at::Tensor dx = k.fresh(k.io, all), dr = k.fresh(k.io, all), di = k.fresh(k.io, all), dd = k.fresh(at::kFloat, D);
        const at::Tensor dh0 = args[12] == Py_True ? k.fresh(at::kFloat, ends) : at::Tensor();
        const size_t bytes = size(b, L, D);
        const at::Tensor ws = bytes ? k.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(k.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(x, r, i, decay, states, reset, c, dy, dh, at_of(dx), at_of(dr), at_of(di), (float *)at_of(dd),
                   (float *)at_of(dh0), b, L, D, k.kind(), at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        return result(st, {dx, dr, di, dd, dh0});
    });
}

// xent_fwd(entry, workspace size's entry, stream, hidden, weight, targets, ignore_index, loss, lse,
// mean): (loss, lse, mean).
PyObject *xent_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 10) return PyErr_Format(PyExc_TypeError, "10 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_xent_fwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_xent_fwd_workspace_for))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        const int64_t ignore = PyLong_AsLongLong(args[6]);
        if (PyErr_Occurred()) return nullptr;
        if (!THPVariable_Check(args[3]) || !THPVariable_Check(args[4]) || THPVariable_Unpack(args[4]).dim() != 2) Py_RETURN_NONE;
        Call k(args[3], 2);
        if (!k.ok) Py_RETURN_NONE;
        const int64_t T = k.first.size(0), K = k.first.size(1), V = THPVariable_Unpack(args[4]).size(0), head[2] = {V, K};
        const void *const hidden = k.need(args[3], k.io, k.first.sizes()), *const weight = k.need(args[4], k.io, head);
        const int64_t *const targets = (const int64_t *)k.need(args[5], at::kLong, T);
        if (!k.ok) Py_RETURN_NONE;
        const at::Tensor loss = k.out(args[7], at::kFloat, T), lse = k.out(args[8], at::kFloat, T), mean = k.out(args[9], at::kFloat, 2);
        if (!k.ok) Py_RETURN_NONE;
        const size_t bytes = size(hidden, weight, T, K, V, k.kind());
        const at::Tensor ws = bytes ? k.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(k.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(hidden, weight, targets, ignore, (float *)at_of(loss), (float *)at_of(lse), (float *)at_of(mean), T, K, V,
                   k.kind(), at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int k = 7; k < 10; ++k) written(args[k]);
        return result(st, {loss, lse, mean});
    });
}

// xent_bwd(entry, workspace size's entry, stream, hidden, weight, targets, ignore_index, lse, mean,
// dloss, dmean, want_dhidden, want_dweight): (dhidden, dweight).
PyObject *xent_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 13) return PyErr_Format(PyExc_TypeError, "13 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_xent_bwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_xent_bwd_workspace_for))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        const int64_t ignore = PyLong_AsLongLong(args[6]);
        if (PyErr_Occurred()) return nullptr;
        if (!THPVariable_Check(args[3]) || !THPVariable_Check(args[4]) || THPVariable_Unpack(args[4]).dim() != 2) Py_RETURN_NONE;
        Call k(args[3], 2);
        if (!k.ok) Py_RETURN_NONE;
        const int64_t T = k.first.size(0), K = k.first.size(1), V = THPVariable_Unpack(args[4]).size(0), head[2] = {V, K};
        const void *const hidden = k.need(args[3], k.io, k.first.sizes()), *const weight = k.need(args[4], k.io, head);
        const int64_t *const targets = (const int64_t *)k.need(args[5], at::kLong, T);
        const float *const lse = (const float *)k.need(args[7], at::kFloat, T), *const mean = (const float *)k.need(args[8], at::kFloat, 2);
        const float *const dloss = (const float *)k.in(args[9], at::kFloat, T);
        const float *dmean = nullptr;
        if (args[10] != Py_None) {
            if (!THPVariable_Check(args[10]) || THPVariable_Unpack(args[10]).numel() != 1) Py_RETURN_NONE;
            dmean = (const float *)k.need(args[10], at::kFloat, THPVariable_Unpack(args[10]).sizes());
        }
        if (!k.ok) Py_RETURN_NONE;
        const at::Tensor dh = args[11] == Py_True ? k.fresh(k.io, k.first.sizes()) : at::Tensor();
        const at::Tensor dw = args[12] == Py_True ? k.fresh(k.io, head) : at::Tensor();
        const size_t bytes = size(hidden, weight, dloss, T, K, V, k.kind());
        const at::Tensor ws = bytes ? k.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(k.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(hidden, weight, targets, ignore, lse, mean, dloss, dmean, at_of(dh), at_of(dw), T, K, V, k.kind(),
                   at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        return result(st, {dh, dw});
    });
}

// A tensor's number of dimensions, -1 for anything else.
int64_t dims_of(PyObject *o) { return THPVariable_Check(o) ? THPVariable_Unpack(o).dim() : -1; }

// What the calls of the linear attention share: the sizes, and the addresses of q, k, v and the decays.
// args: q, k, v, log_decay.
struct Linattn {
    int64_t b, L, H, Hk, K, V;
    const void *q, *k, *v;
    const float *g;
    int32_t per_token;
    bool read(Call &c, PyObject *const *args, bool step) {
        if (dims_of(args[2]) != 4) return false;
        const at::IntArrayRef qs = c.first.sizes(), vs = THPVariable_Unpack(args[2]).sizes();
        b = qs[0], L = qs[1], Hk = qs[2], K = qs[3], H = vs[2], V = vs[3];
        const int64_t value[4] = {b, L, H, V}, token[3] = {b, L, H}, layer[2] = {b, H};
        per_token = dims_of(args[3]) == 3;
        q = c.need(args[0], c.io, qs);
        k = c.need(args[1], c.io, qs);
        v = c.need(args[2], c.io, value);
        g = (const float *)(per_token ? c.need(args[3], at::kFloat, token)
                                      : step ? c.need(args[3], at::kFloat, layer) : c.need(args[3], at::kFloat, H));
        return c.ok && H <= INT32_MAX && Hk <= INT32_MAX && K <= INT32_MAX && V <= INT32_MAX;
    }
};
float scale_of(PyObject *o, int64_t K) { return o == Py_None ? (float)(1.0 / std::sqrt((double)K)) : (float)PyFloat_AsDouble(o); }

// linattn_fwd(entry, workspace size's entry, stream, q, k, v, log_decay, h0, scale, o, h_final, states,
// want_h_final, save): (o, h_final, states).
PyObject *linattn_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "14 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_linattn_fwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_linattn_fwd_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        if (dims_of(args[3]) != 4) Py_RETURN_NONE;
        Call c(args[3], 4);
        Linattn t;
        if (!c.ok || !t.read(c, args + 3, false)) Py_RETURN_NONE;
        const float scale = scale_of(args[8], t.K);
        if (PyErr_Occurred()) return nullptr;
        const int64_t every = c.io == at::kFloat ? SSM_LINATTN_CHUNK_F32 : SSM_LINATTN_CHUNK_BF16;
        const int64_t out[4] = {t.b, t.L, t.H, t.V}, state[4] = {t.b, t.H, t.K, t.V},
                      rows[5] = {t.b, t.H, (t.L + every - 1) / every, t.K, t.V};
        const float *const h0 = (const float *)c.in(args[7], at::kFloat, state);
        if (!c.ok) Py_RETURN_NONE;
        const at::Tensor o = c.out(args[9], c.io, out);
        const at::Tensor h = args[10] != Py_None || args[12] == Py_True ? c.out(args[10], at::kFloat, state) : at::Tensor();
        const at::Tensor states = args[11] != Py_None || args[13] == Py_True ? c.out(args[11], at::kFloat, rows) : at::Tensor();
        if (!c.ok) Py_RETURN_NONE;
        const size_t bytes = size(t.b, t.L, (int32_t)t.H, (int32_t)t.Hk, (int32_t)t.K, (int32_t)t.V, c.kind());
        const at::Tensor ws = bytes ? c.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(t.q, t.k, t.v, t.g, t.per_token, h0, scale, at_of(o), (float *)at_of(h), (float *)at_of(states), t.b, t.L, (int32_t)t.H,
                   (int32_t)t.Hk, (int32_t)t.K, (int32_t)t.V, c.kind(), at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int k = 9; k < 12; ++k) written(args[k]);
        return result(st, {o, h, states});
    });
}

// linattn_bwd(entry, workspace size's entry, stream, q, k, v, log_decay, states, do, dh_final, scale,
// want_dh0): (dq, dk, dv, dlog_decay, dh0).
PyObject *linattn_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 12) return PyErr_Format(PyExc_TypeError, "12 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_linattn_bwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_linattn_bwd_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        if (dims_of(args[3]) != 4) Py_RETURN_NONE;
        Call c(args[3], 4);
        Linattn t;
        if (!c.ok || !t.read(c, args + 3, false)) Py_RETURN_NONE;
        const float scale = scale_of(args[10], t.K);
        if (PyErr_Occurred()) return nullptr;
        const int64_t every = c.io == at::kFloat ? SSM_LINATTN_CHUNK_F32 : SSM_LINATTN_CHUNK_BF16;
        const int64_t out[4] = {t.b, t.L, t.H, t.V}, state[4] = {t.b, t.H, t.K, t.V},
                      rows[5] = {t.b, t.H, (t.L + every - 1) / every, t.K, t.V};
        const float *const states = (const float *)c.need(args[7], at::kFloat, rows);
        const void *const d_o = c.need(args[8], c.io, out);
        const float *const dh = (const float *)c.in(args[9], at::kFloat, state);
        if (!c.ok) Py_RETURN_NONE;
        const at::Tensor dq = c.fresh(c.io, c.first.sizes()), dk = c.fresh(c.io, c.first.sizes()), dv = c.fresh(c.io, out);
        const at::Tensor dg = c.fresh(at::kFloat, THPVariable_Unpack(args[6]).sizes());
        const at::Tensor dh0 = args[11] == Py_True ? c.fresh(at::kFloat, state) : at::Tensor();
        const size_t bytes = size(t.b, t.L, (int32_t)t.H, (int32_t)t.Hk, (int32_t)t.K, (int32_t)t.V, t.per_token, c.kind());
        const at::Tensor ws = bytes ? c.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(t.q, t.k, t.v, t.g, t.per_token, states, d_o, dh, scale, at_of(dq), at_of(dk), at_of(dv), (float *)at_of(dg),
                   (float *)at_of(dh0), t.b, t.L, (int32_t)t.H, (int32_t)t.Hk, (int32_t)t.K, (int32_t)t.V, c.kind(), at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        return result(st, {dq, dk, dv, dg, dh0});
    });
}

// linattn_step(entry, stream, h, q_t, k_t, v_t, log_decay, scale, o_t or None): o_t.
PyObject *linattn_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 9) return PyErr_Format(PyExc_TypeError, "9 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_linattn_step))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        if (dims_of(args[3]) != 4) Py_RETURN_NONE;
        Call c(args[3], 4);
        Linattn t;
        if (!c.ok || !t.read(c, args + 3, true)) Py_RETURN_NONE;
        const float scale = scale_of(args[7], t.K);
        if (PyErr_Occurred()) return nullptr;
        const int64_t out[4] = {t.b, t.L, t.H, t.V}, state[5] = {t.b, t.L, t.H, t.K, t.V};
        float *const h = (float *)c.need(args[2], at::kFloat, state);
        if (!c.ok) Py_RETURN_NONE;
        const at::Tensor o = c.out(args[8], c.io, out);
        if (!c.ok) Py_RETURN_NONE;
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(h, t.q, t.k, t.v, t.g, t.per_token, scale, at_of(o), t.b, t.L, (int32_t)t.H, (int32_t)t.Hk, (int32_t)t.K, (int32_t)t.V,
                   c.kind(), stream);
        Py_END_ALLOW_THREADS
        if (st != SSM_OK) return PyLong_FromLong(st);
        written(args[2]);
        written(args[8]);
        return wrap(o);
    });
}

// The norm's inputs: x [..., dim], weight [dim], residual or None in x's type or float32.
struct Norm {
    int64_t rows = 0, dim = 0;
    at::ScalarType res;
    const void *x, *residual;
    const float *weight;
    bool read(Call &c, PyObject *x_, PyObject *weight_, PyObject *residual_) {
        const at::IntArrayRef all = c.first.sizes();
        if (all.empty()) return false;
        dim = all.back();
        if (dim < 1 || dim > INT32_MAX) return false;
        rows = c.first.numel() / dim;
        res = c.io;
        if (residual_ != Py_None && THPVariable_Check(residual_) && THPVariable_Unpack(residual_).scalar_type() == at::kFloat) res = at::kFloat;
        x = c.need(x_, c.io, all);
        residual = c.in(residual_, res, all);
        weight = (const float *)c.need(weight_, at::kFloat, dim);
        return c.ok;
    }
    ssm_dtype res_kind() const { return res == at::kFloat ? SSM_F32 : SSM_BF16; }
};

// rmsnorm_fwd(entry, stream, x, weight, residual, eps, y, residual_out, rstd, want_rstd): (y, residual_out, rstd).
PyObject *rmsnorm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 10) return PyErr_Format(PyExc_TypeError, "10 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_rmsnorm_fwd))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        const double eps = PyFloat_AsDouble(args[5]);
        if (PyErr_Occurred()) return nullptr;
        if (dims_of(args[2]) < 1) Py_RETURN_NONE;
        Call c(args[2], (size_t)dims_of(args[2]));
        Norm t;
        if (!c.ok || !t.read(c, args[2], args[3], args[4])) Py_RETURN_NONE;
        if (args[4] == Py_None && args[7] != Py_None) Py_RETURN_NONE;
        const at::IntArrayRef all = c.first.sizes(), lead = all.slice(0, all.size() - 1);
        const at::Tensor y = c.out(args[6], c.io, all);
        const at::Tensor added = args[4] != Py_None ? c.out(args[7], t.res, all) : at::Tensor();
        const at::Tensor rstd = args[8] != Py_None || args[9] == Py_True ? c.out(args[8], at::kFloat, lead) : at::Tensor();
        if (!c.ok) Py_RETURN_NONE;
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(t.x, t.residual, t.weight, eps, at_of(y), at_of(added), (float *)at_of(rstd), t.rows, (int32_t)t.dim, c.kind(), t.res_kind(),
                   stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int k = 6; k < 9; ++k) written(args[k]);
        return result(st, {y, added, rstd});
    });
}

// rmsnorm_fwd_q8(entry, stream, x, weight, residual, eps, code, group, codes, scales, residual_out):
// (codes, scales, residual_out).
PyObject *rmsnorm_fwd_q8(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 11) return PyErr_Format(PyExc_TypeError, "11 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_rmsnorm_fwd_q8))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        const double eps = PyFloat_AsDouble(args[5]);
        const long code = PyLong_AsLong(args[6]), group = PyLong_AsLong(args[7]);
        if (PyErr_Occurred()) return nullptr;
        if (dims_of(args[2]) < 1 || group < 0 || group > INT32_MAX) Py_RETURN_NONE;
        Call c(args[2], (size_t)dims_of(args[2]));
        Norm t;
        if (!c.ok || !t.read(c, args[2], args[3], args[4])) Py_RETURN_NONE;
        if (args[4] == Py_None && args[10] != Py_None) Py_RETURN_NONE;
        const at::IntArrayRef all = c.first.sizes();
        std::vector<int64_t> scale(all.begin(), all.end());
        scale.back() = group ? (t.dim + group - 1) / group : 1;
        const at::Tensor codes = c.out(args[8], code == SSM_E4M3 ? at::kFloat8_e4m3fn : at::kChar, all);
        const at::Tensor scales = c.out(args[9], at::kFloat, scale);
        const at::Tensor added = args[4] != Py_None ? c.out(args[10], t.res, all) : at::Tensor();
        if (!c.ok) Py_RETURN_NONE;
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(t.x, t.residual, t.weight, eps, at_of(codes), (float *)at_of(scales), (ssm_code)code, (int32_t)group, at_of(added), t.rows,
                   (int32_t)t.dim, c.kind(), t.res_kind(), stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int k = 8; k < 11; ++k) written(args[k]);
        return result(st, {codes, scales, added});
    });
}

// rmsnorm_bwd(entry, workspace size's entry, stream, dy, s, weight, rstd, ds): (dx, dresidual or None, dweight).
PyObject *rmsnorm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 8) return PyErr_Format(PyExc_TypeError, "8 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_rmsnorm_bwd))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_rmsnorm_bwd_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        if (PyErr_Occurred()) return nullptr;
        if (dims_of(args[3]) < 1 || args[4] == Py_None) Py_RETURN_NONE;
        Call c(args[3], (size_t)dims_of(args[3]));
        Norm t;
        if (!c.ok || !t.read(c, args[3], args[5], args[4])) Py_RETURN_NONE;
        const at::IntArrayRef all = c.first.sizes();
        const float *const rstd = (const float *)c.need(args[6], at::kFloat, all.slice(0, all.size() - 1));
        const void *const ds = c.in(args[7], t.res, all);
        if (!c.ok) Py_RETURN_NONE;
        const at::Tensor dx = c.fresh(c.io, all), dres = t.res == c.io ? at::Tensor() : c.fresh(t.res, all), dw = c.fresh(at::kFloat, t.dim);
        const size_t bytes = size(t.rows, (int32_t)t.dim);
        const at::Tensor ws = bytes ? c.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(t.x, t.residual, ds, t.weight, rstd, at_of(dx), at_of(dres), (float *)at_of(dw), t.rows, (int32_t)t.dim, c.kind(), t.res_kind(),
                   at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        return result(st, {dx, dres, dw});
    });
}

// q8_values(entry, stream, codes, scales, group, out): out.
PyObject *q8_values(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 6) return PyErr_Format(PyExc_TypeError, "6 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_q8_values))PyLong_AsVoidPtr(args[0]);
        void *const stream = PyLong_AsVoidPtr(args[1]);
        const long group = PyLong_AsLong(args[4]);
        if (PyErr_Occurred()) return nullptr;
        if (dims_of(args[2]) < 1 || group < 0 || group > INT32_MAX) Py_RETURN_NONE;
        const at::Tensor &codes = THPVariable_Unpack(args[2]);
        const at::ScalarType type = codes.scalar_type();
        const at::IntArrayRef all = codes.sizes();
        if (!codes.is_cuda() || !codes.is_contiguous() || (type != at::kFloat8_e4m3fn && type != at::kChar)) Py_RETURN_NONE;
        const int64_t dim = all.back(), rows = dim > 0 ? codes.numel() / dim : 0;
        if (dim < 1 || dim > INT32_MAX) Py_RETURN_NONE;
        std::vector<int64_t> scale(all.begin(), all.end());
        scale.back() = group ? (dim + group - 1) / group : 1;
        const int device = (int)codes.get_device();
        bool ok = true;
        const float *const scales = (const float *)address(args[3], at::kFloat, scale, device, &ok);
        float *given = (float *)optional(args[5], at::kFloat, all, device, &ok);
        if (!ok) Py_RETURN_NONE;
        const at::Tensor out = given ? THPVariable_Unpack(args[5]) : at::empty(all, codes.options().dtype(at::kFloat));
        const c10::DeviceGuard on(codes.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(codes.data_ptr(), scales, type == at::kChar ? SSM_INT8 : SSM_E4M3, (int32_t)group, (float *)out.data_ptr(), rows,
                   (int32_t)dim, stream);
        Py_END_ALLOW_THREADS
        if (st != SSM_OK) return PyLong_FromLong(st);
        written(args[5]);
        return wrap(out);
    });
}

// A setting of the sampling: a tensor with a value for every row, or a number for all.
template <typename T>
const T *setting(Call &c, PyObject *o, at::ScalarType type, int64_t rows, double *all) {
    if (THPVariable_Check(o)) {
        *all = 0;
        return (const T *)c.need(o, type, rows);
    }
    *all = PyFloat_AsDouble(o);
    return nullptr;
}

// sample(entry, workspace size's entry, stream, logits, u, temperature, top_k, top_p, min_p, tokens, logprob,
// want_logprob): (tokens, logprob or None).
PyObject *sample(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 12) return PyErr_Format(PyExc_TypeError, "12 arguments expected, got %zd", n);
    return no_exceptions([&]() -> PyObject * {
        const auto entry = (decltype(&ssm_sample))PyLong_AsVoidPtr(args[0]);
        const auto size = (decltype(&ssm_sample_workspace))PyLong_AsVoidPtr(args[1]);
        void *const stream = PyLong_AsVoidPtr(args[2]);
        if (PyErr_Occurred()) return nullptr;
        if (dims_of(args[3]) != 2) Py_RETURN_NONE;
        Call c(args[3], 2);
        if (!c.ok) Py_RETURN_NONE;
        const int64_t rows = c.first.size(0), vocab = c.first.size(1);
        double t_all, k_all, p_all, m_all;
        const void *const logits = c.need(args[3], c.io, c.first.sizes());
        const float *const u = (const float *)c.need(args[4], at::kFloat, rows);
        const float *const t = setting<float>(c, args[5], at::kFloat, rows, &t_all);
        const int32_t *const k = setting<int32_t>(c, args[6], at::kInt, rows, &k_all);
        const float *const p = setting<float>(c, args[7], at::kFloat, rows, &p_all), *const m = setting<float>(c, args[8], at::kFloat, rows, &m_all);
        if (PyErr_Occurred()) return nullptr;
        if (!c.ok || k_all != std::floor(k_all) || k_all > INT32_MAX || k_all < INT32_MIN) Py_RETURN_NONE;
        const at::Tensor tokens = c.out(args[9], at::kLong, rows);
        const at::Tensor logprob = args[10] != Py_None || args[11] == Py_True ? c.out(args[10], at::kFloat, rows) : at::Tensor();
        if (!c.ok) Py_RETURN_NONE;
        const size_t bytes = size(rows, vocab);
        const at::Tensor ws = bytes ? c.fresh(at::kByte, (int64_t)bytes) : at::Tensor();
        const c10::DeviceGuard on(c.first.device());
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(logits, u, t, (float)t_all, k, (int32_t)k_all, p, (float)p_all, m, (float)m_all, (int64_t *)at_of(tokens),
                   (float *)at_of(logprob), rows, vocab, c.kind(), at_of(ws), bytes, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK)
            for (int i = 9; i < 11; ++i) written(args[i]);
        return result(st, {tokens, logprob});
    });
}

// The node behind a Python object of autograd's graph, or none.
std::shared_ptr<torch::autograd::Node> node_of(PyObject *o) {
    if (torch::autograd::THPCppFunction_Check(o)) return ((torch::autograd::THPCppFunction *)o)->cdata;
    if (THPFunction_Check(o)) return ((THPFunction *)o)->cdata.lock();
    return nullptr;
}

// leaves_elsewhere(next_functions, stream_id): whether a function that a node's gradients come to, the leaves at
// the end among them, works on a stream that is neither this one nor, by the module's `joins`, one that can take
// part in its capture.
PyObject *leaves_elsewhere(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    if (n != 2 || !PyTuple_Check(args[0])) return PyErr_Format(PyExc_TypeError, "a tuple and a stream's id expected");
    return no_exceptions([&]() -> PyObject * {
        const int64_t stream = PyLong_AsLongLong(args[1]);
        if (PyErr_Occurred()) return nullptr;
        std::vector<std::shared_ptr<torch::autograd::Node>> todo;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[0]); ++i) {
            PyObject *const edge = PyTuple_GET_ITEM(args[0], i);
            if (PyTuple_Check(edge) && PyTuple_GET_SIZE(edge) > 0) todo.push_back(node_of(PyTuple_GET_ITEM(edge, 0)));
        }
        std::unordered_set<torch::autograd::Node *> seen;
        std::unordered_map<int64_t, bool> joins;
        joins[stream] = true;
        while (!todo.empty()) {
            const std::shared_ptr<torch::autograd::Node> node = std::move(todo.back());
            todo.pop_back();
            if (!node || !seen.insert(node.get()).second) continue;
            if (const auto on = node->stream()) {
                const auto known = joins.find(on->id());
                bool yes;
                if (known != joins.end()) {
                    yes = known->second;
                } else {
                    PyObject *const asked = PyObject_CallMethod(self, "joins", "L", (long long)on->id());
                    const int truth = asked ? PyObject_IsTrue(asked) : -1;
                    Py_XDECREF(asked);
                    if (truth < 0) return nullptr;
                    yes = joins[on->id()] = truth != 0;
                }
                if (!yes) Py_RETURN_TRUE;
            }
            for (const auto &edge : node->next_edges()) todo.push_back(edge.function);
        }
        Py_RETURN_FALSE;
    });
}

PyMethodDef methods[] = {
    {"gated_fwd", (PyCFunction)(void (*)(void))gated_fwd, METH_FASTCALL, "ssm_gated_fwd for tensors."},
    {"gated_bwd", (PyCFunction)(void (*)(void))gated_bwd, METH_FASTCALL, "ssm_gated_bwd for tensors."},
    {"xent_fwd", (PyCFunction)(void (*)(void))xent_fwd, METH_FASTCALL, "ssm_xent_fwd for tensors."},
    {"xent_bwd", (PyCFunction)(void (*)(void))xent_bwd, METH_FASTCALL, "ssm_xent_bwd for tensors."},
    {"gated_step", (PyCFunction)(void (*)(void))gated_step, METH_FASTCALL, "ssm_gated_step for tensors."},
    {"adamw_step", (PyCFunction)(void (*)(void))adamw_step, METH_FASTCALL, "ssm_adamw_step for lists of tensors."},
    {"linattn_fwd", (PyCFunction)(void (*)(void))linattn_fwd, METH_FASTCALL, "ssm_linattn_fwd for tensors."},
    {"linattn_bwd", (PyCFunction)(void (*)(void))linattn_bwd, METH_FASTCALL, "ssm_linattn_bwd for tensors."},
    {"linattn_step", (PyCFunction)(void (*)(void))linattn_step, METH_FASTCALL, "ssm_linattn_step for tensors."},
    {"rmsnorm_fwd", (PyCFunction)(void (*)(void))rmsnorm_fwd, METH_FASTCALL, "ssm_rmsnorm_fwd for tensors."},
    {"rmsnorm_fwd_q8", (PyCFunction)(void (*)(void))rmsnorm_fwd_q8, METH_FASTCALL, "ssm_rmsnorm_fwd_q8 for tensors."},
    {"rmsnorm_bwd", (PyCFunction)(void (*)(void))rmsnorm_bwd, METH_FASTCALL, "ssm_rmsnorm_bwd for tensors."},
    {"q8_values", (PyCFunction)(void (*)(void))q8_values, METH_FASTCALL, "ssm_q8_values for tensors."},
    {"leaves_elsewhere", (PyCFunction)(void (*)(void))leaves_elsewhere, METH_FASTCALL, "Whether a gradient goes to another stream."},
    {"sample", (PyCFunction)(void (*)(void))sample, METH_FASTCALL, "ssm_sample for tensors."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_table", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_table(void) { return PyModule_Create(&module); }
