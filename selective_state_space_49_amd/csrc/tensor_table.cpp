// tensor_table.cpp -- a CPython extension for the calls whose marshalling in Python would take
// longer than their kernels.
//
// A step over a stack of layers passes several hundred tensors. Asking each of them from
// Python for its address, size, type, device and layout takes 0.45 us a tensor (124 us for
// 281), longer than the step's kernels; here it takes 0.02 us. A single token's call has seven
// tensors and a kernel of 2.6 us.
//
// The entry points of the library come as addresses, from the binding that has loaded it.
#include "ssm_scan.h"

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
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

template <typename F>
PyObject *no_exceptions(F fn) {
    try {
        return fn();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// gated_step(entry, stream, h, x_t, r_t, i_t, decay, c, y_t or None): y_t; the status where the
// library refuses; None where an argument is not as it should be.
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
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry(h, xp, r, i, decay, (float)c, y, all[0], all[1], all[2], io == at::kFloat ? SSM_F32 : SSM_BF16, stream);
        Py_END_ALLOW_THREADS
        if (st == SSM_OK) return out;
        Py_DECREF(out);
        return PyLong_FromLong(st);
    });
}

// adamw_step(entry, stream, block, params, grads, exp_avg, exp_avg_sq, avg_scale, avg_sq_scale,
// grad_scale, lr, beta1, beta2, eps, weight_decay, step): the status; None where an array of the
// moments is not as it should be; a Python error where a parameter or gradient is not.
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
        ssm_status st;
        Py_BEGIN_ALLOW_THREADS
        st = entry((int32_t)t.params.size(), t.params.data(), t.grads.data(), t.sizes.data(), t.kinds.data(),
                   t.grad_kinds.data(), m, v, ms, vs, gs, f[0], f[1], f[2], f[3], f[4], step, stream);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(st);
    });
}

PyMethodDef methods[] = {
    {"gated_step", (PyCFunction)(void (*)(void))gated_step, METH_FASTCALL, "ssm_gated_step for tensors."},
    {"adamw_step", (PyCFunction)(void (*)(void))adamw_step, METH_FASTCALL, "ssm_adamw_step for lists of tensors."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_table", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_table(void) { return PyModule_Create(&module); }
