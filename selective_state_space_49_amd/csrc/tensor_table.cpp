// tensor_table.cpp -- a CPython extension that reads lists of tensors for ssm_adamw_step.
//
// A step over a stack of layers passes several hundred tensors. Asking each of them from
// Python for its address, size, type, device and layout takes 0.45 us a tensor (124 us for
// 281), longer than the step's kernels; here it takes 0.02 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>

namespace {

constexpr int kF32 = 0, kBf16 = 1;  // ssm_dtype

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
    return t.scalar_type() == at::kFloat ? kF32 : kBf16;
}

// table(params, grads, block): bytes of n addresses, n gradient addresses (0 for None), n
// sizes, n parameter types, n gradient types; their address; and the sum of the sizes in
// blocks, each rounded up.
PyObject *table(PyObject *, PyObject *args) {
    PyObject *params, *grads;
    long long block;
    if (!PyArg_ParseTuple(args, "O!O!L", &PyList_Type, &params, &PyList_Type, &grads, &block)) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(params);
    if (PyList_GET_SIZE(grads) != n)
        return PyErr_Format(PyExc_ValueError, "%zd parameters and %zd gradients", n, PyList_GET_SIZE(grads));
    PyObject *bytes = PyBytes_FromStringAndSize(nullptr, n * (3 * 8 + 2 * 4));
    if (!bytes) return nullptr;
    char *const base = PyBytes_AS_STRING(bytes);
    auto put = [&](Py_ssize_t column, Py_ssize_t k, const void *v, size_t size) {
        std::memcpy(base + (column < 3 ? column * n * 8 : 3 * n * 8 + (column - 3) * n * 4) + k * (Py_ssize_t)size, v, size);
    };
    long long blocks = 0;
    int device = -1;
    try {
        for (Py_ssize_t k = 0; k < n; ++k) {
            PyObject *po = PyList_GET_ITEM(params, k), *go = PyList_GET_ITEM(grads, k);
            if (!THPVariable_Check(po) || (go != Py_None && !THPVariable_Check(go))) {
                PyErr_Format(PyExc_TypeError, "parameter and gradient %zd must be tensors", k);
                break;
            }
            const at::Tensor &p = THPVariable_Unpack(po);
            const int32_t pk = kind_of(p, &device, "parameter", k);
            if (pk < 0) break;
            const uint64_t pa = (uint64_t)(uintptr_t)p.data_ptr();
            const int64_t size = p.numel();
            uint64_t ga = 0;
            int32_t gk = kF32;
            if (go != Py_None) {
                const at::Tensor &g = THPVariable_Unpack(go);
                gk = kind_of(g, &device, "gradient", k);
                if (gk < 0) break;
                if (g.sizes() != p.sizes()) {
                    PyErr_Format(PyExc_ValueError, "gradient %zd must have its parameter's shape", k);
                    break;
                }
                ga = (uint64_t)(uintptr_t)g.data_ptr();
            }
            put(0, k, &pa, 8);
            put(1, k, &ga, 8);
            put(2, k, &size, 8);
            put(3, k, &pk, 4);
            put(4, k, &gk, 4);
            blocks += (size + block - 1) / block;
        }
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    if (PyErr_Occurred()) {
        Py_DECREF(bytes);
        return nullptr;
    }
    return Py_BuildValue("NKL", bytes, (unsigned long long)(uintptr_t)base, blocks);
}

PyMethodDef methods[] = {{"table", table, METH_VARARGS, "The host arrays of ssm_adamw_step for lists of tensors."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_table", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_table(void) { return PyModule_Create(&module); }
