// tensors.cpp -- the Python binding's fast path for making output tensors.
//
// A small call of the 8-bit checkpoint operators takes the GPU a few
// microseconds, and torch.empty from Python more than that: on a Grace core,
// around a launch of 2.5 us, 4.0 us in its argument parser and dispatcher,
// and 1.7 us more in the launch that follows, whose code they displace from
// the caches.  The allocation itself takes 0.5.  empty() below goes to it
// directly (1.0 us, and 0.4 in the launch), and returns the same tensor.
//
// Built beside the library for the torch that is installed; without it the
// binding uses torch.empty.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

namespace {

// empty(rows, cols, bf16, device): an uninitialised contiguous float32 (or
// bfloat16) CUDA matrix, from the caching allocator's current stream.
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "empty(rows, cols, bf16, device)");
        return nullptr;
    }
    const long long rows = PyLong_AsLongLong(args[0]);
    const long long cols = PyLong_AsLongLong(args[1]);
    const long bf16 = PyLong_AsLong(args[2]);
    const long device = PyLong_AsLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (rows < 0 || cols < 0 || device < 0 || device > 127) {
        PyErr_SetString(PyExc_ValueError, "negative size or no device index");
        return nullptr;
    }
    HANDLE_TH_ERRORS
    const int64_t size[2] = {rows, cols};
    return THPVariable_Wrap(at::Tensor(at::detail::empty_cuda(
        at::IntArrayRef(size, 2), bf16 ? at::kBFloat16 : at::kFloat,
        at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device)), std::nullopt)));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(empty)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
