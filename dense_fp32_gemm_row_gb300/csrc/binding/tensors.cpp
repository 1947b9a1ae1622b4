// tensors.cpp -- the Python binding's fast path for the 8-bit checkpoint
// operators: tensors in, tensors and checkpoints out, one call each.
//
// A small call of these operators takes the GPU a few microseconds, and its
// host side more than that.  On a Grace core, around a launch of 2.5 us, making
// an output by torch.empty from Python takes 4.0 us in its argument parser and
// dispatcher and 1.7 more in the launch that follows, whose code they displace
// from the caches; looking at the operands, making the checkpoint object and
// the foreign-function call take 2 to 3 us.  Here the allocator is called
// directly and the rest costs a few hundred nanoseconds.
//
// Each function handles the ordinary call -- exact tensors of the right type,
// shape and strides on the current device, outputs not given -- and returns
// None for anything else: q8.py then goes through the call step by step, with
// its checks and its errors.  Built beside the library for the torch that is
// installed; without it q8.py does everything that way.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <new>
#include <optional>

#include "gemm_f32.h"

namespace {

// The library's entry points, by address: this module is not linked with it.
struct Library {
    decltype(&gemm_f32_q8_store) store;
    decltype(&gemm_f32_q8_restore) restore;
    decltype(&gemm_f32_q8_wgrad) wgrad;
    decltype(&gemm_f32_q8_gated) gated;
    decltype(&gemm_f32_q8_gated_backward) gated_backward;
    PyObject* check;     // the binding's check(status, where), which raises
    PyTypeObject* type;  // its checkpoint class, which has one slot:
    PyObject* slot;      // the name of the slot for a Held
} lib = {};

// ---- checkpoints ---------------------------------------------------------------

// A checkpoint's arrays and what keeps them: one tensor of bytes made here, or
// the two tensors that the checkpoint was made of.  Whoever has these tensors
// can give them other memory, so q is only as good as the last live().
struct Held {
    PyObject_HEAD
    gemm_f32_q8 q;
    int device;
    at::Tensor bytes;          // the arrays lie in it, from `at`, or
    at::Tensor codes, scales;  // are these
    long long at;
};
PyTypeObject HeldType = {PyVarObject_HEAD_INIT(nullptr, 0)};

Held* held(PyObject* o) { return reinterpret_cast<Held*>(o); }

Held* new_held(const gemm_f32_q8& q, int device) {
    Held* h = held(HeldType.tp_alloc(&HeldType, 0));
    if (!h) throw std::bad_alloc();
    new (&h->bytes) at::Tensor();
    new (&h->codes) at::Tensor();
    new (&h->scales) at::Tensor();
    h->q = q;
    h->device = device;
    return h;
}

void held_dealloc(PyObject* self) {
    Held* h = held(self);
    h->bytes.~Tensor();
    h->codes.~Tensor();
    h->scales.~Tensor();
    Py_TYPE(self)->tp_free(self);
}

// Whether a tensor's last row of `width` bytes lies in its memory.
bool covers(const at::Tensor& t, long long width) {
    const unsigned long long end = t.storage_offset() + (t.size(0) - 1) * t.stride(0) + width;
    return t.storage().nbytes() >= end;
}

// The checkpoint of two byte tensors, if they are as one has to be.
bool describe(const at::Tensor& c, const at::Tensor& s, long long cols, int format,
              gemm_f32_q8* q) {
    for (const at::Tensor* t : {&c, &s})
        if (t->layout() != at::kStrided || !t->is_cuda() || t->scalar_type() != at::kByte ||
            t->dim() != 2)
            return false;
    const long long rows = c.size(0), blocks = (cols + 31) >> 5;
    if (rows < 2 || rows > INT_MAX || cols < 1 || cols > INT_MAX || s.size(0) != rows ||
        c.size(1) < cols || s.size(1) < blocks || c.stride(1) != 1 || s.stride(1) != 1 ||
        c.stride(0) < cols || s.stride(0) < blocks || c.device() != s.device() ||
        !covers(c, cols) || !covers(s, blocks))
        return false;
    q->codes = static_cast<unsigned char*>(c.data_ptr());
    q->scales = static_cast<unsigned char*>(s.data_ptr());
    q->ldcodes = c.stride(0);
    q->ldscales = s.stride(0);
    q->rows = static_cast<int>(rows);
    q->cols = static_cast<int>(cols);
    q->format = format;
    return ((reinterpret_cast<uintptr_t>(q->codes) | reinterpret_cast<uintptr_t>(q->scales) |
             static_cast<uintptr_t>(q->ldcodes | q->ldscales)) & 15) == 0;
}

// Brings h->q up to where its tensors' memory is now; false if that is no
// longer the checkpoint's.
bool live(Held* h) {
    if (!h->bytes.defined()) {
        gemm_f32_q8 now;
        if (!describe(h->codes, h->scales, h->q.cols, h->q.format, &now) ||
            now.rows != h->q.rows || h->codes.device().index() != h->device)
            return false;
        h->q = now;
        return true;
    }
    if (h->bytes.storage().nbytes() < static_cast<size_t>(h->bytes.numel())) return false;
    unsigned char* base = static_cast<unsigned char*>(h->bytes.data_ptr());
    if (!base) return true;  // no elements
    h->q.codes = base + h->at;
    h->q.scales = h->q.codes + h->q.rows * h->q.ldcodes;
    return true;
}

// A row of codes and one of exponents, each padded to 16 bytes.
gemm_f32_q8 layout(long long rows, long long cols, int format) {
    gemm_f32_q8 q = {};
    q.ldcodes = (cols + 15) & ~15LL;
    q.ldscales = (((cols + 31) >> 5) + 15) & ~15LL;
    q.rows = static_cast<int>(rows);
    q.cols = static_cast<int>(cols);
    q.format = format;
    return q;
}

at::Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, int device) {
    return at::Tensor(at::detail::empty_cuda(
        size, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt));
}

// Owns a reference until it is handed on.
struct Ref {
    PyObject* p = nullptr;
    ~Ref() { Py_XDECREF(p); }
    Held* operator->() const { return held(p); }
    PyObject* take() {
        PyObject* r = p;
        p = nullptr;
        return r;
    }
};

// The binding's object around a Held; its class has no other state to set up.
PyObject* checkpoint(const Ref& h) {
    PyObject* q = lib.type->tp_alloc(lib.type, 0);
    if (q && PyObject_SetAttr(q, lib.slot, h.p) < 0) Py_CLEAR(q);
    return q;
}

// `n` uninitialised checkpoints of one layout in one allocation.
void make(const gemm_f32_q8& shape, int device, int n, Ref* out) {
    const long long each = shape.rows * (shape.ldcodes + shape.ldscales);
    const int64_t size = n * each;
    const at::Tensor bytes = new_tensor(at::IntArrayRef(&size, 1), at::kByte, device);
    for (int i = 0; i < n; ++i) {
        Held* h = new_held(shape, device);
        out[i].p = reinterpret_cast<PyObject*>(h);
        h->bytes = bytes;
        h->at = i * each;
        live(h);
    }
}

// held.tensors() -> (codes, scales)
PyObject* held_tensors(PyObject* self, PyObject*) {
    HANDLE_TH_ERRORS
    Held* h = held(self);
    if (h->bytes.defined() && !h->codes.defined()) {
        const long long rows = h->q.rows;
        h->codes = h->bytes.as_strided({rows, h->q.ldcodes}, {h->q.ldcodes, 1}, h->at);
        h->scales = h->bytes.as_strided({rows, h->q.ldscales}, {h->q.ldscales, 1},
                                        h->at + rows * h->q.ldcodes);
    }
    Ref c{THPVariable_Wrap(h->codes)}, s{THPVariable_Wrap(h->scales)};
    return c.p && s.p ? PyTuple_Pack(2, c.p, s.p) : nullptr;
    END_HANDLE_TH_ERRORS
}

template <typename T, T gemm_f32_q8::* field>
PyObject* held_number(PyObject* self, void*) {
    return PyLong_FromLongLong(static_cast<long long>(held(self)->q.*field));
}
template <unsigned char* gemm_f32_q8::* field>
PyObject* held_address(PyObject* self, void*) {
    HANDLE_TH_ERRORS
    if (!live(held(self))) {
        PyErr_SetString(PyExc_ValueError, "the checkpoint's tensors no longer hold it");
        return nullptr;
    }
    return PyLong_FromVoidPtr(held(self)->q.*field);
    END_HANDLE_TH_ERRORS
}
PyObject* held_device(PyObject* self, void*) { return PyLong_FromLong(held(self)->device); }

PyMethodDef held_methods[] = {{"tensors", held_tensors, METH_NOARGS, nullptr},
                              {nullptr, nullptr, 0, nullptr}};
PyGetSetDef held_fields[] = {
    {"rows", held_number<int, &gemm_f32_q8::rows>, nullptr, nullptr, nullptr},
    {"cols", held_number<int, &gemm_f32_q8::cols>, nullptr, nullptr, nullptr},
    {"format", held_number<int, &gemm_f32_q8::format>, nullptr, nullptr, nullptr},
    {"ldcodes", held_number<long long, &gemm_f32_q8::ldcodes>, nullptr, nullptr, nullptr},
    {"ldscales", held_number<long long, &gemm_f32_q8::ldscales>, nullptr, nullptr, nullptr},
    {"codes", held_address<&gemm_f32_q8::codes>, nullptr, nullptr, nullptr},
    {"scales", held_address<&gemm_f32_q8::scales>, nullptr, nullptr, nullptr},
    {"device", held_device, nullptr, nullptr, nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};

// ---- operands ------------------------------------------------------------------

bool is_held(PyObject* o) { return Py_TYPE(o) == &HeldType && live(held(o)); }

// A float32 CUDA matrix with contiguous rows on the current device.
struct Matrix {
    float* p;
    long long rows, cols, ld;
    int device;
};
bool matrix(PyObject* o, Matrix* m) {
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.scalar_type() != at::kFloat || t.dim() != 2)
        return false;
    m->rows = t.size(0);
    m->cols = t.size(1);
    m->device = t.device().index();
    if (m->rows > INT_MAX || m->cols > INT_MAX) return false;
    if (m->device != c10::cuda::current_device()) return false;
    if (m->cols > 1 && t.stride(1) != 1) return false;
    m->ld = m->rows > 1 ? t.stride(0) : m->cols > 1 ? m->cols : 1;
    if (m->ld < m->cols || m->ld < 1) return false;
    m->p = static_cast<float*>(t.data_ptr());
    return true;
}

at::Tensor empty(long long rows, long long cols, bool bf16, int device) {
    const int64_t size[2] = {rows, cols};
    return new_tensor(at::IntArrayRef(size, 2), bf16 ? at::kBFloat16 : at::kFloat, device);
}
float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }
long long row(long long cols) { return cols > 1 ? cols : 1; }
cudaStream_t stream_of(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

bool ints(PyObject* const* args, Py_ssize_t n, long* out) {
    for (Py_ssize_t i = 0; i < n; ++i) out[i] = PyLong_AsLong(args[i]);
    return !PyErr_Occurred();
}
bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return n == want;
}

// Runs f() without the interpreter's lock; false, with the error set, if it failed.
template <typename F>
bool call(const char* where, F f) {
    int st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS if (st == 0) return true;
    Py_XDECREF(PyObject_CallFunction(lib.check, "is", st, where));
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, st);
    return false;
}

// ---- the functions -------------------------------------------------------------

// bind(store, restore, wgrad, gated, gated_backward, check, type, torch): the
// library's addresses, what the binding gives, and the version of the torch
// that is running, which has to be the one whose headers this was built with
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!count(n, 8)) return nullptr;
    const char* running = PyUnicode_AsUTF8(args[7]);
    if (!running) return nullptr;
    if (std::strcmp(running, TENSORS_TORCH) != 0) {
        PyErr_Format(PyExc_ImportError, "built for torch %s, not %s", TENSORS_TORCH, running);
        return nullptr;
    }
    void* p[5];
    for (int i = 0; i < 5; ++i) p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    lib.store = reinterpret_cast<decltype(lib.store)>(p[0]);
    lib.restore = reinterpret_cast<decltype(lib.restore)>(p[1]);
    lib.wgrad = reinterpret_cast<decltype(lib.wgrad)>(p[2]);
    lib.gated = reinterpret_cast<decltype(lib.gated)>(p[3]);
    lib.gated_backward = reinterpret_cast<decltype(lib.gated_backward)>(p[4]);
    if (!PyType_Check(args[6])) {
        PyErr_SetString(PyExc_TypeError, "the checkpoint class is a type");
        return nullptr;
    }
    if (!lib.slot) lib.slot = PyUnicode_InternFromString("_held");
    if (!lib.slot) return nullptr;
    Py_INCREF(args[5]);
    Py_INCREF(args[6]);
    Py_XDECREF(lib.check);
    Py_XDECREF(lib.type);
    lib.check = args[5];
    lib.type = reinterpret_cast<PyTypeObject*>(args[6]);
    Py_RETURN_NONE;
}

// empty(rows, cols, bf16, device): an uninitialised matrix
PyObject* py_empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 4)) return nullptr;
    const long long rows = PyLong_AsLongLong(args[0]), cols = PyLong_AsLongLong(args[1]);
    long v[2];
    if (!ints(args + 2, 2, v) || PyErr_Occurred()) return nullptr;
    if (rows < 0 || cols < 0 || v[1] < 0 || v[1] > 127) {
        PyErr_SetString(PyExc_ValueError, "negative size or no device index");
        return nullptr;
    }
    return THPVariable_Wrap(empty(rows, cols, v[0] != 0, static_cast<int>(v[1])));
    END_HANDLE_TH_ERRORS
}

// make(rows, cols, format, device): an uninitialised checkpoint
PyObject* py_make(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long v[4];
    if (!count(n, 4) || !ints(args, 4, v)) return nullptr;
    if (v[0] < 0 || v[1] < 0 || v[0] > INT_MAX || v[1] > INT_MAX || v[3] < 0 || v[3] > 127) {
        PyErr_SetString(PyExc_ValueError, "a size or device out of range");
        return nullptr;
    }
    Ref out;
    make(layout(v[0], v[1], static_cast<int>(v[2])), static_cast<int>(v[3]), 1, &out);
    return checkpoint(out);
    END_HANDLE_TH_ERRORS
}

// wrap(codes, scales, cols, format): the Held of two byte tensors, or None
PyObject* wrap(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long v[2];
    if (!count(n, 4)) return nullptr;
    if (!THPVariable_CheckExact(args[0]) || !THPVariable_CheckExact(args[1]) ||
        !PyLong_CheckExact(args[2]))
        Py_RETURN_NONE;
    if (!ints(args + 2, 2, v)) return nullptr;
    const at::Tensor &c = THPVariable_Unpack(args[0]), &s = THPVariable_Unpack(args[1]);
    gemm_f32_q8 q = {};
    if (!describe(c, s, v[0], static_cast<int>(v[1]), &q)) Py_RETURN_NONE;
    Held* h = new_held(q, c.device().index());
    h->codes = c;
    h->scales = s;
    return reinterpret_cast<PyObject*>(h);
    END_HANDLE_TH_ERRORS
}

// store(x, format) -> checkpoint
PyObject* store(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long format;
    Matrix x;
    if (!count(n, 2) || !ints(args + 1, 1, &format)) return nullptr;
    if (!matrix(args[0], &x)) Py_RETURN_NONE;
    Ref out;
    make(layout(x.rows, x.cols, static_cast<int>(format)), x.device, 1, &out);
    const cudaStream_t s = stream_of(x.device);
    if (!call("q8_store", [&] { return lib.store(x.p, x.ld, &out->q, s); })) return nullptr;
    return checkpoint(out);
    END_HANDLE_TH_ERRORS
}

// restore(checkpoint, bf16) -> tensor
PyObject* restore(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long bf16;
    if (!count(n, 2) || !ints(args + 1, 1, &bf16)) return nullptr;
    if (!is_held(args[0]) || held(args[0])->device != c10::cuda::current_device()) Py_RETURN_NONE;
    const Held* h = held(args[0]);
    const at::Tensor x = empty(h->q.rows, h->q.cols, bf16 != 0, h->device);
    void* p = x.data_ptr();
    const cudaStream_t s = stream_of(h->device);
    if (!call("q8_restore", [&] {
            return lib.restore(&h->q, p, row(h->q.cols),
                               bf16 ? GEMM_F32_Q8_TO_BF16 : GEMM_F32_Q8_TO_F32, s);
        }))
        return nullptr;
    return THPVariable_Wrap(x);
    END_HANDLE_TH_ERRORS
}

// wgrad(checkpoint, dy) -> dw
PyObject* wgrad(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Matrix dy;
    if (!count(n, 2)) return nullptr;
    if (!is_held(args[0]) || !matrix(args[1], &dy)) Py_RETURN_NONE;
    const Held* h = held(args[0]);
    if (dy.rows != h->q.rows || dy.device != h->device) Py_RETURN_NONE;
    const at::Tensor dw = empty(h->q.cols, dy.cols, false, h->device);
    float* p = floats(dw);
    const cudaStream_t s = stream_of(h->device);
    if (!call("q8_wgrad", [&] {
            return lib.wgrad(&h->q, dy.p, dy.ld, static_cast<int>(dy.cols), 1.0f, 0.0f, p,
                             row(dy.cols), GEMM_F32_ALGO_AUTO, 0, s);
        }))
        return nullptr;
    return THPVariable_Wrap(dw);
    END_HANDLE_TH_ERRORS
}

PyObject* three(Ref& a, Ref& b, Ref& c) {
    PyObject* out = a.p && b.p && c.p ? PyTuple_New(3) : nullptr;
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, a.take());
    PyTuple_SET_ITEM(out, 1, b.take());
    PyTuple_SET_ITEM(out, 2, c.take());
    return out;
}

// gated(gate, up, act, format) -> (h, checkpoint of gate, checkpoint of up)
PyObject* gated(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long v[2];
    Matrix g, u;
    if (!count(n, 4) || !ints(args + 2, 2, v)) return nullptr;
    if (!matrix(args[0], &g) || !matrix(args[1], &u) || g.rows != u.rows || g.cols != u.cols)
        Py_RETURN_NONE;
    const at::Tensor y = empty(g.rows, g.cols, false, g.device);
    Ref q[2];
    make(layout(g.rows, g.cols, static_cast<int>(v[1])), g.device, 2, q);
    float* p = floats(y);
    const cudaStream_t s = stream_of(g.device);
    if (!call("q8_gated", [&] {
            return lib.gated(static_cast<int>(v[0]), g.p, g.ld, u.p, u.ld, p, row(g.cols), &q[0]->q,
                             &q[1]->q, s);
        }))
        return nullptr;
    Ref t{THPVariable_Wrap(y)}, gq{checkpoint(q[0])}, uq{checkpoint(q[1])};
    return three(t, gq, uq);
    END_HANDLE_TH_ERRORS
}

// gated_backward(gate, up, dh, act, want_h) -> (dgate, dup, checkpoint or None)
PyObject* gated_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long v[2];
    Matrix d;
    if (!count(n, 5) || !ints(args + 3, 2, v)) return nullptr;
    if (!is_held(args[0]) || !is_held(args[1]) || !matrix(args[2], &d)) Py_RETURN_NONE;
    const Held *g = held(args[0]), *u = held(args[1]);
    if (d.rows != g->q.rows || d.cols != g->q.cols || u->q.rows != g->q.rows ||
        u->q.cols != g->q.cols || u->q.format != g->q.format || d.device != g->device ||
        u->device != g->device)
        Py_RETURN_NONE;
    const at::Tensor dg = empty(d.rows, d.cols, false, d.device);
    const at::Tensor du = empty(d.rows, d.cols, false, d.device);
    Ref q;
    if (v[1]) make(layout(d.rows, d.cols, g->q.format), d.device, 1, &q);
    float *pg = floats(dg), *pu = floats(du);
    const cudaStream_t s = stream_of(d.device);
    if (!call("q8_gated_backward", [&] {
            return lib.gated_backward(static_cast<int>(v[0]), &g->q, &u->q, d.p, d.ld, pg,
                                      row(d.cols), pu, row(d.cols), q.p ? &q->q : nullptr, s);
        }))
        return nullptr;
    Ref tg{THPVariable_Wrap(dg)}, tu{THPVariable_Wrap(du)}, hq;
    if (q.p) {
        hq.p = checkpoint(q);
    } else {
        Py_INCREF(Py_None);
        hq.p = Py_None;
    }
    return three(tg, tu, hq);
    END_HANDLE_TH_ERRORS
}

typedef PyObject* (*Fast)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction as_c(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {{"bind", as_c(bind), METH_FASTCALL, nullptr},
                         {"empty", as_c(py_empty), METH_FASTCALL, nullptr},
                         {"make", as_c(py_make), METH_FASTCALL, nullptr},
                         {"wrap", as_c(wrap), METH_FASTCALL, nullptr},
                         {"store", as_c(store), METH_FASTCALL, nullptr},
                         {"restore", as_c(restore), METH_FASTCALL, nullptr},
                         {"wgrad", as_c(wgrad), METH_FASTCALL, nullptr},
                         {"gated", as_c(gated), METH_FASTCALL, nullptr},
                         {"gated_backward", as_c(gated_backward), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) {
    HeldType.tp_name = "dense_fp32_gemm_row_gb300._tensors.Held";
    HeldType.tp_basicsize = sizeof(Held);
    HeldType.tp_dealloc = held_dealloc;
    HeldType.tp_flags = Py_TPFLAGS_DEFAULT;
    HeldType.tp_methods = held_methods;
    HeldType.tp_getset = held_fields;
    if (PyType_Ready(&HeldType) < 0) return nullptr;
    return PyModule_Create(&module);
}
