// tensors.cpp -- the Python binding's fast path for the 8-bit checkpoint
// operators and the 8-bit integer layers: tensors in, tensors, checkpoints and
// 8-bit matrices out, one call each.
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
// None for anything else: q8.py or i8.py then goes through the call step by
// step, with its checks and its errors.  Built beside the library for the torch
// that is installed; without it they do everything that way.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
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

// A dense CUDA tensor whose memory holds its values as they are, not a view of
// their negatives.
bool plain(const at::Tensor& t) {
    return t.layout() == at::kStrided && t.is_cuda() && !t.is_neg();
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
        if (!plain(*t) || t->scalar_type() != at::kByte || t->dim() != 2)
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
    if (!plain(t) || t.scalar_type() != at::kFloat || t.dim() != 2)
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

// ---- 8-bit integer layers ------------------------------------------------------

struct I8Library {
    decltype(&gemm_f32_i8_store) store;
    decltype(&gemm_f32_i8_norm) norm;
    decltype(&gemm_f32_i8_matmul) matmul;
    decltype(&gemm_f32_i8_gated) gated;
    PyTypeObject* type;                // the binding's class, with three slots:
    PyObject *codes, *scales, *cols;   // their names
} i8 = {};

// An 8-bit matrix as its tensors have it now; the tensors are kept until the
// call has been made.
struct I8Operand {
    gemm_f32_i8 q = {};
    int device = -1;
    Ref codes, scales;
};
bool i8_describe(const at::Tensor& c, const at::Tensor& s, long long cols, I8Operand* m) {
    if (!plain(c) || c.scalar_type() != at::kChar || c.dim() != 2 || !plain(s) ||
        s.scalar_type() != at::kFloat || s.dim() != 1)
        return false;
    const long long rows = c.size(0), width = c.size(1);
    if (rows < 1 || rows > INT_MAX || cols < 1 || cols > INT_MAX || width < cols ||
        s.size(0) != rows || (width > 1 && c.stride(1) != 1) || (rows > 1 && s.stride(0) != 1) ||
        c.device() != s.device())
        return false;
    const long long ld = rows > 1 ? c.stride(0) : (width + 15) & ~15LL;
    if (ld < cols || !covers(c, cols) ||
        s.storage().nbytes() < 4 * static_cast<unsigned long long>(s.storage_offset() + rows))
        return false;
    m->q.codes = static_cast<signed char*>(c.data_ptr());
    m->q.scales = static_cast<float*>(s.data_ptr());
    m->q.ld = ld;
    m->q.rows = static_cast<int>(rows);
    m->q.cols = static_cast<int>(cols);
    m->device = c.device().index();
    return ((reinterpret_cast<uintptr_t>(m->q.codes) | static_cast<uintptr_t>(ld)) & 15) == 0;
}
// False without an error: not the ordinary case.
bool i8_operand(PyObject* o, I8Operand* m) {
    if (Py_TYPE(o) != i8.type) return false;
    m->codes.p = PyObject_GetAttr(o, i8.codes);
    m->scales.p = PyObject_GetAttr(o, i8.scales);
    const Ref cols{PyObject_GetAttr(o, i8.cols)};
    if (!m->codes.p || !m->scales.p || !cols.p) {
        PyErr_Clear();
        return false;
    }
    if (!THPVariable_CheckExact(m->codes.p) || !THPVariable_CheckExact(m->scales.p) ||
        !PyLong_CheckExact(cols.p))
        return false;
    const long long n = PyLong_AsLongLong(cols.p);
    if (n == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return i8_describe(THPVariable_Unpack(m->codes.p), THPVariable_Unpack(m->scales.p), n, m) &&
           m->device == c10::cuda::current_device();
}

// A new matrix of rows padded to 16 bytes, codes and scales behind them in one
// allocation (a second one and its end cost a microsecond).
struct I8New {
    at::Tensor codes, scales;
    gemm_f32_i8 q;
    I8New(long long rows, long long cols, int device) {
        const long long ld = (cols + 15) & ~15LL;
        const int64_t bytes = rows * ld + 4 * rows, size[2] = {rows, ld}, strides[2] = {ld, 1};
        codes = new_tensor(at::IntArrayRef(&bytes, 1), at::kChar, device);
        scales = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(codes.storage()),
                                                          codes.key_set(),
                                                          caffe2::TypeMeta::Make<float>());
        scales.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(size, 1),
                                                            at::IntArrayRef(strides + 1, 1),
                                                            rows * ld / 4);
        codes.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(size, 2),
                                                           at::IntArrayRef(strides, 2));
        q = {static_cast<signed char*>(codes.data_ptr()), floats(scales), ld,
             static_cast<int>(rows), static_cast<int>(cols)};
    }
    // The binding's object.
    PyObject* object() const {
        Ref o{i8.type->tp_alloc(i8.type, 0)};
        const Ref c{THPVariable_Wrap(codes)}, s{THPVariable_Wrap(scales)},
            n{PyLong_FromLong(q.cols)};
        if (!o.p || !c.p || !s.p || !n.p || PyObject_SetAttr(o.p, i8.codes, c.p) < 0 ||
            PyObject_SetAttr(o.p, i8.scales, s.p) < 0 || PyObject_SetAttr(o.p, i8.cols, n.p) < 0)
            return nullptr;
        return o.take();
    }
};

// A float32 or bfloat16 CUDA matrix with contiguous rows and elements, on the
// current device.
struct AnyMatrix {
    void* p;
    long long rows, cols, ld;
    int device, type;
};
bool any_matrix(PyObject* o, AnyMatrix* m) {
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!plain(t) || t.dim() != 2) return false;
    const at::ScalarType type = t.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) return false;
    m->type = type == at::kFloat ? GEMM_F32_TYPE_F32 : GEMM_F32_TYPE_BF16;
    m->rows = t.size(0);
    m->cols = t.size(1);
    m->device = t.device().index();
    if (m->rows < 1 || m->cols < 1 || m->rows > INT_MAX || m->cols > INT_MAX) return false;
    if (m->device != c10::cuda::current_device()) return false;
    if (m->cols > 1 && t.stride(1) != 1) return false;
    m->ld = m->rows > 1 ? t.stride(0) : m->cols;
    if (m->ld < m->cols) return false;
    m->p = t.data_ptr();
    return true;
}

at::Tensor i8_output(long long rows, long long cols, int type, int device) {
    const int64_t size[2] = {rows, cols};
    return new_tensor(at::IntArrayRef(size, 2),
                      type == GEMM_F32_TYPE_BF16  ? at::kBFloat16
                      : type == GEMM_F32_TYPE_I32 ? at::kInt
                                                  : at::kFloat,
                      device);
}

// bind_i8(store, norm, matmul, gated, type): after bind()
PyObject* bind_i8(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!count(n, 5)) return nullptr;
    void* p[4];
    for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    if (!PyType_Check(args[4])) {
        PyErr_SetString(PyExc_TypeError, "the class of 8-bit matrices is a type");
        return nullptr;
    }
    if (!i8.codes) i8.codes = PyUnicode_InternFromString("codes");
    if (!i8.scales) i8.scales = PyUnicode_InternFromString("scales");
    if (!i8.cols) i8.cols = PyUnicode_InternFromString("cols");
    if (!i8.codes || !i8.scales || !i8.cols) return nullptr;
    i8.store = reinterpret_cast<decltype(i8.store)>(p[0]);
    i8.norm = reinterpret_cast<decltype(i8.norm)>(p[1]);
    i8.matmul = reinterpret_cast<decltype(i8.matmul)>(p[2]);
    i8.gated = reinterpret_cast<decltype(i8.gated)>(p[3]);
    Py_INCREF(args[4]);
    Py_XDECREF(i8.type);
    i8.type = reinterpret_cast<PyTypeObject*>(args[4]);
    Py_RETURN_NONE;
}

// i8_fits(codes, scales, cols): whether they are an ordinary matrix
PyObject* i8_fits(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 3)) return nullptr;
    if (!THPVariable_CheckExact(args[0]) || !THPVariable_CheckExact(args[1]) ||
        !PyLong_CheckExact(args[2]))
        Py_RETURN_FALSE;
    const long long cols = PyLong_AsLongLong(args[2]);
    if (cols == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_FALSE;
    }
    I8Operand m;
    if (i8_describe(THPVariable_Unpack(args[0]), THPVariable_Unpack(args[1]), cols, &m))
        Py_RETURN_TRUE;
    Py_RETURN_FALSE;
    END_HANDLE_TH_ERRORS
}

// i8_store(x) -> matrix
PyObject* i8_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    AnyMatrix x;
    if (!count(n, 1)) return nullptr;
    if (!any_matrix(args[0], &x)) Py_RETURN_NONE;
    const I8New out(x.rows, x.cols, x.device);
    const cudaStream_t s = stream_of(x.device);
    if (!call("i8_store", [&] { return i8.store(x.p, x.type, x.ld, &out.q, s); })) return nullptr;
    return out.object();
    END_HANDLE_TH_ERRORS
}

// i8_norm(x, weight, residual or None, eps) -> (matrix, sum or None)
PyObject* i8_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    AnyMatrix x, r = {};
    if (!count(n, 4)) return nullptr;
    if (!any_matrix(args[0], &x) || !THPVariable_CheckExact(args[1]) || !PyFloat_CheckExact(args[3]))
        Py_RETURN_NONE;
    const double given = PyFloat_AS_DOUBLE(args[3]);
    const float eps = static_cast<float>(given);
    const at::Tensor& w = THPVariable_Unpack(args[1]);
    if (!plain(w) || w.device().index() != x.device ||
        w.scalar_type() != (x.type == GEMM_F32_TYPE_F32 ? at::kFloat : at::kBFloat16) ||
        w.dim() != 1 || w.size(0) != x.cols || (x.cols > 1 && w.stride(0) != 1) ||
        !(given >= 1e-30) || !std::isfinite(eps))
        Py_RETURN_NONE;
    const bool residual = args[2] != Py_None;
    if (residual && (!any_matrix(args[2], &r) || r.type != x.type || r.rows != x.rows ||
                     r.cols != x.cols))
        Py_RETURN_NONE;
    const I8New out(x.rows, x.cols, x.device);
    at::Tensor sum;
    if (residual) sum = i8_output(x.rows, x.cols, x.type, x.device);
    void *pw = w.data_ptr(), *ps = residual ? sum.data_ptr() : nullptr;
    const cudaStream_t s = stream_of(x.device);
    if (!call("i8_norm", [&] {
            return i8.norm(x.p, x.ld, r.p, r.ld, pw, eps, x.type, ps, x.cols, &out.q, s);
        }))
        return nullptr;
    Ref q{out.object()}, t;
    if (residual) {
        t.p = THPVariable_Wrap(sum);
    } else {
        Py_INCREF(Py_None);
        t.p = Py_None;
    }
    return q.p && t.p ? PyTuple_Pack(2, q.p, t.p) : nullptr;
    END_HANDLE_TH_ERRORS
}

// i8_matmul(a, w, type) -> tensor
PyObject* i8_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long type;
    I8Operand a, w;
    if (!count(n, 3) || !ints(args + 2, 1, &type)) return nullptr;
    if (!i8_operand(args[0], &a) || !i8_operand(args[1], &w) || a.q.cols != w.q.cols ||
        a.q.cols > GEMM_F32_I8_MAX_COLS || a.device != w.device)
        Py_RETURN_NONE;
    const at::Tensor y = i8_output(a.q.rows, w.q.rows, static_cast<int>(type), a.device);
    void* p = y.data_ptr();
    const cudaStream_t s = stream_of(a.device);
    if (!call("i8_matmul", [&] {
            return i8.matmul(&a.q, &w.q, p, static_cast<int>(type), w.q.rows, GEMM_F32_ALGO_AUTO, 0,
                             s);
        }))
        return nullptr;
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// i8_gated(a, gate, up, act, type) -> tensor
PyObject* i8_gated(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long v[2];
    I8Operand a, g, u;
    if (!count(n, 5) || !ints(args + 3, 2, v)) return nullptr;
    if (!i8_operand(args[0], &a) || !i8_operand(args[1], &g) || !i8_operand(args[2], &u) ||
        a.q.cols != g.q.cols || a.q.cols > GEMM_F32_I8_MAX_COLS || u.q.cols != g.q.cols ||
        u.q.rows != g.q.rows || a.device != g.device || a.device != u.device)
        Py_RETURN_NONE;
    const at::Tensor h = i8_output(a.q.rows, g.q.rows, static_cast<int>(v[1]), a.device);
    void* p = h.data_ptr();
    const cudaStream_t s = stream_of(a.device);
    if (!call("i8_gated", [&] {
            return i8.gated(static_cast<int>(v[0]), &a.q, &g.q, &u.q, p, static_cast<int>(v[1]),
                            g.q.rows, GEMM_F32_ALGO_AUTO, 0, s);
        }))
        return nullptr;
    return THPVariable_Wrap(h);
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
                         {"bind_i8", as_c(bind_i8), METH_FASTCALL, nullptr},
                         {"i8_fits", as_c(i8_fits), METH_FASTCALL, nullptr},
                         {"i8_store", as_c(i8_store), METH_FASTCALL, nullptr},
                         {"i8_norm", as_c(i8_norm), METH_FASTCALL, nullptr},
                         {"i8_matmul", as_c(i8_matmul), METH_FASTCALL, nullptr},
                         {"i8_gated", as_c(i8_gated), METH_FASTCALL, nullptr},
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
