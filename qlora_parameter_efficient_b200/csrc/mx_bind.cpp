// mx_bind.cpp -- the short way from Python into the microscaled calls of libqlora.
//
// At one token or a few dozen the GPU work of these calls takes 4 to 15 us, and going through ctypes (argument
// conversion, a Stream object, torch.empty) takes as long again.  This module checks the arguments, allocates
// the outputs and makes the same C call in under a microsecond of its own.  It handles the plain case only
// -- every tensor as documented, on the current device -- and answers None for anything else, which
// the Python functions then check, and refuse with a reason or run, themselves.  It holds no state but
// the addresses of the library's functions.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/qlora.h"

namespace {

struct Lib {
    decltype(&qlora_workspace_bytes) workspace_bytes;
    decltype(&mxfp4_quantize) mx_quantize;
    decltype(&mxfp4_dequantize) mx_dequantize;
    decltype(&qlora_act8_quantize) a8_quantize;
    decltype(&qlora_act8_dequantize) a8_dequantize;
    decltype(&qlora_linear_fwd_mxfp4) fwd;
    decltype(&qlora_linear_bwd_mxfp4) bwd_mx;
    decltype(&qlora_linear_bwd_act8) bwd_a8;
} g_lib;

// An argument that is not what the plain case takes.
struct NotPlain {};

// Tensors of one call: all contiguous, on one CUDA device, which is the current one.
struct Args {
    int device = -1;

    const at::Tensor& any(PyObject* o) {
        if (!THPVariable_Check(o)) throw NotPlain{};
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || !t.is_contiguous()) throw NotPlain{};
        if (device < 0) {
            device = t.get_device();
            if (device != c10::cuda::current_device()) throw NotPlain{};
        } else if (t.get_device() != device) {
            throw NotPlain{};
        }
        return t;
    }
    void* get(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols) {
        const at::Tensor& t = any(o);
        if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) throw NotPlain{};
        return t.data_ptr();
    }
    void* flat(PyObject* o, at::ScalarType type, int64_t n) {
        const at::Tensor& t = any(o);
        if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n) throw NotPlain{};
        return t.data_ptr();
    }
    at::Tensor empty(at::ScalarType type, at::IntArrayRef shape) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

constexpr auto kBf = at::kBFloat16;
constexpr auto kF32 = at::kFloat;

// Without the interpreter's lock, as any call that may wait for the GPU or for the allocator.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// An output: the caller's tensor, checked at once, or one made by ptr() (which needs no interpreter).
struct Out {
    PyObject* given;
    at::ScalarType type;
    int64_t rows, cols;
    void* p = nullptr;
    at::Tensor made;

    Out(Args& a, PyObject* o, at::ScalarType type, int64_t rows, int64_t cols)
        : given(o), type(type), rows(rows), cols(cols) {
        if (given != Py_None) p = a.get(given, type, rows, cols);
    }
    void* ptr(const Args& a) {
        if (given == Py_None) {
            made = a.empty(type, {rows, cols});
            p = made.data_ptr();
        }
        return p;
    }
    // new reference to the tensor, None where there is none
    PyObject* object() {
        if (made.defined()) return THPVariable_Wrap(std::move(made));
        Py_INCREF(given);
        return given;
    }
};

// (a, b) or (a, b, c) of new references, all taken over
PyObject* tuple(PyObject* a, PyObject* b, PyObject* c = nullptr) {
    PyObject* t = a && b ? PyTuple_New(c ? 3 : 2) : nullptr;
    if (!t) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    if (c) PyTuple_SET_ITEM(t, 2, c);
    return t;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw NotPlain{};
    return v != 0;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return static_cast<float>(v);
}

// [rows, cols] of a two-dimensional tensor.
void shape2(PyObject* o, int64_t& rows, int64_t& cols) {
    if (!THPVariable_Check(o)) throw NotPlain{};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 2) throw NotPlain{};
    rows = t.size(0);
    cols = t.size(1);
}

qlora_dtype source_type(const at::Tensor& t) {
    if (t.scalar_type() == kBf) return QLORA_BF16;
    if (t.scalar_type() == kF32) return QLORA_F32;
    throw NotPlain{};
}

// The caller's workspace, or one made by ptr().
struct Workspace {
    size_t bytes = 0;
    void* p = nullptr;
    at::Tensor made;

    Workspace(Args& a, PyObject* ws, int op, int64_t T, int64_t d_out, int64_t d_in, int32_t r) {
        if (ws == Py_None) {
            bytes = g_lib.workspace_bytes(op, QLORA_BF16, T, d_out, d_in, r);
            if (!bytes) throw NotPlain{};
        } else {
            const at::Tensor& t = a.any(ws);
            bytes = t.nbytes();
            p = t.data_ptr();
        }
    }
    void* ptr(const Args& a) {
        if (!p) {
            made = a.empty(at::kByte, {static_cast<int64_t>(bytes)});
            p = made.data_ptr();
        }
        return p;
    }
};

PyObject* status(qlora_status s) { return PyLong_FromLong(static_cast<long>(s)); }

// Run f; None where the call is not a plain one, and no C++ exception past this point (an
// allocation that fails raises torch's own error on the way that Python takes then).
template <typename F>
PyObject* plain(F f) {
    try {
        return f();
    } catch (const NotPlain&) {
    } catch (const std::exception&) {
    }
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NONE;
}

// init(addresses): of the eight functions, in Lib's order
PyObject* init(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 8) return PyErr_Format(PyExc_TypeError, "init takes 8 addresses");
    void* p[8];
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (!p[i]) return PyErr_Format(PyExc_ValueError, "address %d is null", i);
    }
    g_lib.workspace_bytes = reinterpret_cast<decltype(g_lib.workspace_bytes)>(p[0]);
    g_lib.mx_quantize = reinterpret_cast<decltype(g_lib.mx_quantize)>(p[1]);
    g_lib.mx_dequantize = reinterpret_cast<decltype(g_lib.mx_dequantize)>(p[2]);
    g_lib.a8_quantize = reinterpret_cast<decltype(g_lib.a8_quantize)>(p[3]);
    g_lib.a8_dequantize = reinterpret_cast<decltype(g_lib.a8_dequantize)>(p[4]);
    g_lib.fwd = reinterpret_cast<decltype(g_lib.fwd)>(p[5]);
    g_lib.bwd_mx = reinterpret_cast<decltype(g_lib.bwd_mx)>(p[6]);
    g_lib.bwd_a8 = reinterpret_cast<decltype(g_lib.bwd_a8)>(p[7]);
    Py_RETURN_NONE;
}

// quantize(is_act8, x) -> (codes, scales) | status | None
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "quantize takes 2 arguments");
    return plain([&]() -> PyObject* {
        Args a;
        const bool act8 = v[0] == Py_True;
        const at::Tensor& x = a.any(v[1]);
        const qlora_dtype dt = source_type(x);
        if (x.dim() != 2) throw NotPlain{};
        const int64_t rows = x.size(0), cols = x.size(1);
        if (rows < 1 || cols < 64 || cols % 64) throw NotPlain{};
        at::Tensor q, s;
        qlora_status st;
        {
            Unlocked free;
            q = a.empty(act8 ? at::kChar : at::kByte, {rows, act8 ? cols : cols / 2});
            s = act8 ? a.empty(at::kByte, {rows, cols / 32})
                     : a.empty(at::kByte, {512 * ((rows + 127) / 128) * ((cols + 127) / 128)});
            st = act8 ? g_lib.a8_quantize(x.data_ptr(), dt, rows, cols, static_cast<int8_t*>(q.data_ptr()),
                                          static_cast<uint8_t*>(s.data_ptr()), a.stream())
                      : g_lib.mx_quantize(x.data_ptr(), dt, rows, cols, static_cast<uint8_t*>(q.data_ptr()),
                                          static_cast<uint8_t*>(s.data_ptr()), a.stream());
        }
        if (st != QLORA_OK) return status(st);
        return tuple(THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)));
    });
}

// dequantize(is_act8, codes, scales, rows, cols, is_bf16) -> tensor | status | None
PyObject* dequantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 6) return PyErr_Format(PyExc_TypeError, "dequantize takes 6 arguments");
    return plain([&]() -> PyObject* {
        Args a;
        const bool act8 = v[0] == Py_True, bf = v[5] == Py_True;
        const int64_t rows = integer(v[3]), cols = integer(v[4]);
        const void* q = a.get(v[1], act8 ? at::kChar : at::kByte, rows, act8 ? cols : cols / 2);
        const void* s = act8 ? a.get(v[2], at::kByte, rows, cols / 32)
                             : a.flat(v[2], at::kByte, 512 * ((rows + 127) / 128) * ((cols + 127) / 128));
        const qlora_dtype dt = bf ? QLORA_BF16 : QLORA_F32;
        at::Tensor out;
        qlora_status st;
        {
            Unlocked free;
            out = a.empty(bf ? kBf : kF32, {rows, cols});
            if (act8) {
                const qlora_act8 h = {static_cast<const int8_t*>(q), static_cast<const uint8_t*>(s)};
                st = g_lib.a8_dequantize(&h, rows, cols, out.data_ptr(), dt, a.stream());
            } else {
                const qlora_mxfp4 h = {static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(s), rows, cols};
                st = g_lib.mx_dequantize(&h, out.data_ptr(), dt, a.stream());
            }
        }
        return st == QLORA_OK ? THPVariable_Wrap(std::move(out)) : status(st);
    });
}

// forward(codes, scales, d_out, d_in, X, A, B, alpha, H, U_save, save_u, ws) -> (H, U) | status | None
PyObject* forward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 12) return PyErr_Format(PyExc_TypeError, "forward takes 12 arguments");
    return plain([&]() -> PyObject* {
        Args a;
        const int64_t d_out = integer(v[2]), d_in = integer(v[3]);
        int64_t T, r, k;
        shape2(v[4], T, k);
        shape2(v[5], r, k);
        if (T < 1 || r < 1 || r > 128) throw NotPlain{};
        const qlora_mxfp4 w = {static_cast<const uint8_t*>(a.get(v[0], at::kByte, d_out, d_in / 2)),
                               static_cast<const uint8_t*>(
                                   a.flat(v[1], at::kByte, 512 * ((d_out + 127) / 128) * ((d_in + 127) / 128))),
                               d_out, d_in};
        const void* X = a.get(v[4], kBf, T, d_in);
        const void* A = a.get(v[5], kBf, r, d_in);
        const void* B = a.get(v[6], kBf, d_out, r);
        const float alpha = real(v[7]);
        const int32_t rank = static_cast<int32_t>(r);
        Workspace ws(a, v[11], QLORA_OP_FWD_MXFP4, T, d_out, d_in, rank);
        Out H(a, v[8], kBf, T, d_out), U(a, v[9], kBf, T, r);
        const bool want_u = truth(v[10]);
        qlora_status st;
        {
            Unlocked free;
            void* h = H.ptr(a);
            void* u = U.p || want_u ? U.ptr(a) : nullptr;
            void* w8 = ws.ptr(a);
            st = g_lib.fwd(&w, X, T, A, B, rank, alpha, h, u, w8, ws.bytes, a.stream());
        }
        return st == QLORA_OK ? tuple(H.object(), U.object()) : status(st);
    });
}

// backward(codes, scales, c2, d_out, d_in, X, scales8, dH, A, B, alpha, U, dX, dA, dB, want_dx, accumulate, ws)
//   c2: None for an MXFP4 base (scales: its tiles), else the NF4 group constants (scales: absmax bytes)
//   scales8: None for a bf16 X, else the scales of the 8-bit checkpoint X
//   -> (dX, dA, dB) | status | None
PyObject* backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 18) return PyErr_Format(PyExc_TypeError, "backward takes 18 arguments");
    return plain([&]() -> PyObject* {
        Args a;
        const int64_t d_out = integer(v[3]), d_in = integer(v[4]);
        const bool nf4 = v[2] != Py_None, act8 = v[6] != Py_None, acc = truth(v[16]);
        int64_t T, r, k;
        shape2(v[7], T, k);
        shape2(v[8], r, k);
        if (T < 1 || r < 1 || r > 128 || d_in < 64 || d_in % 64 || (nf4 && !act8)) throw NotPlain{};
        if (acc && (v[13] == Py_None || v[14] == Py_None)) throw NotPlain{};
        const auto* codes = static_cast<const uint8_t*>(a.get(v[0], at::kByte, d_out, d_in / 2));
        const int64_t blocks = d_out * d_in / 64;
        const auto* scales = static_cast<const uint8_t*>(
            a.flat(v[1], at::kByte, nf4 ? blocks : 512 * ((d_out + 127) / 128) * ((d_in + 127) / 128)));
        const auto* c2 = nf4 ? static_cast<const float*>(a.flat(v[2], kF32, (blocks + 255) / 256)) : nullptr;
        const void* X = a.get(v[5], act8 ? at::kChar : kBf, T, d_in);
        const qlora_act8 x8 = {static_cast<const int8_t*>(X),
                               act8 ? static_cast<const uint8_t*>(a.get(v[6], at::kByte, T, d_in / 32)) : nullptr};
        const void* dH = a.get(v[7], kBf, T, d_out);
        const void* A = a.get(v[8], kBf, r, d_in);
        const void* B = a.get(v[9], kBf, d_out, r);
        const float alpha = real(v[10]);
        const void* U = v[11] == Py_None ? nullptr : a.get(v[11], kBf, T, r);
        const int32_t rank = static_cast<int32_t>(r);
        Workspace ws(a, v[17], nf4 ? QLORA_OP_BWD_ACT8 : QLORA_OP_BWD_MXFP4, T, d_out, d_in, rank);
        Out dX(a, v[12], kBf, T, d_in), dA(a, v[13], kF32, r, d_in), dB(a, v[14], kF32, d_out, r);
        const bool want_dx = truth(v[15]);
        const uint32_t flags = acc ? QLORA_BWD_ACCUMULATE : 0;
        qlora_status st;
        {
            Unlocked free;
            void* gx = dX.p || want_dx ? dX.ptr(a) : nullptr;
            float* ga = static_cast<float*>(dA.ptr(a));
            float* gb = static_cast<float*>(dB.ptr(a));
            void* w8 = ws.ptr(a);
            if (nf4) {
                const qlora_nf4 w = {codes, scales, c2, d_out, d_in};
                st = g_lib.bwd_a8(&w, &x8, dH, T, A, B, rank, alpha, U, gx, ga, gb, w8, ws.bytes, flags, a.stream());
            } else {
                const qlora_mxfp4 w = {codes, scales, d_out, d_in};
                st = g_lib.bwd_mx(&w, act8 ? nullptr : X, act8 ? &x8 : nullptr, dH, T, A, B, rank, alpha, U, gx, ga, gb,
                                  w8, ws.bytes, flags, a.stream());
            }
        }
        return st == QLORA_OK ? tuple(dX.object(), dA.object(), dB.object()) : status(st);
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"init", FAST(init), "addresses of the library's functions"},
                           {"quantize", FAST(quantize), "MXFP4 or 8-bit checkpoint of a matrix"},
                           {"dequantize", FAST(dequantize), "values of either"},
                           {"forward", FAST(forward), "qlora_linear_fwd_mxfp4"},
                           {"backward", FAST(backward), "qlora_linear_bwd_mxfp4, qlora_linear_bwd_act8"},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mx_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_bind() { return PyModule_Create(&g_module); }
