// Python module _tensors: the calls over torch tensors of i8.py, norm.py and f8.py's
// f8_requantize, from the tensors to the C ABI in one step.  The checks are those of f8.py's
// _matrix and its like; in Python they took 5 to 9 us a call (17 tensors), longer than the
// launch and, with few rows, than the kernels.  Nothing is kept between calls but the
// addresses of the library's functions and torch's functions for streams and devices.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdarg>
#include <cstdint>

#include "sgemm_i8.h"
#include "sgemm_norm.h"

namespace {

decltype(&sgemm_i8_gemm) i8_gemm_fn = nullptr;
decltype(&sgemm_i8_quantize) i8_quantize_fn = nullptr;
decltype(&sgemm_f8_requantize) f8_requantize_fn = nullptr;
decltype(&sgemm_block_norm) block_norm_fn = nullptr;
decltype(&sgemm_block_norm_bwd) block_norm_bwd_fn = nullptr;
PyObject *raw_stream = nullptr, *current_device = nullptr, *set_device = nullptr, *stream_name = nullptr;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const char *format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Refused{};
}
bool given(PyObject *o) { return o != Py_None; }

const at::Tensor &tensor(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, "%s: a tensor is needed", name);
    return THPVariable_Unpack(o);
}

// Element types that a place takes, and the C ABI's number of one (-1: another).
enum Table { TYPES, FORMATS, F32, I8 };
const char *const kNames[] = {"float32 / float16 / bfloat16", "float8_e4m3fn / float8_e5m2", "float32", "int8"};
int kind_of(const at::Tensor &t, Table table)
{
    const at::ScalarType s = t.scalar_type();
    switch (table) {
    case TYPES:
        return s == at::kFloat ? SGEMM_TYPE_F32 : s == at::kHalf ? SGEMM_TYPE_FP16 : s == at::kBFloat16 ? SGEMM_TYPE_BF16 : -1;
    case FORMATS:
        return s == at::ScalarType::Float8_e4m3fn ? SGEMM_F8_E4M3 : s == at::ScalarType::Float8_e5m2 ? SGEMM_F8_E5M2 : -1;
    case F32:
        return s == at::kFloat ? SGEMM_TYPE_F32 : -1;
    default:
        return s == at::kChar ? 0 : -1;
    }
}

// The device of a call: that of its first tensor, which must be a GPU.
int device_of(const char *name, PyObject *o)
{
    const at::Tensor &t = tensor(name, o);
    if (!t.is_cuda())
        refuse(PyExc_TypeError, "tensors on a GPU are needed");
    return (int)t.get_device();
}

// A 2-D device tensor with unit stride along its rows.
struct Matrix {
    int kind = 0;
    int64_t rows = 0, cols = 0, ld = 0;
    void *p = nullptr;
};
Matrix matrix_of(const char *name, const at::Tensor &t, int64_t rows, int64_t cols, int64_t ld, int64_t step, int kind)
{
    if (step != 1 && cols > 1)
        refuse(PyExc_ValueError, "%s must have unit stride along its last dimension", name);
    if (ld < cols || ld == 0) {
        if (rows > 1 && cols > 0)
            refuse(PyExc_ValueError, "%s rows overlap (row stride below the row length)", name);
        ld = cols > 0 ? cols : 1;
    } else if (rows <= 1) {
        ld = cols > 0 ? cols : 1;
    }
    return Matrix{kind, rows, cols, ld, t.data_ptr()};
}
Matrix matrix(const char *name, PyObject *o, Table table, int device)
{
    const at::Tensor &t = tensor(name, o);
    const int kind = kind_of(t, table);
    if (kind < 0 || t.dim() != 2 || !t.is_cuda() || t.get_device() != device)
        refuse(PyExc_TypeError, "%s: a 2-D %s tensor on the call's device is needed", name, kNames[table]);
    return matrix_of(name, t, t.size(0), t.size(1), t.stride(0), t.stride(1), kind);
}
// The same of a given shape; without a tensor: NULL.
Matrix shaped(const char *name, PyObject *o, Table table, int device, int64_t rows, int64_t cols, int kind = -1)
{
    if (!given(o))
        return Matrix{};
    const Matrix m = matrix(name, o, table, device);
    if (m.rows != rows || m.cols != cols)
        refuse(PyExc_ValueError, "%s has shape (%lld, %lld), not (%lld, %lld)", name, (long long)m.rows, (long long)m.cols,
               (long long)rows, (long long)cols);
    if (kind >= 0 && m.kind != kind)
        refuse(PyExc_ValueError, "%s must be of the call's type", name);
    return m;
}
// n consecutive values; without a tensor: NULL.
struct Vector {
    int kind = 0;
    void *p = nullptr;
};
Vector vector(const char *name, PyObject *o, int64_t n, Table table, int device)
{
    if (!given(o))
        return Vector{};
    const at::Tensor &t = tensor(name, o);
    const int kind = kind_of(t, table);
    if (kind < 0 || t.dim() != 1 || !t.is_cuda() || t.get_device() != device)
        refuse(PyExc_TypeError, "%s: a 1-D %s tensor on the call's device is needed", name, kNames[table]);
    if (t.size(0) != n || (n > 1 && t.stride(0) != 1))
        refuse(PyExc_ValueError, "%s must hold %lld consecutive values", name, (long long)n);
    return Vector{kind, t.data_ptr()};
}
float *floats(const char *name, PyObject *o, int64_t n, int device)
{
    return static_cast<float *>(vector(name, o, n, F32, device).p);
}
struct Lent {
    void *p = nullptr;
    int64_t bytes = 0;
};
Lent workspace(PyObject *o, int device)
{
    if (!given(o))
        return Lent{};
    const at::Tensor &t = tensor("workspace", o);
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
        refuse(PyExc_ValueError, "workspace must be a contiguous tensor on the call's device");
    return Lent{t.data_ptr(), (int64_t)t.nbytes()};
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Refused{};
    return v;
}
int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused{};
    return v;
}

// Calls f(stream) with the device current and without the interpreter's lock; the status as
// a Python integer.
template <class F> PyObject *launch(int device, PyObject *stream, F f)
{
    PyObject *o = nullptr;
    if (given(stream)) {
        o = PyObject_GetAttr(stream, stream_name);
    } else {
        PyObject *index = PyLong_FromLong(device);
        o = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
        Py_XDECREF(index);
    }
    if (!o)
        throw Refused{};
    void *s = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    if (!s && PyErr_Occurred())
        throw Refused{};
    o = PyObject_CallNoArgs(current_device);
    if (!o)
        throw Refused{};
    const long before = PyLong_AsLong(o);
    Py_DECREF(o);
    auto make_current = [](long d) {
        PyObject *r = PyObject_CallFunction(set_device, "l", d);
        if (!r)
            throw Refused{};
        Py_DECREF(r);
    };
    if (before != device)
        make_current(device);
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f(s);
    Py_END_ALLOW_THREADS
    if (before != device)
        make_current(before);
    return PyLong_FromLong(status);
}

template <class F> PyObject *guarded(Py_ssize_t n, Py_ssize_t wanted, F f)
{
    if (n != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are needed", wanted);
        return nullptr;
    }
    if (!raw_stream) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *i8_gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        const int d = device_of("C", a[4]);
        const Matrix A = matrix("A", a[0], I8, d), B = matrix("B", a[2], I8, d), C = matrix("C", a[4], TYPES, d);
        if (B.cols != A.cols || C.rows != A.rows || C.cols != B.rows)
            refuse(PyExc_ValueError, "shape mismatch: A (%lld, %lld), B (%lld, %lld), C (%lld, %lld)", (long long)A.rows,
                   (long long)A.cols, (long long)B.rows, (long long)B.cols, (long long)C.rows, (long long)C.cols);
        if (!given(a[1]) || !given(a[3]))
            refuse(PyExc_TypeError, "SA and SB are needed");
        const float *SA = floats("SA", a[1], A.rows, d), *SB = floats("SB", a[3], B.rows, d);
        const float alpha = (float)number(a[5]), beta = (float)number(a[6]);
        const Lent w = workspace(a[7], d);
        return launch(d, a[8], [&](void *s) {
            return i8_gemm_fn(C.kind, A.rows, B.rows, A.cols, alpha, static_cast<const int8_t *>(A.p), A.ld, SA,
                              static_cast<const int8_t *>(B.p), B.ld, SB, beta, C.p, C.ld, w.p, w.bytes, s);
        });
    });
}

PyObject *i8_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        const int d = device_of("X", a[0]);
        const Matrix X = matrix("X", a[0], TYPES, d);
        if (!given(a[1]) || !given(a[2]))
            refuse(PyExc_TypeError, "Q and S are needed");
        const Matrix Q = shaped("Q", a[1], I8, d, X.rows, X.cols);
        float *S = floats("S", a[2], X.rows, d);
        return launch(d, a[3], [&](void *s) {
            return i8_quantize_fn(X.kind, X.rows, X.cols, X.p, X.ld, static_cast<int8_t *>(Q.p), Q.ld, S, s);
        });
    });
}

PyObject *f8_requantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 5, [&] {
        const int d = device_of("X", a[0]);
        const Matrix X = matrix("X", a[0], FORMATS, d);
        if (!given(a[1]) || !given(a[2]) || !given(a[3]))
            refuse(PyExc_TypeError, "SX, QT and ST are needed");
        const Matrix QT = shaped("QT", a[2], FORMATS, d, X.cols, X.rows);
        const Matrix SX = shaped("SX", a[1], F32, d, blocks(X.cols), X.rows);
        const Matrix ST = shaped("ST", a[3], F32, d, blocks(X.rows), X.cols);
        return launch(d, a[4], [&](void *s) {
            return f8_requantize_fn(X.kind, QT.kind, X.rows, X.cols, X.p, X.ld, static_cast<const float *>(SX.p), SX.ld, QT.p,
                                    QT.ld, static_cast<float *>(ST.p), ST.ld, s);
        });
    });
}

// The type that the weights of a call share: the rows' or FP32.
struct WeightType {
    int kind, rows_kind;
    bool any = false;
    void take(const char *name, int k)
    {
        if ((k != rows_kind && k != SGEMM_TYPE_F32) || (any && k != kind))
            refuse(PyExc_TypeError, "%s must be of the rows' type or float32, as the other weights", name);
        kind = k;
        any = true;
    }
    void *vector_of(const char *name, PyObject *o, int64_t cols, int device)
    {
        if (!given(o))
            return nullptr;
        const Vector v = vector(name, o, cols, TYPES, device);
        take(name, v.kind);
        return v.p;
    }
};

// A row of cols values, or one for every gate_rows rows.
Matrix gate_matrix(const char *name, PyObject *o, Table table, int device)
{
    const at::Tensor &t = tensor(name, o);
    if (t.dim() != 1)
        return matrix(name, o, table, device);
    const int kind = kind_of(t, table);
    if (kind < 0 || !t.is_cuda() || t.get_device() != device)
        refuse(PyExc_TypeError, "%s: a %s tensor on the call's device is needed", name, kNames[table]);
    return matrix_of(name, t, 1, t.size(0), t.size(0), t.stride(0), kind);
}
struct Gate {
    Matrix m;
    int64_t rows = 0;       // of x for one of the gate's
};
Gate gate_of(PyObject *o, PyObject *gate_rows, int64_t rows, int64_t cols, int device, WeightType &w)
{
    Gate g;
    if (!given(o))
        return g;
    g.m = gate_matrix("gate", o, TYPES, device);
    w.take("gate", g.m.kind);
    if (given(gate_rows)) {
        g.rows = integer(gate_rows);
    } else if (rows > 0) {
        if (g.m.rows == 0 || rows % g.m.rows != 0)
            refuse(PyExc_ValueError, "%lld rows do not divide among %lld rows of gate: gate_rows is needed", (long long)rows,
                   (long long)g.m.rows);
        g.rows = rows / g.m.rows;
    }
    if (g.rows < (rows > 0 ? 1 : 0))
        refuse(PyExc_ValueError, "gate_rows must be positive");
    const int64_t gates = rows > 0 ? rows / g.rows + (rows % g.rows != 0) : g.m.rows;
    if (g.m.cols != cols || g.m.rows != gates)
        refuse(PyExc_ValueError, "gate has shape (%lld, %lld), not (%lld, %lld)", (long long)g.m.rows, (long long)g.m.cols,
               (long long)gates, (long long)cols);
    return g;
}

// An e4m3 matrix with row blocks, and its scales.
struct Kept {
    Matrix q, s;
    float *scales() const { return static_cast<float *>(s.p); }
};
Kept kept_of(const char *name, PyObject *o, const char *s_name, PyObject *s, int64_t rows, int64_t cols, int device)
{
    Kept k;
    if (!given(o))
        return k;
    k.q = shaped(name, o, FORMATS, device, rows, cols, SGEMM_F8_E4M3);
    if (!given(s))
        refuse(PyExc_ValueError, "%s needs %s", name, s_name);
    k.s = shaped(s_name, s, F32, device, blocks(cols), rows);
    return k;
}

// X, O, W, eps, w_post, gate, gate_rows, alpha, H, Y, Q, S, H8, SH, O8, SO, rstd, rstd_post, stream
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 19, [&] {
        const int d = device_of("X", a[0]);
        const Matrix X = matrix("X", a[0], TYPES, d);
        const int64_t rows = X.rows, cols = X.cols;
        const Matrix O = shaped("O", a[1], TYPES, d, rows, cols, X.kind);
        WeightType wt{X.kind, X.kind};
        const void *W = wt.vector_of("W", a[2], cols, d), *WP = wt.vector_of("w_post", a[4], cols, d);
        const float eps = (float)number(a[3]), alpha = (float)number(a[7]);
        const Gate G = gate_of(a[5], a[6], rows, cols, d, wt);
        if (!given(a[1]) && (given(a[4]) || given(a[5]) || given(a[14]) || given(a[17])))
            refuse(PyExc_ValueError, "w_post, gate, O8 and rstd_post belong to O");
        if (given(a[17]) && !given(a[4]))
            refuse(PyExc_ValueError, "rstd_post belongs to w_post");
        if (!given(a[2]) && (given(a[9]) || given(a[10])))
            refuse(PyExc_ValueError, "Y and Q need W");
        const Matrix H = shaped("H", a[8], TYPES, d, rows, cols, X.kind), Y = shaped("Y", a[9], TYPES, d, rows, cols, X.kind);
        Kept Q;
        int format = SGEMM_F8_E4M3;
        if (given(a[10])) {
            if (!given(a[11]))
                refuse(PyExc_ValueError, "Q needs S");
            if (kind_of(tensor("Q", a[10]), I8) == 0) {
                format = SGEMM_Q_I8;
                Q.q = shaped("Q", a[10], I8, d, rows, cols);
                Q.s.p = floats("S", a[11], rows, d);
            } else {
                Q = kept_of("Q", a[10], "S", a[11], rows, cols, d);
            }
        }
        const Kept H8 = kept_of("H8", a[12], "SH", a[13], rows, cols, d), O8 = kept_of("O8", a[14], "SO", a[15], rows, cols, d);
        float *rstd = floats("rstd", a[16], rows, d), *rstd_post = floats("rstd_post", a[17], rows, d);
        return launch(d, a[18], [&](void *s) {
            return block_norm_fn(X.kind, wt.kind, rows, cols, X.p, X.ld, O.p, O.ld, W, WP, G.m.p, G.m.ld, G.rows, alpha, eps,
                                 H.p, H.ld, Y.p, Y.ld, format, Q.q.p, Q.q.ld, Q.scales(), Q.s.ld, H8.q.p, H8.q.ld, H8.scales(),
                                 H8.s.ld, O8.q.p, O8.q.ld, O8.scales(), O8.s.ld, rstd, rstd_post, s);
        });
    });
}

// dY, H, O, W, rstd, dX, dO, SH, SO, w_post, rstd_post, gate, gate_rows, alpha, dH, dW, dW_post, dGate, workspace, stream
PyObject *block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 20, [&] {
        const bool has_dy = given(a[0]);
        if (!has_dy && !given(a[14]))
            refuse(PyExc_ValueError, "one of dY and dH is needed");
        const char *name = has_dy ? "dY" : "dH";
        const int d = device_of(name, has_dy ? a[0] : a[14]);
        const Matrix first = matrix(name, has_dy ? a[0] : a[14], TYPES, d);
        const int64_t rows = first.rows, cols = first.cols;
        const int kind = first.kind;
        const Matrix DY = has_dy ? first : Matrix{}, DH = shaped("dH", a[14], TYPES, d, rows, cols, kind);
        if (!given(a[2]) && (given(a[17]) || given(a[9])))
            refuse(PyExc_ValueError, "w_post and dGate need O");
        if (has_dy && (!given(a[1]) || !given(a[3]) || !given(a[4])))
            refuse(PyExc_ValueError, "dY needs H, W and rstd");
        if (given(a[17]) && !given(a[11]))
            refuse(PyExc_ValueError, "dGate needs gate");
        if (given(a[16]) && !given(a[9]))
            refuse(PyExc_ValueError, "dW_post needs w_post");
        if (given(a[9]) && !given(a[10]))
            refuse(PyExc_ValueError, "w_post needs rstd_post");
        PyObject *const h = has_dy ? a[1] : Py_None, *const o = a[2];
        const bool h8 = given(h) && kind_of(tensor("H", h), FORMATS) >= 0, o8 = given(o) && kind_of(tensor("O", o), FORMATS) >= 0;
        if (given(h) && given(o) && h8 != o8)
            refuse(PyExc_TypeError, "H and O must both be of dY's type or both float8_e4m3fn");
        Kept H, O;
        if (h8 || o8) {
            H = kept_of("H", h, "SH", a[7], rows, cols, d);
            O = kept_of("O", o, "SO", a[8], rows, cols, d);
        } else {
            H.q = shaped("H", h, TYPES, d, rows, cols, kind);
            O.q = shaped("O", o, TYPES, d, rows, cols, kind);
        }
        WeightType wt{kind, kind};
        const void *W = has_dy ? wt.vector_of("W", a[3], cols, d) : nullptr, *WP = wt.vector_of("w_post", a[9], cols, d);
        const Gate G = gate_of(a[11], a[12], rows, cols, d, wt);
        const float alpha = (float)number(a[13]);
        const Matrix DX = shaped("dX", a[5], TYPES, d, rows, cols, kind), DO = shaped("dO", a[6], TYPES, d, rows, cols, kind);
        const float *rstd = has_dy ? floats("rstd", a[4], rows, d) : nullptr;
        const float *rstd_post = given(a[9]) ? floats("rstd_post", a[10], rows, d) : nullptr;
        float *DW = floats("dW", a[15], cols, d), *DWP = floats("dW_post", a[16], cols, d);
        Matrix DG;
        if (given(a[17])) {
            if (tensor("dGate", a[17]).sizes() != tensor("gate", a[11]).sizes())
                refuse(PyExc_ValueError, "dGate must have the gate's shape");
            DG = gate_matrix("dGate", a[17], F32, d);
        }
        const Lent w = workspace(a[18], d);
        return launch(d, a[19], [&](void *s) {
            const int status = block_norm_bwd_fn(
                kind, wt.kind, rows, cols, DY.p, DY.ld, DH.p, DH.ld, h8 || o8, H.q.p, H.q.ld, H.scales(), H.s.ld, O.q.p,
                O.q.ld, O.scales(), O.s.ld, W, WP, rstd, rstd_post, G.m.p, G.m.ld, G.rows, alpha, DX.p, DX.ld, DO.p, DO.ld, DW,
                DWP, static_cast<float *>(DG.p), DG.ld, w.p, w.bytes, s);
            // gates without rows: the C function knows of none, their sums are 0
            if (status == SGEMM_OK && rows == 0 && cols > 0 && DG.rows > 0)
                return i8_gemm_fn(SGEMM_TYPE_F32, DG.rows, cols, 0, 0.0f, nullptr, 1, nullptr, nullptr, 1, nullptr, 0.0f, DG.p,
                                  DG.ld, nullptr, 0, s);
            return status;
        });
    });
}

// bind((addresses of the five C functions), raw_stream, current_device, set_device)
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long f[5];
    PyObject *rs, *cd, *sd;
    if (!PyArg_ParseTuple(args, "(KKKKK)OOO", &f[0], &f[1], &f[2], &f[3], &f[4], &rs, &cd, &sd))
        return nullptr;
    i8_gemm_fn = reinterpret_cast<decltype(i8_gemm_fn)>(f[0]);
    i8_quantize_fn = reinterpret_cast<decltype(i8_quantize_fn)>(f[1]);
    f8_requantize_fn = reinterpret_cast<decltype(f8_requantize_fn)>(f[2]);
    block_norm_fn = reinterpret_cast<decltype(block_norm_fn)>(f[3]);
    block_norm_bwd_fn = reinterpret_cast<decltype(block_norm_bwd_fn)>(f[4]);
    Py_INCREF(rs);
    Py_INCREF(cd);
    Py_INCREF(sd);
    Py_XDECREF(current_device);
    Py_XDECREF(set_device);
    Py_XDECREF(raw_stream);
    current_device = cd;
    set_device = sd;
    raw_stream = rs;
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr}, FAST(i8_gemm), FAST(i8_quantize), FAST(f8_requantize),
                         FAST(block_norm), FAST(block_norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors()
{
    if (!stream_name && !(stream_name = PyUnicode_InternFromString("cuda_stream")))
        return nullptr;
    PyObject *m = PyModule_Create(&module);
    // native.py compares it with what runs: the tensors' layout is that of this torch
#define TEXT(x) #x
#define VERSION(major, minor) TEXT(major) "." TEXT(minor) " " TORCH_VERSION
    if (m && PyModule_AddStringConstant(m, "built_for", VERSION(PY_MAJOR_VERSION, PY_MINOR_VERSION)) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
