// ops_binding.cpp -- the Python binding of include/elq_ops.h, as a CPython module
// over torch tensors.
//
// It does what a binding does and no more: it checks what the C entries cannot see
// (that an argument is a tensor, its device, dtype, shape and strides), allocates
// outputs on the current stream of the tensors' device, and makes one C call.
// It is compiled because the host's time bounds the small calls: a call through
// ctypes took 7.5 to 12.5 us, of which the launch is 2.5.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/elq_ops.h"

namespace {

PyObject* g_error = nullptr;            // elq.ElqError
PyObject* g_memory = nullptr;           // torch.OutOfMemoryError
PyTypeObject* g_rows = nullptr;         // ops.I8Rows
PyObject *s_q, *s_scale, *s_buf, *s_cols;

struct Refused {};                      // a Python exception is set

[[noreturn]] void refuse(int status, const char* what) {
    PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}
void check(bool ok, const char* what, int status = ELQ_ERR_INVALID_ARG) {
    if (!ok) refuse(status, what);
}

int type_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return ELQ_F32;
        case at::kBFloat16: return ELQ_BF16;
        case at::kHalf: return ELQ_F16;
        case at::kChar: return ELQ_I8;
        default: return -1;
    }
}
enum { FLOATS = 1, HALVES = 2, CODES = 4, F32_ONLY = 8 };
bool among(int type, int kinds) {
    if (type == ELQ_F32) return kinds & (FLOATS | F32_ONLY);
    if (type == ELQ_BF16 || type == ELQ_F16) return kinds & (FLOATS | HALVES);
    return type == ELQ_I8 && (kinds & CODES);
}
at::ScalarType scalar_of(int type) {
    return type == ELQ_F32 ? at::kFloat : type == ELQ_BF16 ? at::kBFloat16 : type == ELQ_F16 ? at::kHalf : at::kChar;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    check(THPVariable_Check(o), what);
    return THPVariable_Unpack(o);
}

struct Mat {
    void* p = nullptr;
    int type = 0, dev = 0;
    int64_t rows = 0, cols = 0, ld = 0;
};

int64_t padded(int64_t cols) { return (cols + 15) / 16 * 16; }

// A 2-D tensor of contiguous rows, of one of `kinds`, on device `dev` (any: -1).
Mat matrix(const at::Tensor& t, const char* what, int kinds, int dev) {
    check(t.dim() == 2, what);
    Mat m;
    m.type = type_of(t.scalar_type());
    check(among(m.type, kinds), what, ELQ_ERR_UNSUPPORTED);
    check(t.is_cuda() && (dev < 0 || t.get_device() == dev), what);
    m.dev = (int)t.get_device();
    m.rows = t.size(0);
    m.cols = t.size(1);
    check(m.cols >= 1 && (m.cols == 1 || t.stride(1) == 1), what);
    m.ld = m.rows > 1 ? t.stride(0) : padded(m.cols);
    m.p = t.data_ptr();
    return m;
}

// A contiguous vector of n values, or null for None.
template <typename T>
const T* vector(PyObject* o, int64_t n, const char* what, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, what);
    check(t.scalar_type() == (sizeof(T) == 4 && std::is_same<T, float>::value ? at::kFloat : at::kInt) && t.is_cuda() &&
              t.get_device() == dev && t.numel() == n && t.is_contiguous(),
          what);
    return reinterpret_cast<const T*>(t.data_ptr());
}

struct Owned {                          // one reference
    PyObject* o;
    explicit Owned(PyObject* p) : o(p) {}
    ~Owned() { Py_XDECREF(o); }
    Owned(const Owned&) = delete;
    Owned& operator=(const Owned&) = delete;
};

PyObject* attr(PyObject* o, PyObject* name) {
    PyObject* v = PyObject_GetAttr(o, name);
    if (!v) throw Refused();
    return v;
}
int64_t number(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}

struct Rows {
    Mat m;
    const float* scale = nullptr;
};

// 2-D I8Rows: a buffer of this module's (codes, then scales), or any q and scale.
Rows rows_of(PyObject* o, const char* what, int dev) {
    check(PyObject_TypeCheck(o, g_rows), what);
    Rows r;
    Owned buf(attr(o, s_buf));
    if (buf.o != Py_None) {
        const at::Tensor& b = tensor(buf.o, what);
        r.m.type = ELQ_I8;
        r.m.dev = (int)b.get_device();
        check(dev < 0 || r.m.dev == dev, what);
        Owned c(attr(o, s_cols));
        r.m.cols = number(c.o);
        check(r.m.cols >= 1, what);
        r.m.ld = padded(r.m.cols);
        r.m.rows = b.numel() / (r.m.ld + 4);
        r.m.p = b.data_ptr();
        r.scale = reinterpret_cast<const float*>(static_cast<char*>(r.m.p) + r.m.rows * r.m.ld);
        return r;
    }
    Owned q(attr(o, s_q)), s(attr(o, s_scale));
    r.m = matrix(tensor(q.o, what), what, CODES, dev);
    check(s.o != Py_None, what);
    r.scale = vector<float>(s.o, r.m.rows, what, r.m.dev);
    return r;
}

struct Stack {
    const void* p;
    int64_t ld, stride, E, N, K;
};
// A stack [E][N][K] of contiguous rows of type `type`.
Stack stack(PyObject* o, const char* what, int type, int dev) {
    const at::Tensor& t = tensor(o, what);
    check(t.dim() == 3, what);
    check(type_of(t.scalar_type()) == type, what, ELQ_ERR_UNSUPPORTED);
    check(t.is_cuda() && t.get_device() == dev, what);
    Stack s;
    s.E = t.size(0);
    s.N = t.size(1);
    s.K = t.size(2);
    check(s.E >= 1 && s.N >= 1 && s.K >= 1 && (s.K == 1 || t.stride(2) == 1), what);
    check(s.E <= INT32_MAX && s.N <= INT32_MAX && s.K <= INT32_MAX, what, ELQ_ERR_UNSUPPORTED);
    s.ld = s.N > 1 ? t.stride(1) : padded(s.K);
    s.stride = t.stride(0);
    s.p = t.data_ptr();
    return s;
}

int width(int64_t n, const char* what) {
    check(n <= INT32_MAX, what, ELQ_ERR_UNSUPPORTED);
    return (int)n;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType t, int dev) {
    return at::empty(size, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)dev));
}

// The caller's out (rows x cols of `type`), or a new one.
at::Tensor output(PyObject* out, int64_t rows, int64_t cols, int type, int dev, const char* what, Mat& m) {
    if (out == Py_None) {
        at::Tensor t = empty({rows, cols}, scalar_of(type), dev);
        m.p = t.data_ptr();
        m.ld = cols;
        m.type = type;
        return t;
    }
    const at::Tensor& t = tensor(out, what);
    m = matrix(t, what, FLOATS, dev);
    check(m.type == type && m.rows == rows && m.cols == cols, what);
    // what autograd has saved of it is no longer what it was
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return t;
}

int dtype_arg(PyObject* o, const char* what) {
    check(THPDtype_Check(o), what, ELQ_ERR_UNSUPPORTED);
    const int t = type_of(reinterpret_cast<THPDtype*>(o)->scalar_type);
    check(t >= 0, what, ELQ_ERR_UNSUPPORTED);
    return t;
}

// The device of a call made current, and its current stream.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;
    explicit On(int dev) {
        guard.set_index((c10::DeviceIndex)dev);
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
};

// New codes: a buffer of rows padded to 16 bytes, then the scales (so that its size
// and the columns say the rest).
struct NewRows {
    at::Tensor buf;
    int64_t rows, cols, ld;
    int8_t* q;
    float* scale;
    NewRows(int64_t r, int64_t c, int dev) : rows(r), cols(c), ld(padded(c)) {
        buf = empty({r * (ld + 4)}, at::kChar, dev);
        q = reinterpret_cast<int8_t*>(buf.data_ptr());
        scale = reinterpret_cast<float*>(q + r * ld);
    }
    PyObject* object() {
        PyObject* o = g_rows->tp_alloc(g_rows, 0);
        if (!o) throw Refused();
        Owned b(THPVariable_Wrap(std::move(buf))), c(PyLong_FromLongLong(cols));
        if (!b.o || !c.o || PyObject_SetAttr(o, s_q, Py_None) || PyObject_SetAttr(o, s_scale, Py_None) ||
            PyObject_SetAttr(o, s_buf, b.o) || PyObject_SetAttr(o, s_cols, c.o)) {
            Py_DECREF(o);
            throw Refused();
        }
        return o;
    }
};

void done(elq_status st, const char* what) { check(st == ELQ_OK, what, st); }

// Runs a call's body; C++ exceptions become Python's.
template <typename Body>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, Body body) {
    if (!g_rows || got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", got, want);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused&) {
        return nullptr;
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_memory, e.what_without_backtrace());
        return nullptr;
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

using Args = PyObject* const*;

// (I8Rows, ElqError, torch.OutOfMemoryError), before any other call
PyObject* bind(PyObject*, Args a, Py_ssize_t n) {
    if (n != 3 || !PyType_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "bind: three classes");
        return nullptr;
    }
    for (int i = 0; i < 3; ++i) Py_INCREF(a[i]);
    g_rows = reinterpret_cast<PyTypeObject*>(a[0]);
    g_error = a[1];
    g_memory = a[2];
    Py_RETURN_NONE;
}

// (x, index or None, div)
PyObject* quantize_i8(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        const Mat x = matrix(tensor(a[0], "quantize_i8: x: a tensor"), "quantize_i8: x", FLOATS, -1);
        int64_t rows = x.rows;
        const int32_t* index = nullptr;
        if (a[1] != Py_None) {
            rows = tensor(a[1], "quantize_i8: index").numel();
            index = vector<int32_t>(a[1], rows, "quantize_i8: index", x.dev);
        }
        const int64_t div = number(a[2]);
        check(div >= 1 && div <= INT32_MAX, "quantize_i8: index_div");
        const On on(x.dev);
        NewRows r(rows, x.cols, x.dev);
        done(elq_quantize_i8(x.p, x.type, x.rows, width(x.cols, "quantize_i8: x"), x.ld, index, (int32_t)div, rows, r.q,
                             r.ld, r.scale, on.stream),
             "elq_quantize_i8");
        return r.object();
    });
}

// (gu)
PyObject* swiglu_i8(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 1, [&] {
        const Mat x = matrix(tensor(a[0], "swiglu_i8: gu: a tensor"), "swiglu_i8: gu", FLOATS, -1);
        check(x.cols % 2 == 0, "swiglu_i8: an even number of columns");
        const On on(x.dev);
        NewRows r(x.rows, x.cols / 2, x.dev);
        done(elq_swiglu_i8(x.p, x.type, x.rows, width(x.cols / 2, "swiglu_i8: gu"), x.ld, r.q, r.ld, r.scale, on.stream),
             "elq_swiglu_i8");
        return r.object();
    });
}

// (o, pos, weights)
PyObject* combine_i8(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        const Mat o = matrix(tensor(a[0], "combine_i8: o: a tensor"), "combine_i8: o", FLOATS, -1);
        const at::Tensor& w = tensor(a[2], "combine_i8: weights [T, k]");
        check(w.dim() == 2 && a[1] != Py_None, "combine_i8: weights [T, k], pos");
        const int64_t T = w.size(0), k = w.size(1);
        const float* wp = vector<float>(a[2], T * k, "combine_i8: weights", o.dev);
        const int32_t* pos = vector<int32_t>(a[1], T * k, "combine_i8: pos", o.dev);
        const On on(o.dev);
        NewRows r(T, o.cols, o.dev);
        done(elq_combine_i8(o.p, o.type, o.rows, width(o.cols, "combine_i8: o"), o.ld, pos, wp, T,
                            width(k, "combine_i8: k"), r.q, r.ld, r.scale, on.stream),
             "elq_combine_i8");
        return r.object();
    });
}

// (x, w, bias or None, out_dtype, out or None)
PyObject* i8_matmul(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const Rows x = rows_of(a[0], "i8_matmul: x: 2-D I8Rows", -1);
        const Rows w = rows_of(a[1], "i8_matmul: w: 2-D I8Rows on x's device", x.m.dev);
        check(x.m.cols == w.m.cols, "i8_matmul: K of x and w");
        const int N = width(w.m.rows, "i8_matmul: N"), K = width(x.m.cols, "i8_matmul: K");
        const int yt = dtype_arg(a[3], "i8_matmul: out_dtype");
        check(yt != ELQ_I8, "i8_matmul: out_dtype", ELQ_ERR_UNSUPPORTED);
        const float* bias = vector<float>(a[2], N, "i8_matmul: bias", x.m.dev);
        const On on(x.m.dev);
        Mat y;
        at::Tensor out = output(a[4], x.m.rows, N, yt, x.m.dev, "i8_matmul: out", y);
        done(elq_i8_matmul((const int8_t*)x.m.p, x.m.ld, x.scale, x.m.rows, (const int8_t*)w.m.p, w.m.ld, w.scale, bias, N,
                           K, y.p, yt, y.ld, on.stream),
             "elq_i8_matmul");
        return THPVariable_Wrap(std::move(out));
    });
}

// (x, w, offsets, out_dtype or None, out or None): x and w I8Rows (w with q [E, N, K]), or 16-bit tensors
PyObject* grouped_matmul(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const bool codes = PyObject_TypeCheck(a[0], g_rows);
        Mat x;
        const float *sx = nullptr, *sw = nullptr;
        Stack w;
        if (codes) {
            const Rows r = rows_of(a[0], "grouped_matmul: x: 2-D I8Rows", -1);
            x = r.m;
            sx = r.scale;
            check(PyObject_TypeCheck(a[1], g_rows), "grouped_matmul: w: I8Rows");
            Owned q(attr(a[1], s_q)), s(attr(a[1], s_scale));
            check(q.o != Py_None && s.o != Py_None, "grouped_matmul: w: I8Rows with q [E, N, K]");
            w = stack(q.o, "grouped_matmul: w: [E, N, K]", ELQ_I8, x.dev);
            sw = vector<float>(s.o, w.E * w.N, "grouped_matmul: w.scale", x.dev);
        } else {
            x = matrix(tensor(a[0], "grouped_matmul: x"), "grouped_matmul: x", HALVES, -1);
            w = stack(a[1], "grouped_matmul: w: [E, N, K]", x.type, x.dev);
        }
        check(x.cols == w.K, "grouped_matmul: K of x and w");
        check(a[2] != Py_None, "grouped_matmul: offsets");
        const int32_t* offsets = vector<int32_t>(a[2], w.E + 1, "grouped_matmul: offsets", x.dev);
        int yt = codes ? ELQ_F32 : x.type;
        if (a[3] != Py_None) yt = dtype_arg(a[3], "grouped_matmul: out_dtype");
        else if (a[4] != Py_None) yt = type_of(tensor(a[4], "grouped_matmul: out").scalar_type());
        check(among(yt, FLOATS), "grouped_matmul: out_dtype", ELQ_ERR_UNSUPPORTED);
        const On on(x.dev);
        Mat y;
        at::Tensor out = output(a[4], x.rows, w.N, yt, x.dev, "grouped_matmul: out", y);
        done(elq_grouped_matmul(x.p, x.type, x.ld, sx, x.rows, w.p, w.ld, w.stride, sw, (int32_t)w.E, (int32_t)w.N,
                                (int32_t)w.K, offsets, y.p, yt, y.ld, on.stream),
             "elq_grouped_matmul");
        return THPVariable_Wrap(std::move(out));
    });
}

// (x, weight or None, eps, out_dtype or None, out or None, codes)
PyObject* rms_norm(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const Mat x = matrix(tensor(a[0], "rms_norm: x: a tensor"), "rms_norm: x", FLOATS, -1);
        const int cols = width(x.cols, "rms_norm: x");
        const float* w = vector<float>(a[1], cols, "rms_norm: weight", x.dev);
        const float eps = (float)real(a[2]);
        if (a[5] == Py_True) {
            const On on(x.dev);
            NewRows r(x.rows, cols, x.dev);
            done(elq_rms_norm(x.p, x.type, x.rows, cols, x.ld, w, eps, r.q, ELQ_I8, r.ld, r.scale, on.stream),
                 "elq_rms_norm");
            return r.object();
        }
        int nt = x.type;
        if (a[3] != Py_None) nt = dtype_arg(a[3], "rms_norm: out_dtype");
        else if (a[4] != Py_None) nt = type_of(tensor(a[4], "rms_norm: out").scalar_type());
        check(among(nt, FLOATS), "rms_norm: out_dtype", ELQ_ERR_UNSUPPORTED);
        const On on(x.dev);
        Mat y;
        at::Tensor out = output(a[4], x.rows, cols, nt, x.dev, "rms_norm: out", y);
        done(elq_rms_norm(x.p, x.type, x.rows, cols, x.ld, w, eps, y.p, nt, y.ld, nullptr, on.stream), "elq_rms_norm");
        return THPVariable_Wrap(std::move(out));
    });
}

// (h, y, post_weight, gate, gate_rows or None, res_scale, next_weight, next_dtype or None, eps, out or None) -> (h', n)
PyObject* residual_norm(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const Mat h = matrix(tensor(a[0], "residual_norm: h: a tensor"), "residual_norm: h", FLOATS, -1);
        const Mat y = matrix(tensor(a[1], "residual_norm: y: a tensor"), "residual_norm: y", FLOATS, h.dev);
        check(h.rows == y.rows && h.cols == y.cols, "residual_norm: shapes of h and y");
        elq_residual r = {};
        r.T = h.rows;
        r.cols = width(h.cols, "residual_norm: h");
        r.h_type = h.type;
        r.y_type = y.type;
        r.h = h.p;
        r.y = y.p;
        r.ldh = h.ld;
        r.ldy = y.ld;
        r.post_weight = vector<float>(a[2], h.cols, "residual_norm: post_weight", h.dev);
        r.gate_rows = r.gate_cols = 1;
        r.gate_ld = 1;
        if (a[3] != Py_None) {
            const at::Tensor& g = tensor(a[3], "residual_norm: gate");
            int64_t G = 1, cols = 0;
            if (g.dim() == 1) {
                cols = r.gate_ld = g.numel();
                r.gate = vector<float>(a[3], cols, "residual_norm: gate", h.dev);
            } else {
                const Mat m = matrix(g, "residual_norm: gate", F32_ONLY, h.dev);
                G = m.rows;
                cols = m.cols;
                r.gate = (const float*)m.p;
                r.gate_ld = m.ld;
            }
            check(cols == h.cols || cols == 1, "residual_norm: gate columns");
            r.gate_cols = (int32_t)cols;
            if (a[4] == Py_None) {
                check(G == 1 || G == h.rows, "residual_norm: gate rows");
                r.gate_rows = G == 1 ? std::max<int64_t>(h.rows, 1) : 1;
            } else {
                r.gate_rows = number(a[4]);
            }
            check(r.gate_rows >= 1 && G >= (h.rows + r.gate_rows - 1) / r.gate_rows, "residual_norm: gate rows");
        }
        r.res_scale = (float)real(a[5]);
        r.eps = (float)real(a[8]);
        const On on(h.dev);
        Mat o;
        at::Tensor out = output(a[9], h.rows, h.cols, h.type, h.dev, "residual_norm: out", o);
        r.h_out = o.p;
        r.ld_out = o.ld;
        PyObject* next = nullptr;
        if (a[7] == Py_None) {
            done(elq_residual_norm(&r, on.stream), "elq_residual_norm");
            Py_INCREF(Py_None);
            next = Py_None;
        } else {
            r.next_weight = vector<float>(a[6], h.cols, "residual_norm: next_weight", h.dev);
            r.n_type = dtype_arg(a[7], "residual_norm: next_dtype");
            if (r.n_type == ELQ_I8) {
                NewRows c(h.rows, h.cols, h.dev);
                r.n = c.q;
                r.scale = c.scale;
                r.ldn = c.ld;
                done(elq_residual_norm(&r, on.stream), "elq_residual_norm");
                next = c.object();
            } else {
                Mat m;
                at::Tensor t = output(Py_None, h.rows, h.cols, r.n_type, h.dev, "", m);
                r.n = m.p;
                r.ldn = m.ld;
                done(elq_residual_norm(&r, on.stream), "elq_residual_norm");
                next = THPVariable_Wrap(std::move(t));
            }
        }
        Owned first(THPVariable_Wrap(std::move(out))), second(next);
        if (!first.o || !second.o) throw Refused();
        return PyTuple_Pack(2, first.o, second.o);
    });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(bind),      CALL(quantize_i8),    CALL(swiglu_i8), CALL(combine_i8),
                           CALL(i8_matmul), CALL(grouped_matmul), CALL(rms_norm),  CALL(residual_norm),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) {
    s_q = PyUnicode_InternFromString("_q");
    s_scale = PyUnicode_InternFromString("_scale");
    s_buf = PyUnicode_InternFromString("_buf");
    s_cols = PyUnicode_InternFromString("_cols");
    return PyModule_Create(&g_module);
}
