// binding.cpp -- CPython functions behind the 4-bit operators of the package's
// tensor layer: they check torch tensors, allocate results, and call the C ABI of
// include/ptc.h.  A decoding step's operators take a few microseconds on the
// device; the same marshalling through ctypes took 9 to 14 us per call, this
// takes 4 to 6.  The C entry points are passed in once as addresses (init), so
// this module does not link against libptc.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>

#include "ptc.h"

namespace {

decltype(&ptc_dropout_to) f_dropout;
decltype(&ptc_quantize_fp4) f_quantize;
decltype(&ptc_dequantize_fp4) f_dequantize;
decltype(&gemm_fp4) f_gemm;
decltype(&gemm_a16_fp4) f_gemm_a16;
PyObject *g_check;   // raises PtcError for a status
PyObject *g_stream;  // a stream argument to its handle
PyTypeObject *g_matrix;
PyObject *s_codes, *s_scales, *s_k, *s_fmt, *s_ts;

struct Bad {};  // a Python exception has been set

[[noreturn]] void raise(PyObject *type, const char *text) {
    PyErr_SetString(type, text);
    throw Bad();
}

// An owned reference.
struct Ref {
    PyObject *p;
    explicit Ref(PyObject *o) : p(o) {
        if (!p) throw Bad();
    }
    Ref(const Ref &) = delete;
    ~Ref() { Py_XDECREF(p); }
    PyObject *release() {
        PyObject *o = p;
        p = nullptr;
        return o;
    }
};

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Bad();
    }
    return THPVariable_Unpack(o);
}

// The operators are outside autograd: a gradient is not lost without an error.
const at::Tensor &outside_autograd(const at::Tensor &t, const char *name) {
    if (t.requires_grad() && c10::GradMode::is_enabled()) {
        PyErr_Format(PyExc_RuntimeError,
                     "%s requires grad, and this operator gives no gradient: call it under torch.no_grad() or on a "
                     "detached tensor, with the backward pass written out (as fp4_linear does)",
                     name);
        throw Bad();
    }
    return t;
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    return v;
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad();
    return v;
}

uint64_t seed64(PyObject *o) {
    const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
    if (v == uint64_t(-1) && PyErr_Occurred()) throw Bad();
    return v;
}

int type_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return PTC_OUT_F32;
        case at::kBFloat16: return PTC_OUT_BF16;
        case at::kHalf: return PTC_OUT_F16;
        default: raise(PyExc_TypeError, "tensors are float32, bfloat16 or float16");
    }
}

at::ScalarType dtype_of(PyObject *o) {
    if (!THPDtype_Check(o)) raise(PyExc_TypeError, "a torch dtype is expected");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// A 2-D device tensor with unit column stride.
struct Rows {
    void *p;
    int64_t rows, cols, ld;
};

Rows rows_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda() || t.dim() != 2) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D device tensor", name);
        throw Bad();
    }
    Rows r{t.data_ptr(), t.size(0), t.size(1), 0};
    r.ld = r.rows > 1 ? t.stride(0) : r.cols;
    if ((r.cols > 1 && t.stride(1) != 1) || r.ld < r.cols) {
        PyErr_Format(PyExc_ValueError, "%s must have unit column stride and rows that do not overlap", name);
        throw Bad();
    }
    return r;
}

int format_of(PyObject *o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0) return PTC_FP4_MX;
        if (PyUnicode_CompareWithASCIIString(o, "nvfp4") == 0) return PTC_FP4_NV;
    }
    raise(PyExc_ValueError, "fmt is 'mxfp4' or 'nvfp4'");
}

int64_t scale_bytes(int64_t rows, int64_t k, int fmt) {
    const int64_t four = fmt == PTC_FP4_NV ? 64 : 128;
    return (rows + 127) / 128 * ((k + four - 1) / four) * 512;
}

const float *matrix_scale(PyObject *o, int fmt, c10::DeviceIndex index) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "tensor_scale");
    if (fmt != PTC_FP4_NV) raise(PyExc_ValueError, "only nvfp4 has a tensor scale");
    if (t.scalar_type() != at::kFloat || t.numel() != 1 || !t.is_cuda() || t.get_device() != index)
        raise(PyExc_ValueError, "tensor_scale is a float32 tensor of one element on the matrix's device");
    return t.data_ptr<float>();
}

// A 4-bit matrix, checked every time it is used.
struct Matrix {
    void *codes, *scales;
    int64_t rows, pitch, k;
    int fmt;
    const float *g;
    c10::DeviceIndex index;
    at::Device device{at::kCPU};
};

Matrix matrix(PyObject *codes, PyObject *scales, PyObject *k, PyObject *fmt, PyObject *ts) {
    Matrix m;
    m.fmt = format_of(fmt);
    const at::Tensor &c = tensor(codes, "codes"), &s = tensor(scales, "scales");
    if (c.scalar_type() != at::kByte || s.scalar_type() != at::kByte) raise(PyExc_TypeError, "codes and scales are uint8");
    const Rows r = rows_of(c, "codes");
    m.k = integer(k);
    m.codes = r.p;
    m.rows = r.rows;
    // (One row, or rows of no values, have no pitch.)
    m.pitch = r.rows > 1 && m.k > 0 ? r.ld : std::max<int64_t>(16, (r.cols + 15) / 16 * 16);
    if (m.k < 0 || m.k > (int64_t(1) << 30)) raise(PyExc_ValueError, "K must be 0 .. 2^30");
    if (r.cols < (m.k + 31) / 32 * 16 || m.pitch % 16)
        raise(PyExc_ValueError, "codes must hold 16 * ceil(K / 32) bytes per row, rows a multiple of 16 bytes apart");
    if (!s.is_cuda() || !s.is_contiguous() || s.numel() < scale_bytes(m.rows, m.k, m.fmt))
        raise(PyExc_ValueError, "scales must be contiguous and hold whole tiles of 128 rows x 4 blocks");
    if (s.get_device() != c.get_device()) raise(PyExc_ValueError, "codes and scales must be on one device");
    m.scales = s.data_ptr();
    m.device = c.device();
    m.index = c.get_device();
    m.g = matrix_scale(ts, m.fmt, m.index);
    return m;
}

Matrix matrix_of(PyObject *o) {
    if (Py_TYPE(o) != g_matrix && !PyObject_TypeCheck(o, g_matrix)) raise(PyExc_TypeError, "an Fp4Matrix is expected");
    Ref c(PyObject_GetAttr(o, s_codes)), s(PyObject_GetAttr(o, s_scales)), k(PyObject_GetAttr(o, s_k)),
        f(PyObject_GetAttr(o, s_fmt)), t(PyObject_GetAttr(o, s_ts));
    return matrix(c.p, s.p, k.p, f.p, t.p);
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, at::Device device) {
    return at::empty(size, at::TensorOptions().dtype(type).device(device));
}

// A new 4-bit matrix object; its tensors outlive the call in it.
struct NewMatrix {
    Ref object;
    void *codes, *scales;
    int64_t pitch;
    NewMatrix(int64_t rows, int64_t k, int fmt, PyObject *fmt_o, PyObject *ts, at::Device device)
        : object(g_matrix->tp_alloc(g_matrix, 0)) {
        const int64_t width = (k + 31) / 32 * 16;
        at::Tensor c = empty({rows, width}, at::kByte, device), s = empty({scale_bytes(rows, k, fmt)}, at::kByte, device);
        codes = c.data_ptr();
        scales = s.data_ptr();
        pitch = width ? width : 16;
        Ref co(THPVariable_Wrap(std::move(c))), so(THPVariable_Wrap(std::move(s))), ko(PyLong_FromLongLong(k));
        if (PyObject_SetAttr(object.p, s_codes, co.p) || PyObject_SetAttr(object.p, s_scales, so.p) ||
            PyObject_SetAttr(object.p, s_k, ko.p) || PyObject_SetAttr(object.p, s_fmt, fmt_o) ||
            PyObject_SetAttr(object.p, s_ts, ts))
            throw Bad();
    }
};

// Where a call runs: the tensors' device and the stream argument, or the device's
// current stream.  While it lives both are current, so results come from that
// stream's memory: a block that the caching allocator hands out again may still be
// in use on the stream it belongs to, and on no other.  A call on another stream
// than the caller's also tells the allocator so (used): the caller may release its
// inputs, and results, without waiting for that stream.
class Target {
    c10::cuda::CUDAStream caller_;
    void *handle_;
    bool elsewhere_ = false;  // on another stream than the caller's
    c10::cuda::OptionalCUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;

  public:
    Target(c10::DeviceIndex index, PyObject *stream) : caller_(c10::cuda::getCurrentCUDAStream(index)) {
        void *const own = caller_.stream();
        handle_ = own;
        if (stream != Py_None) {
            Ref h(PyObject_CallOneArg(g_stream, stream));
            handle_ = reinterpret_cast<void *>(uintptr_t(seed64(h.p)));
            if (handle_ == cudaStreamLegacy) handle_ = nullptr;  // (torch knows the default stream by that)
            elsewhere_ = handle_ != own;
        }
        if (elsewhere_)
            stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle_), index));
        else if (c10::cuda::current_device() != index)
            device_.set_index(index);
    }
    // f(stream), its status raised.
    template <typename F>
    void run(F f) const {
        const int status = f(handle_);
        if (status) {
            Ref code(PyLong_FromLong(status));
            Ref none(PyObject_CallOneArg(g_check, code.p));
            throw Bad();
        }
    }
    // Of a launched call: tensors of the caller's (a tensor, a 4-bit matrix or None),
    // and results of this stream's memory.
    void used(PyObject *o) const {
        if (elsewhere_) record(o, c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle_), caller_.device_index()));
    }
    void made(PyObject *o) const {
        if (elsewhere_) record(o, caller_);
    }

  private:
    static void record(PyObject *o, c10::cuda::CUDAStream stream) {
        if (THPVariable_Check(o)) {
            THPVariable_Unpack(o).record_stream(stream);
        } else if (o != Py_None) {
            for (PyObject *name : {s_codes, s_scales, s_ts}) record(Ref(PyObject_GetAttr(o, name)).p, stream);
        }
    }
};

// The result tensor: `out`, or a new one.
at::Tensor result(PyObject *out, int64_t rows, int64_t cols, at::ScalarType type, c10::DeviceIndex index, at::Device device) {
    if (out == Py_None) return empty({rows, cols}, type, device);
    const at::Tensor &t = outside_autograd(tensor(out, "out"), "out");
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || !t.is_cuda() || t.get_device() != index)
        raise(PyExc_ValueError, "out must have the result's shape and device");
    return t;
}

PyObject *give(const Target &target, PyObject *out, at::Tensor t) {
    if (out != Py_None) {
        target.used(out);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();  // (written in place)
        Py_INCREF(out);
        return out;
    }
    Ref made(THPVariable_Wrap(std::move(t)));
    target.made(made.p);
    return made.release();
}

void expect(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

#define PTC_BODY_BEGIN \
    HANDLE_TH_ERRORS   \
    try {
#define PTC_BODY_END     \
    } catch (const Bad &) { \
        return nullptr;  \
    }                    \
    END_HANDLE_TH_ERRORS

// (x, p, seed, offset, residual, out, stream, out_dtype)
PyObject *py_dropout(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 8);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    const at::ScalarType st = a[7] == Py_None ? x.scalar_type() : dtype_of(a[7]);
    const int out_type = type_of(st);
    const Rows rx = rows_of(x, "x");
    const c10::DeviceIndex index = x.get_device();
    auto like = [&](const at::Tensor &t, const char *name) {
        if (t.scalar_type() != st || t.sizes() != x.sizes() || !t.is_cuda() || t.get_device() != index) {
            PyErr_Format(PyExc_ValueError, "%s must have the result's shape, dtype and device", name);
            throw Bad();
        }
    };
    Rows rr{nullptr, 0, 0, 0};
    if (a[4] != Py_None) {
        const at::Tensor &r = outside_autograd(tensor(a[4], "residual"), "residual");
        like(r, "residual");
        rr = rows_of(r, "residual");
    }
    if (a[5] != Py_None) like(tensor(a[5], "out"), "out");
    const Target target(index, a[6]);
    at::Tensor y = result(a[5], rx.rows, rx.cols, st, index, x.device());
    const Rows ry = rows_of(y, "out");
    const double p = real(a[1]);
    const uint64_t seed = seed64(a[2]), offset = uint64_t(integer(a[3]));
    target.run([&](void *s) {
        return f_dropout(rx.rows, rx.cols, rx.p, rx.ld, type, rr.p, rr.ld, ry.p, ry.ld, out_type, p, seed, offset, s);
    });
    target.used(a[0]);
    target.used(a[4]);
    return give(target, a[5], std::move(y));
    PTC_BODY_END
}

// (x, fmt, transposed: 0 rows, 1 columns, 2 both, rounding, tensor_scale, p, seed, offset, stream)
PyObject *py_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 9);
    const int fmt = format_of(a[1]);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    const Rows rx = rows_of(x, "x");
    const c10::DeviceIndex index = x.get_device();
    const float *g = matrix_scale(a[4], fmt, index);
    const int64_t which = integer(a[2]);
    const int rounding = int(integer(a[3]));
    const double p = real(a[5]);
    const uint64_t seed = seed64(a[6]), offset = uint64_t(integer(a[7]));
    const Target target(index, a[8]);
    auto run = [&](NewMatrix *q, NewMatrix *t) {
        target.run([&](void *s) {
            return f_quantize(rx.rows, rx.cols, rx.p, rx.ld, type, fmt, rounding, g, q ? q->codes : nullptr, q ? q->pitch : 0,
                              q ? q->scales : nullptr, t ? t->codes : nullptr, t ? t->pitch : 0, t ? t->scales : nullptr, p,
                              seed, offset, s);
        });
        target.used(a[0]);
        target.used(a[4]);
        for (const NewMatrix *m : {q, t})
            if (m) target.made(m->object.p);
    };
    if (which == 0) {
        NewMatrix q(rx.rows, rx.cols, fmt, a[1], a[4], x.device());
        run(&q, nullptr);
        return q.object.release();
    }
    NewMatrix t(rx.cols, rx.rows, fmt, a[1], a[4], x.device());
    if (which == 1) {
        run(nullptr, &t);
        return t.object.release();
    }
    NewMatrix q(rx.rows, rx.cols, fmt, a[1], a[4], x.device());
    run(&q, &t);
    return PyTuple_Pack(2, q.object.p, t.object.p);
    PTC_BODY_END
}

// dtype argument (None: `or_else`) or out's.
at::ScalarType out_type(PyObject *dtype, PyObject *out, at::ScalarType or_else) {
    if (out != Py_None) return tensor(out, "out").scalar_type();
    return dtype == Py_None ? or_else : dtype_of(dtype);
}

// (q, dtype, out, stream)
PyObject *py_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 4);
    const Matrix m = matrix_of(a[0]);
    const at::ScalarType st = out_type(a[1], a[2], at::kBFloat16);
    const int type = type_of(st);
    const Target target(m.index, a[3]);
    at::Tensor y = result(a[2], m.rows, m.k, st, m.index, m.device);
    const Rows ry = rows_of(y, "out");
    target.run([&](void *s) {
        return f_dequantize(m.rows, m.k, m.codes, m.pitch, m.scales, m.fmt, m.g, ry.p, ry.ld, type, s);
    });
    target.used(a[0]);
    return give(target, a[2], std::move(y));
    PTC_BODY_END
}

// (A, Bt, out_dtype, out, stream)
PyObject *py_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 5);
    const Matrix A = matrix_of(a[0]), B = matrix_of(a[1]);
    if (A.fmt != B.fmt) raise(PyExc_ValueError, "both matrices must have the same format");
    if (A.k != B.k) raise(PyExc_ValueError, "inner dimensions differ");
    if (A.index != B.index) raise(PyExc_ValueError, "both matrices must be on one device");
    const at::ScalarType st = out_type(a[2], a[3], at::kBFloat16);
    const int type = type_of(st);
    const Target target(A.index, a[4]);
    at::Tensor c = result(a[3], A.rows, B.rows, st, A.index, A.device);
    const Rows rc = rows_of(c, "out");
    target.run([&](void *s) {
        return f_gemm(A.rows, B.rows, A.k, A.fmt, A.codes, A.pitch, A.scales, A.g, B.codes, B.pitch, B.scales, B.g,
                      rc.p, rc.ld, type, s);
    });
    target.used(a[0]);
    target.used(a[1]);
    return give(target, a[3], std::move(c));
    PTC_BODY_END
}

// (x, Wt, out, stream)
PyObject *py_matmul_a16(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 4);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    if (type == PTC_OUT_F32) raise(PyExc_TypeError, "matmul_a16_fp4 takes bfloat16 or float16 activations");
    const Rows rx = rows_of(x, "x");
    const Matrix W = matrix_of(a[1]);
    if (rx.cols != W.k) raise(PyExc_ValueError, "inner dimensions differ");
    if (x.get_device() != W.index || (a[2] != Py_None && tensor(a[2], "out").scalar_type() != x.scalar_type()))
        raise(PyExc_ValueError, "x, the weights and out must share a device, x and out a dtype");
    const Target target(W.index, a[3]);
    at::Tensor c = result(a[2], rx.rows, W.rows, x.scalar_type(), W.index, W.device);
    const Rows rc = rows_of(c, "out");
    target.run([&](void *s) {
        return f_gemm_a16(rx.rows, W.rows, W.k, type, rx.p, rx.ld, W.fmt, W.codes, W.pitch, W.scales, W.g, rc.p, rc.ld, s);
    });
    target.used(a[0]);
    target.used(a[1]);
    return give(target, a[2], std::move(c));
    PTC_BODY_END
}

// (codes, scales, K, fmt, tensor_scale): raises what is wrong with them
PyObject *py_check_matrix(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 5);
    matrix(a[0], a[1], a[2], a[3], a[4]);
    Py_RETURN_NONE;
    PTC_BODY_END
}

// (addresses of the five C entry points, status check, stream handle, Fp4Matrix)
PyObject *py_init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 8);
    f_dropout = reinterpret_cast<decltype(f_dropout)>(uintptr_t(seed64(a[0])));
    f_quantize = reinterpret_cast<decltype(f_quantize)>(uintptr_t(seed64(a[1])));
    f_dequantize = reinterpret_cast<decltype(f_dequantize)>(uintptr_t(seed64(a[2])));
    f_gemm = reinterpret_cast<decltype(f_gemm)>(uintptr_t(seed64(a[3])));
    f_gemm_a16 = reinterpret_cast<decltype(f_gemm_a16)>(uintptr_t(seed64(a[4])));
    if (!PyType_Check(a[7])) raise(PyExc_TypeError, "a type is expected");
    Py_XSETREF(g_check, Py_NewRef(a[5]));
    Py_XSETREF(g_stream, Py_NewRef(a[6]));
    PyTypeObject *old = g_matrix;
    g_matrix = reinterpret_cast<PyTypeObject *>(Py_NewRef(a[7]));
    Py_XDECREF(old);
    if (!s_codes) {
        s_codes = PyUnicode_InternFromString("_codes");
        s_scales = PyUnicode_InternFromString("_scales");
        s_k = PyUnicode_InternFromString("_K");
        s_fmt = PyUnicode_InternFromString("_fmt");
        s_ts = PyUnicode_InternFromString("_ts");
    }
    Py_RETURN_NONE;
    PTC_BODY_END
}

#define PTC_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PTC_METHOD("init", py_init),
                           PTC_METHOD("dropout", py_dropout),
                           PTC_METHOD("quantize", py_quantize),
                           PTC_METHOD("dequantize", py_dequantize),
                           PTC_METHOD("matmul", py_matmul),
                           PTC_METHOD("matmul_a16", py_matmul_a16),
                           PTC_METHOD("check_matrix", py_check_matrix),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
