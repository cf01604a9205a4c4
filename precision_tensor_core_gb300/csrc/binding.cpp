// binding.cpp -- CPython functions behind the 4-bit operators and the norms of the
// package's tensor layer: they check torch tensors, allocate results, and call the C ABI of
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
#include <type_traits>

#include "ptc.h"

namespace {

decltype(&ptc_dropout_to) f_dropout;
decltype(&ptc_quantize_fp4) f_quantize;
decltype(&ptc_dequantize_fp4) f_dequantize;
decltype(&gemm_fp4) f_gemm;
decltype(&gemm_a16_fp4) f_gemm_a16;
decltype(&gemm_a16_s4_workspace) f_gemm_a16_s4_workspace;
decltype(&gemm_a16_s4) f_gemm_a16_s4;
decltype(&ptc_moe_a16_s4_workspace) f_moe_workspace;
decltype(&ptc_moe_a16_s4) f_moe;
decltype(&ptc_rms_norm) f_norm;
decltype(&ptc_rms_norm_s8) f_norm_s8;
decltype(&ptc_rms_norm_backward_workspace) f_norm_workspace;
decltype(&ptc_rms_norm_backward) f_norm_backward;
PyObject *g_check;   // raises PtcError for a status
PyObject *g_stream;  // a stream argument to its handle
PyTypeObject *g_matrix, *g_s4;  // Fp4Matrix, S4Matrix
PyObject *s_codes, *s_scales, *s_k, *s_fmt, *s_ts, *s_group, *s_zeros;

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

// Grouped 4-bit integer weights, of one matrix or of several (experts), checked every
// time they are used.
struct S4 {
    void *codes, *scales, *zeros;
    int64_t experts, rows, pitch, expert, k, group;
    int type;
    bool many;
    c10::DeviceIndex index;
    at::Device device{at::kCPU};
};

S4 s4(PyObject *codes, PyObject *scales, PyObject *k, PyObject *group, PyObject *zeros) {
    S4 m;
    const at::Tensor &c = tensor(codes, "codes"), &s = tensor(scales, "scales");
    if (c.scalar_type() != at::kByte) raise(PyExc_TypeError, "codes are uint8");
    if (s.scalar_type() != at::kBFloat16 && s.scalar_type() != at::kHalf)
        raise(PyExc_TypeError, "scales are bfloat16 or float16");
    if (!c.is_cuda() || (c.dim() != 2 && c.dim() != 3)) raise(PyExc_ValueError, "codes must be a 2-D or 3-D device tensor");
    m.many = c.dim() == 3;
    m.experts = m.many ? c.size(0) : 1;
    m.rows = c.size(-2);
    m.k = integer(k);
    m.group = integer(group);
    if (m.k < 0 || m.k > (int64_t(1) << 30)) raise(PyExc_ValueError, "K must be 0 .. 2^30");
    if (m.group != 32 && m.group != 64 && (m.group <= 0 || m.group % 128))
        raise(PyExc_ValueError, "group is 32, 64 or a multiple of 128");
    // (One row, or rows of no values, have no pitch; nor has one expert.)
    const int64_t least = std::max<int64_t>(16, (c.size(-1) + 15) / 16 * 16);
    m.pitch = m.rows > 1 && m.k > 0 ? c.stride(-2) : least;
    m.expert = m.experts > 1 ? c.stride(0) : 0;
    if (c.size(-1) < (m.k + 1) / 2 || (c.size(-1) > 1 && c.stride(-1) != 1) || m.pitch < c.size(-1) || m.pitch % 16 ||
        m.expert % 16 || (m.experts > 1 && m.rows > 0 && m.expert < (m.rows - 1) * m.pitch + c.size(-1)))
        raise(PyExc_ValueError, "codes must hold ceil(K / 2) bytes per row, rows (and experts) a multiple of 16 bytes apart");
    const int64_t count = m.experts * ((m.rows + 15) / 16) * ((m.k + m.group - 1) / m.group) * 16;
    auto tiles = [&](const at::Tensor &t, const char *name) {
        if (t.scalar_type() != s.scalar_type() || !t.is_cuda() || t.get_device() != c.get_device() || !t.is_contiguous() ||
            t.numel() < count) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous, of the scales' dtype on the codes' device, and hold whole "
                         "tiles of 16 rows", name);
            throw Bad();
        }
        return t.data_ptr();
    };
    m.scales = tiles(s, "scales");
    m.zeros = zeros == Py_None ? nullptr : tiles(tensor(zeros, "zeros"), "zeros");
    m.codes = c.data_ptr();
    m.type = s.scalar_type() == at::kHalf ? PTC_OUT_F16 : PTC_OUT_BF16;
    m.device = c.device();
    m.index = c.get_device();
    return m;
}

S4 s4_of(PyObject *o) {
    if (Py_TYPE(o) != g_s4 && !PyObject_TypeCheck(o, g_s4)) raise(PyExc_TypeError, "an S4Matrix is expected");
    Ref c(PyObject_GetAttr(o, s_codes)), s(PyObject_GetAttr(o, s_scales)), k(PyObject_GetAttr(o, s_k)),
        g(PyObject_GetAttr(o, s_group)), z(PyObject_GetAttr(o, s_zeros));
    return s4(c.p, s.p, k.p, g.p, z.p);
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
    // Of a launched call: tensors of the caller's (a tensor, a matrix object or None),
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
            for (PyObject *name : {s_codes, s_scales, PyObject_TypeCheck(o, g_s4) ? s_zeros : s_ts}) record(Ref(PyObject_GetAttr(o, name)).p, stream);
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

// (x, Wt, out, stream)
PyObject *py_matmul_a16_s4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 4);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    if (type == PTC_OUT_F32) raise(PyExc_TypeError, "matmul_a16_s4 takes bfloat16 or float16 activations");
    const Rows rx = rows_of(x, "x");
    const S4 W = s4_of(a[1]);
    if (W.many) raise(PyExc_ValueError, "the weights are several matrices (experts)");
    if (rx.cols != W.k) raise(PyExc_ValueError, "inner dimensions differ");
    if (x.get_device() != W.index || (a[2] != Py_None && tensor(a[2], "out").scalar_type() != x.scalar_type()))
        raise(PyExc_ValueError, "x, the weights and out must share a device, x and out a dtype");
    const Target target(W.index, a[3]);
    at::Tensor c = result(a[2], rx.rows, W.rows, x.scalar_type(), W.index, W.device);
    const Rows rc = rows_of(c, "out");
    const int64_t bytes = f_gemm_a16_s4_workspace(rx.rows, W.k);
    at::Tensor ws;
    if (bytes > 0) ws = empty({bytes}, at::kByte, W.device);
    target.run([&](void *s) {
        return f_gemm_a16_s4(rx.rows, W.rows, W.k, type, rx.p, rx.ld, W.codes, W.pitch, W.group, W.type, W.scales, W.zeros,
                             rc.p, rc.ld, bytes > 0 ? ws.data_ptr() : nullptr, bytes, s);
    });
    target.used(a[0]);
    target.used(a[1]);
    return give(target, a[2], std::move(c));
    PTC_BODY_END
}

// (x, router, gate_up, down, top_k, renormalize, out, return_routing, stream)
PyObject *py_moe(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 9);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x"), &router = outside_autograd(tensor(a[1], "router"), "router");
    const int type = type_of(x.scalar_type()), router_type = type_of(router.scalar_type());
    if (type == PTC_OUT_F32) raise(PyExc_TypeError, "moe_a16_s4 takes bfloat16 or float16 activations");
    if (router_type != type && router_type != PTC_OUT_F32) raise(PyExc_TypeError, "router is of x's dtype or float32");
    const Rows rx = rows_of(x, "x"), rr = rows_of(router, "router");
    const S4 gu = s4_of(a[2]), dn = s4_of(a[3]);
    const int64_t top_k = integer(a[4]);
    const int renormalize = PyObject_IsTrue(a[5]), routing = PyObject_IsTrue(a[7]);
    if (renormalize < 0 || routing < 0) throw Bad();
    if (!gu.many || !dn.many) raise(PyExc_ValueError, "gate_up and down hold several matrices (experts)");
    if (gu.experts != dn.experts || gu.experts != rr.rows || gu.k != rx.cols || rr.cols != rx.cols || gu.rows != 2 * dn.k ||
        dn.rows != rx.cols)
        raise(PyExc_ValueError, "sizes differ: x (tokens, hidden), router (experts, hidden), gate_up (experts, 2 inner, hidden), "
                                "down (experts, hidden, inner)");
    if (gu.group != dn.group || gu.type != dn.type) raise(PyExc_ValueError, "gate_up and down must share their group and scales' dtype");
    const c10::DeviceIndex index = x.get_device();
    if (gu.index != index || dn.index != index || router.get_device() != index ||
        (a[6] != Py_None && tensor(a[6], "out").scalar_type() != x.scalar_type()))
        raise(PyExc_ValueError, "x, router, the weights and out must share a device, x and out a dtype");
    const int64_t bytes = rx.rows ? f_moe_workspace(rx.rows, rx.cols, dn.k, gu.experts, top_k) : 0;
    const Target target(index, a[8]);
    at::Tensor y = result(a[6], rx.rows, rx.cols, x.scalar_type(), index, x.device());
    const Rows ry = rows_of(y, "out");
    at::Tensor ids, weights, ws = empty({bytes}, at::kByte, x.device());
    if (routing && top_k >= 0 && (bytes > 0 || rx.rows == 0)) {  // (of other sizes the call is refused)
        ids = empty({rx.rows, top_k}, at::kInt, x.device());
        weights = empty({rx.rows, top_k}, at::kFloat, x.device());
    }
    target.run([&](void *s) {
        return f_moe(rx.rows, rx.cols, dn.k, gu.experts, top_k, renormalize, type, rx.p, rx.ld, rr.p, rr.ld, router_type, gu.group,
                     gu.type, gu.codes, gu.pitch, gu.expert, gu.scales, gu.zeros, dn.codes, dn.pitch, dn.expert, dn.scales, dn.zeros,
                     ry.p, ry.ld, ids.defined() ? static_cast<int32_t *>(ids.data_ptr()) : nullptr,
                     weights.defined() ? static_cast<float *>(weights.data_ptr()) : nullptr, ws.data_ptr(), bytes, s);
    });
    for (int i : {0, 1, 2, 3}) target.used(a[i]);
    if (!routing) return give(target, a[6], std::move(y));
    Ref yo(give(target, a[6], std::move(y))), io(give(target, Py_None, std::move(ids))), wo(give(target, Py_None, std::move(weights)));
    return PyTuple_Pack(3, yo.p, io.p, wo.p);
    PTC_BODY_END
}

// What the norms share: x, an optional tensor of x's shape, type and device, and the weight.
const at::Tensor &same_as(const at::Tensor &x, const char *of, const at::Tensor &t, const char *name) {
    if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes() || !t.is_cuda() || t.get_device() != x.get_device()) {
        PyErr_Format(PyExc_ValueError, "%s must have %s's shape, dtype and device", name, of);
        throw Bad();
    }
    return t;
}

Rows optional_rows(const at::Tensor &x, const char *of, PyObject *o, const char *name) {
    if (o == Py_None) return {nullptr, 0, 0, 0};
    return rows_of(same_as(x, of, outside_autograd(tensor(o, name), name), name), name);
}

const void *norm_weight(const at::Tensor &x, PyObject *o, int type, int *w_type) {
    *w_type = type;
    if (o == Py_None) return nullptr;
    const at::Tensor &w = outside_autograd(tensor(o, "weight"), "weight");
    *w_type = type_of(w.scalar_type());
    if (w.dim() != 1 || w.size(0) != x.size(1) || !w.is_contiguous() || !w.is_cuda() || w.get_device() != x.get_device() ||
        (*w_type != type && *w_type != PTC_OUT_F32))
        raise(PyExc_ValueError, "weight must be a contiguous vector of x's columns, of x's dtype or float32, on x's device");
    return w.data_ptr();
}

float epsilon(PyObject *o) {
    const double e = real(o);
    if (!(e >= 0.0 && e <= 3.0e38)) raise(PyExc_ValueError, "eps must be finite and not negative");
    return float(e);
}

// (x, weight, eps, residual, out, sum_out, stream)
PyObject *py_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 7);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    const Rows rx = rows_of(x, "x");
    const c10::DeviceIndex index = x.get_device();
    int wt;
    const void *w = norm_weight(x, a[1], type, &wt);
    const float eps = epsilon(a[2]);
    const Rows rr = optional_rows(x, "x", a[3], "residual");
    const bool res = a[3] != Py_None;
    if (a[4] != Py_None) same_as(x, "x", tensor(a[4], "out"), "out");
    if (a[5] != Py_None) {
        if (!res) raise(PyExc_ValueError, "sum_out is written only with a residual");
        same_as(x, "x", tensor(a[5], "sum_out"), "sum_out");
    }
    const Target target(index, a[6]);
    at::Tensor y = result(a[4], rx.rows, rx.cols, x.scalar_type(), index, x.device());
    at::Tensor sum = res ? result(a[5], rx.rows, rx.cols, x.scalar_type(), index, x.device()) : at::Tensor();
    const Rows ry = rows_of(y, "out"), rs = res ? rows_of(sum, "sum_out") : Rows{nullptr, 0, 0, 0};
    target.run([&](void *s) {
        return f_norm(rx.rows, rx.cols, rx.p, rx.ld, type, rr.p, rr.ld, rs.p, rs.ld, w, wt, eps, ry.p, ry.ld, s);
    });
    for (int i : {0, 1, 3}) target.used(a[i]);
    if (!res) return give(target, a[4], std::move(y));
    Ref yo(give(target, a[4], std::move(y))), so(give(target, a[5], std::move(sum)));
    return PyTuple_Pack(2, yo.p, so.p);
    PTC_BODY_END
}

// (x, weight, eps, residual, sum_out, stream)
PyObject *py_norm_s8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 6);
    const at::Tensor &x = outside_autograd(tensor(a[0], "x"), "x");
    const int type = type_of(x.scalar_type());
    const Rows rx = rows_of(x, "x");
    const c10::DeviceIndex index = x.get_device();
    int wt;
    const void *w = norm_weight(x, a[1], type, &wt);
    const float eps = epsilon(a[2]);
    const Rows rr = optional_rows(x, "x", a[3], "residual");
    const bool res = a[3] != Py_None;
    if (a[4] != Py_None) {
        if (!res) raise(PyExc_ValueError, "sum_out is written only with a residual");
        same_as(x, "x", tensor(a[4], "sum_out"), "sum_out");
    }
    const Target target(index, a[5]);
    // (rows of a multiple of 16 bytes, as the INT8 products take them)
    at::Tensor wide = empty({rx.rows, (rx.cols + 15) / 16 * 16}, at::kChar, x.device());
    at::Tensor codes = wide.size(1) == rx.cols ? wide : wide.narrow(1, 0, rx.cols);
    at::Tensor scale = empty({rx.rows}, at::kFloat, x.device());
    at::Tensor sum = res ? result(a[4], rx.rows, rx.cols, x.scalar_type(), index, x.device()) : at::Tensor();
    const Rows rs = res ? rows_of(sum, "sum_out") : Rows{nullptr, 0, 0, 0};
    target.run([&](void *s) {
        return f_norm_s8(rx.rows, rx.cols, rx.p, rx.ld, type, rr.p, rr.ld, rs.p, rs.ld, w, wt, eps,
                         static_cast<int8_t *>(wide.data_ptr()), wide.size(1), static_cast<float *>(scale.data_ptr()), s);
    });
    for (int i : {0, 1, 3}) target.used(a[i]);
    Ref co(give(target, Py_None, std::move(codes))), sc(give(target, Py_None, std::move(scale)));
    if (!res) return PyTuple_Pack(2, co.p, sc.p);
    Ref so(give(target, a[4], std::move(sum)));
    return PyTuple_Pack(3, co.p, sc.p, so.p);
    PTC_BODY_END
}

// (dy, s, weight, eps, dsum, out, stream)
PyObject *py_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 7);
    const at::Tensor &dy = outside_autograd(tensor(a[0], "dy"), "dy");
    const int type = type_of(dy.scalar_type());
    const Rows rd = rows_of(dy, "dy");
    const c10::DeviceIndex index = dy.get_device();
    const Rows rs = rows_of(same_as(dy, "dy", outside_autograd(tensor(a[1], "s"), "s"), "s"), "s");
    int wt;
    const void *w = norm_weight(dy, a[2], type, &wt);
    const float eps = epsilon(a[3]);
    const Rows rr = optional_rows(dy, "dy", a[4], "dsum");
    if (a[5] != Py_None) same_as(dy, "dy", tensor(a[5], "out"), "out");
    const Target target(index, a[6]);
    at::Tensor dx = result(a[5], rd.rows, rd.cols, dy.scalar_type(), index, dy.device());
    at::Tensor dw = empty({rd.cols}, at::kFloat, dy.device());
    const int64_t bytes = f_norm_workspace(rd.rows, rd.cols);
    at::Tensor ws = empty({bytes}, at::kByte, dy.device());
    const Rows rx = rows_of(dx, "out");
    target.run([&](void *s) {
        return f_norm_backward(rd.rows, rd.cols, rd.p, rd.ld, rs.p, rs.ld, type, rr.p, rr.ld, w, wt, eps, rx.p, rx.ld,
                               static_cast<float *>(dw.data_ptr()), ws.data_ptr(), bytes, s);
    });
    for (int i : {0, 1, 2, 4}) target.used(a[i]);
    Ref xo(give(target, a[5], std::move(dx))), wo(give(target, Py_None, std::move(dw)));
    return PyTuple_Pack(2, xo.p, wo.p);
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

// (codes, scales, K, group, zeros): raises what is wrong with them
PyObject *py_check_s4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 5);
    s4(a[0], a[1], a[2], a[3], a[4]);
    Py_RETURN_NONE;
    PTC_BODY_END
}

// (addresses of the thirteen C entry points, status check, stream handle, Fp4Matrix, S4Matrix)
PyObject *py_init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    PTC_BODY_BEGIN
    expect(n, 17);
    auto entry = [&](auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(uintptr_t(seed64(*a++))); };
    entry(f_dropout);
    entry(f_quantize);
    entry(f_dequantize);
    entry(f_gemm);
    entry(f_gemm_a16);
    entry(f_gemm_a16_s4_workspace);
    entry(f_gemm_a16_s4);
    entry(f_moe_workspace);
    entry(f_moe);
    entry(f_norm);
    entry(f_norm_s8);
    entry(f_norm_workspace);
    entry(f_norm_backward);
    if (!PyType_Check(a[2]) || !PyType_Check(a[3])) raise(PyExc_TypeError, "a type is expected");
    Py_XSETREF(g_check, Py_NewRef(a[0]));
    Py_XSETREF(g_stream, Py_NewRef(a[1]));
    auto type = [](PyTypeObject *&to, PyObject *o) {
        PyTypeObject *old = to;
        to = reinterpret_cast<PyTypeObject *>(Py_NewRef(o));
        Py_XDECREF(old);
    };
    type(g_matrix, a[2]);
    type(g_s4, a[3]);
    if (!s_codes) {
        s_codes = PyUnicode_InternFromString("_codes");
        s_scales = PyUnicode_InternFromString("_scales");
        s_k = PyUnicode_InternFromString("_K");
        s_fmt = PyUnicode_InternFromString("_fmt");
        s_ts = PyUnicode_InternFromString("_ts");
        s_group = PyUnicode_InternFromString("_group");
        s_zeros = PyUnicode_InternFromString("_zeros");
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
                           PTC_METHOD("matmul_a16_s4", py_matmul_a16_s4),
                           PTC_METHOD("moe_a16_s4", py_moe),
                           PTC_METHOD("check_s4", py_check_s4),
                           PTC_METHOD("rms_norm", py_norm),
                           PTC_METHOD("rms_norm_s8", py_norm_s8),
                           PTC_METHOD("rms_norm_backward", py_norm_backward),
                           PTC_METHOD("check_matrix", py_check_matrix),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
