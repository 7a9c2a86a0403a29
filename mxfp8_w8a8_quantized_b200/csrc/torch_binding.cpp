/*
 * torch_binding.cpp -- the Python side of the operators that a serving
 * program calls once per token: the RMS norm, the gated activation and the
 * MXFP4 layer.  It checks the tensors, allocates the outputs that were not
 * given, and calls the C-ABI of libmxfp8.so with their addresses on the
 * current CUDA stream; there is no arithmetic here and no fallback.
 *
 * A kernel for one token takes about 3 us and its launch about as long; the
 * same checks and allocations written in Python cost 9 us more per call (norm of
 * one token, 13.8 us), which is why these calls do not go through ctypes.
 *
 * The library is called without the interpreter's lock: a launch waits while the
 * queue of launches is full, and other Python threads run on meanwhile.  What the
 * call uses is held by its arguments and this frame.
 *
 * Every function takes positional arguments; mxfp8.py declares the signatures,
 * defaults and documentation.  A wrong tensor raises ValueError before the
 * library is called; a status other than 0 raises MXFP8Error.
 */
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <string>

#include "fp8_rowwise.h"
#include "mxfp4.h"
#include "mxfp8.h"
#include "nvfp4.h"

namespace {

/* Formats, as mxfp8.py numbers them. */
enum Fmt : long { MXFP8 = 0, FP8RW = 1, NVFP4 = 2, MXFP4 = 3 };

PyObject *g_error = nullptr; /* MXFP8Error */

[[noreturn]] void refuse(const std::string &why)
{
    PyErr_SetString(PyExc_ValueError, why.c_str());
    throw python_error();
}

std::string shape_of(at::IntArrayRef s)
{
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

bool given(PyObject *o)
{
    return o != Py_None;
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

/* The current device, on which the call's first tensor must live. */
int device_of(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda())
        refuse(std::string(name) + " must be a CUDA tensor");
    const int dev = t.get_device(), cur = c10::cuda::current_device();
    if (dev != cur)
        refuse(std::string(name) + " is on cuda:" + std::to_string(dev) + ", but the current device is cuda:" +
               std::to_string(cur));
    return dev;
}

const at::Tensor &on_device(PyObject *o, const char *name, int dev)
{
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda() || t.get_device() != dev)
        refuse(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev));
    return t;
}

/* A contiguous tensor of one type. */
const at::Tensor &dense(PyObject *o, const char *name, int dev, at::ScalarType type)
{
    const at::Tensor &t = on_device(o, name, dev);
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_contiguous())
        refuse(std::string(name) + " must be contiguous");
    return t;
}

/* An int argument of the C-ABI: a wider value is no other value's last 32 bits. */
int small_int(PyObject *o, const char *name)
{
    int beyond = 0;
    const long v = PyLong_AsLongAndOverflow(o, &beyond);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    if (beyond != 0 || v != (int)v)
        refuse(std::string(name) + " is out of range");
    return (int)v;
}

/* A 2-D BF16 tensor whose rows may be strided. */
struct Rows {
    void *p;
    int64_t M, K, ld;
};

Rows rows(PyObject *o, const char *name, int dev, const Rows *like = nullptr)
{
    const at::Tensor &t = on_device(o, name, dev);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 2)
        refuse(std::string(name) + " must be a 2-D BF16 CUDA tensor");
    Rows r{t.data_ptr(), t.size(0), t.size(1), t.stride(0)};
    if (like && (r.M != like->M || r.K != like->K))
        refuse(std::string(name) + " must be " + shape_of({like->M, like->K}) + ", got " + shape_of(t.sizes()));
    if (r.M <= 1)
        r.ld = r.K;
    if ((t.stride(1) != 1 && r.K > 1) || r.ld < r.K)
        refuse(std::string(name) + " must have unit column stride and row stride >= its columns");
    return r;
}

/* Whether two [M, K] views share memory (views of different row strides count
 * as sharing where their address ranges meet). */
bool overlap(const Rows &a, const Rows &b)
{
    if (a.M == 0 || a.K == 0)
        return false;
    const int64_t pa = (int64_t)(intptr_t)a.p, pb = (int64_t)(intptr_t)b.p;
    const int64_t na = 2 * ((a.M - 1) * a.ld + a.K), nb = 2 * ((b.M - 1) * b.ld + b.K);
    if (pa >= pb + nb || pb >= pa + na)
        return false;
    if (a.ld != b.ld)
        return true;
    const int64_t row = 2 * a.ld, d = ((pb - pa) % row + row) % row; /* columns of one buffer? */
    return d < 2 * a.K || row - d < 2 * a.K;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), c10::nullopt));
}

/* An output [a, b] that the caller may have given. */
at::Tensor matrix_out(PyObject *o, const char *name, int dev, at::ScalarType type, int64_t a, int64_t b)
{
    if (!given(o))
        return fresh({a, b}, type, dev);
    const at::Tensor &t = dense(o, name, dev, type);
    if (t.dim() != 2 || t.size(0) != a || t.size(1) != b)
        refuse(std::string(name) + " must be " + shape_of({a, b}) + ", got " + shape_of(t.sizes()));
    return t;
}

/* An output of n values; a given one may be longer. */
at::Tensor vector_out(PyObject *o, const char *name, int dev, at::ScalarType type, int64_t n)
{
    if (!given(o))
        return fresh({n}, type, dev);
    const at::Tensor &t = dense(o, name, dev, type);
    if (t.dim() != 1 || t.size(0) < n)
        refuse(std::string(name) + " must hold " + std::to_string(n) + " values, got " + shape_of(t.sizes()));
    return t;
}

/* Bytes of the tensor-core scale layout, `group` elements of K per atom. */
int64_t atom_bytes(int64_t rows, int64_t K, int64_t group)
{
    return std::max<int64_t>((rows + 127) / 128 * ((K + group - 1) / group) * 512, 1);
}

/* Codes and scales of an [M, K] result. */
struct Quantized {
    at::Tensor codes, scales;
    const float *g = nullptr;
    int layout = MXFP8_SF_TCGEN05;
};

Quantized quantized_out(long fmt, PyObject *codes, PyObject *scales, PyObject *extra, int dev, int64_t M, int64_t K)
{
    Quantized q;
    const bool fp4 = fmt == NVFP4 || fmt == MXFP4;
    if (fmt == NVFP4) {
        const at::Tensor &g = dense(extra, "global_scale", dev, at::kFloat);
        if (g.numel() != 1)
            refuse("global_scale must hold one FP32 value");
        q.g = g.data_ptr<float>();
    } else if (fmt == MXFP8) {
        q.layout = small_int(extra, "layout");
    }
    q.codes = matrix_out(codes, "codes", dev, at::kByte, M, fp4 ? K / 2 : K);
    if (fmt == FP8RW)
        q.scales = vector_out(scales, "scales", dev, at::kFloat, M);
    else
        q.scales = vector_out(scales, "scales", dev, at::kByte,
                              fmt == MXFP8 && q.layout != MXFP8_SF_TCGEN05 ? std::max<int64_t>(M * K / 32, 1)
                                                                           : atom_bytes(M, K, fmt == NVFP4 ? 64 : 128));
    return q;
}

mxfp8_stream_t stream_of(int dev)
{
    return reinterpret_cast<mxfp8_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

void check(mxfp8_status st, const char *where)
{
    if (st == MXFP8_OK)
        return;
    PyObject *e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "is", (int)st, where);
    if (e) {
        PyErr_SetObject((PyObject *)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    throw python_error();
}

/* Calls the library, the interpreter's lock released. */
template <class... P, class... A>
void call(const char *where, mxfp8_status (*function)(P...), A... args)
{
    PyThreadState *state = PyEval_SaveThread();
    const mxfp8_status st = function(args...);
    PyEval_RestoreThread(state);
    check(st, where);
}

void count(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        throw python_error();
    }
}

long integer(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

PyObject *tuple2(const at::Tensor &a, const at::Tensor &b)
{
    THPObjectPtr t(PyTuple_New(2));
    if (!t)
        throw python_error();
    PyTuple_SET_ITEM(t.get(), 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t.get(), 1, THPVariable_Wrap(b));
    return t.release();
}

/* rmsnorm(fmt, x, weight, eps, residual, extra, codes, scales, residual_out);
 * extra: the scale layout (MXFP8) or the global scale (NVFP4) */
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    const long fmt = integer(a[0]);
    const int dev = device_of(a[1], "x");
    const Rows x = rows(a[1], "x", dev);
    const at::Tensor &w = on_device(a[2], "weight", dev);
    const at::ScalarType wt = w.scalar_type();
    if (wt != at::kBFloat16 && wt != at::kHalf && wt != at::kFloat)
        refuse("weight must be a BF16, FP16 or FP32 CUDA tensor");
    if (w.dim() != 1 || w.size(0) != x.K || !w.is_contiguous())
        refuse("weight must be a contiguous [" + std::to_string(x.K) + "], got " + shape_of(w.sizes()));
    const int wdt = wt == at::kBFloat16 ? MXFP8_DTYPE_BF16 : wt == at::kHalf ? MXFP8_DTYPE_F16 : MXFP8_DTYPE_F32;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred())
        throw python_error();
    Rows r{nullptr, 0, 0, 0}, h{nullptr, 0, 0, 0};
    at::Tensor stream_out;
    if (given(a[4])) {
        r = rows(a[4], "residual", dev, &x);
        if (given(a[8])) {
            h = rows(a[8], "residual_out", dev, &x);
            for (const Rows &t : {x, r})
                if (overlap(h, t) && (h.p != t.p || h.ld != t.ld))
                    refuse("residual_out must be x, residual or memory of its own");
            stream_out = THPVariable_Unpack(a[8]);
        } else {
            stream_out = fresh({x.M, x.K}, at::kBFloat16, dev);
            h = Rows{stream_out.data_ptr(), x.M, x.K, x.K};
        }
    } else if (given(a[8])) {
        refuse("residual_out needs a residual");
    }
    const Quantized q = quantized_out(fmt, a[6], a[7], a[5], dev, x.M, x.K);
    void *codes = q.codes.data_ptr(), *scales = q.scales.data_ptr();
    const mxfp8_stream_t s = stream_of(dev);
    switch (fmt) {
    case MXFP8:
        call("mxfp8_rmsnorm_quantize", mxfp8_rmsnorm_quantize, x.p, x.ld, r.p, r.ld, h.p, h.ld, w.data_ptr(), wdt,
             (float)eps, x.M, x.K, codes, scales, q.layout, s);
        break;
    case FP8RW:
        call("fp8rw_rmsnorm_quantize", fp8rw_rmsnorm_quantize, x.p, x.ld, r.p, r.ld, h.p, h.ld, w.data_ptr(), wdt,
             (float)eps, x.M, x.K, codes, static_cast<float *>(scales), s);
        break;
    case NVFP4:
        call("nvfp4_rmsnorm_quantize", nvfp4_rmsnorm_quantize, x.p, x.ld, r.p, r.ld, h.p, h.ld, w.data_ptr(), wdt,
             (float)eps, x.M, x.K, q.g, codes, scales, s);
        break;
    default:
        call("mxfp4_rmsnorm_quantize", mxfp4_rmsnorm_quantize, x.p, x.ld, r.p, r.ld, h.p, h.ld, w.data_ptr(), wdt,
             (float)eps, x.M, x.K, codes, scales, s);
    }
    THPObjectPtr t(PyTuple_New(3));
    if (!t)
        throw python_error();
    PyTuple_SET_ITEM(t.get(), 0, THPVariable_Wrap(q.codes));
    PyTuple_SET_ITEM(t.get(), 1, THPVariable_Wrap(q.scales));
    PyObject *ho = given(a[4]) ? (given(a[8]) ? Py_NewRef(a[8]) : THPVariable_Wrap(stream_out)) : Py_NewRef(a[1]);
    PyTuple_SET_ITEM(t.get(), 2, ho);
    return t.release();
    END_HANDLE_TH_ERRORS
}

/* gated(fmt, gate, up, act, extra, codes, scales) */
PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 7);
    const long fmt = integer(a[0]);
    const int dev = device_of(a[1], "gate");
    const Rows g = rows(a[1], "gate", dev);
    const Rows u = rows(a[2], "up", dev, &g);
    const int act = small_int(a[3], "act");
    const Quantized q = quantized_out(fmt, a[5], a[6], a[4], dev, g.M, g.K);
    void *codes = q.codes.data_ptr(), *scales = q.scales.data_ptr();
    const mxfp8_stream_t s = stream_of(dev);
    switch (fmt) {
    case MXFP8:
        call("mxfp8_gated_quantize", mxfp8_gated_quantize, g.p, g.ld, u.p, u.ld, act, g.M, g.K, codes, scales,
             q.layout, s);
        break;
    case FP8RW:
        call("fp8rw_gated_quantize", fp8rw_gated_quantize, g.p, g.ld, u.p, u.ld, act, g.M, g.K, codes,
             static_cast<float *>(scales), s);
        break;
    case NVFP4:
        call("nvfp4_gated_quantize", nvfp4_gated_quantize, g.p, g.ld, u.p, u.ld, act, g.M, g.K, q.g, codes, scales,
             s);
        break;
    default:
        call("mxfp4_gated_quantize", mxfp4_gated_quantize, g.p, g.ld, u.p, u.ld, act, g.M, g.K, codes, scales, s);
    }
    return tuple2(q.codes, q.scales);
    END_HANDLE_TH_ERRORS
}

/* quantize(x, codes, scales): BF16 to MXFP4 */
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 3);
    const int dev = device_of(a[0], "x");
    const Rows x = rows(a[0], "x", dev);
    const Quantized q = quantized_out(MXFP4, a[1], a[2], Py_None, dev, x.M, x.K);
    call("mxfp4_quantize_bf16", mxfp4_quantize_bf16, x.p, x.M, x.K, x.ld, q.codes.data_ptr(), q.scales.data_ptr(),
         stream_of(dev));
    return tuple2(q.codes, q.scales);
    END_HANDLE_TH_ERRORS
}

/* An MXFP4 matrix: packed codes [rows, K / 2] and their scales. */
struct Operand {
    const void *codes, *scales;
    int64_t rows, K;
};

Operand operand(PyObject *codes, PyObject *scales, const char *cn, const char *sn, int dev)
{
    const at::Tensor &q = dense(codes, cn, dev, at::kByte);
    const at::Tensor &s = dense(scales, sn, dev, at::kByte);
    if (q.dim() != 2)
        refuse(std::string(cn) + " must be 2-D");
    const Operand r{q.data_ptr(), s.data_ptr(), q.size(0), 2 * q.size(1)};
    if (r.rows > 0 && s.numel() < atom_bytes(r.rows, r.K, 128))
        refuse(std::string(sn) + " are too short for " + shape_of(q.sizes()) + " packed codes");
    return r;
}

const void *bias_of(PyObject *o, int64_t N, int dev)
{
    if (!given(o))
        return nullptr;
    const at::Tensor &b = dense(o, "bias", dev, at::kHalf);
    if (b.numel() != N)
        refuse("bias must hold " + std::to_string(N) + " values, got " + std::to_string(b.numel()));
    return b.data_ptr();
}

/* gemm(xq, xscale, wq, wscale, bias, out) */
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    const int dev = device_of(a[0], "x codes");
    const Operand x = operand(a[0], a[1], "x codes", "x scales", dev);
    const Operand w = operand(a[2], a[3], "w codes", "w scales", dev);
    if (x.K != w.K)
        refuse("x and w must have the same K, got " + std::to_string(x.K) + " and " + std::to_string(w.K));
    const void *b = bias_of(a[4], w.rows, dev);
    const at::Tensor y = matrix_out(a[5], "out", dev, at::kBFloat16, x.rows, w.rows);
    call("mxfp4_gemm", mxfp4_gemm, x.codes, x.scales, x.rows, x.K, w.codes, w.scales, w.rows, b, y.data_ptr(),
         stream_of(dev));
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

/* linear(x, wq, wscale, bias, out, workspace) */
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    const int dev = device_of(a[0], "x");
    const at::Tensor &x = dense(a[0], "x", dev, at::kBFloat16);
    const Operand w = operand(a[1], a[2], "w codes", "w scales", dev);
    if (x.dim() != 2 || x.size(1) != w.K)
        refuse("x must be [M, " + std::to_string(w.K) + "], got " + shape_of(x.sizes()));
    const int64_t M = x.size(0);
    const void *b = bias_of(a[3], w.rows, dev);
    const at::Tensor y = matrix_out(a[4], "out", dev, at::kBFloat16, M, w.rows);
    const at::Tensor wk = given(a[5]) ? dense(a[5], "workspace", dev, at::kByte)
                                      : fresh({(M * w.K / 2 + 255) / 256 * 256 + atom_bytes(M, w.K, 128)}, at::kByte, dev);
    call("mxfp4_linear", mxfp4_linear, x.data_ptr(), M, w.K, w.codes, w.scales, w.rows, b, y.data_ptr(),
         wk.data_ptr(), (size_t)wk.numel(), stream_of(dev));
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *e)
{
    Py_XSETREF(g_error, Py_NewRef(e));
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__native(void)
{
    PyObject *m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", MXFP8_BUILT_FOR) != 0) { /* build.native_tag() */
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
