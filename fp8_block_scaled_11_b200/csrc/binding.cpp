// binding.cpp -- the checks and calls of the norm's and the 4-bit operators'
// Python functions (ops.py), as an extension module.
//
// These operators take a few microseconds on the GPU for a token, so what a call
// costs the host shows: with the same checks in Python and the arguments through
// ctypes, a norm's call took 12 us of which the kernel's launch is 2.5.  Nothing
// is allocated or kept here: ops.py allocates what the caller does not give.
//
// Every function returns the library's status (0: launched); a tensor of another
// shape, type, layout or device raises ValueError or TypeError before the library is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "fp8bs.h"

namespace {

// A refusal, raised as the Python exception `type` at the module's boundary.
struct Refusal {
    PyObject* type;
    std::string text;
};

[[noreturn]] void refuse(PyObject* type, const char* what, const std::string& text)
{
    throw Refusal{type, std::string(what) + ": " + text};
}

const at::Tensor& tensor(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what, "expected a tensor");
    return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t)
{
    return t == at::kBFloat16 ? "bf16" : t == at::kFloat ? "fp32" : t == at::kByte ? "uint8" : "another type";
}

std::string on(const at::Device& d) { return " on " + d.str(); }

fp8bs_dtype code(const at::Tensor& t, const char* what)
{
    if (t.scalar_type() == at::kBFloat16) return FP8BS_BF16;
    if (t.scalar_type() != at::kFloat) refuse(PyExc_TypeError, what, "unsupported dtype (bf16 or fp32)");
    return FP8BS_F32;
}

// Address and leading dimension (elements) of a row-major matrix.
struct Mat {
    void* p = nullptr;
    int64_t ld = 0;
};

Mat row_major(const at::Tensor& t, const char* what)
{
    if (t.stride(1) != 1 && t.size(1) != 1) refuse(PyExc_ValueError, what, "expected a row-major matrix (unit column stride)");
    return {t.data_ptr(), t.size(0) != 1 ? t.stride(0) : t.size(1)};        // one row: any stride will do
}

Mat matrix(PyObject* o, int64_t rows, int64_t cols, at::ScalarType type, const at::Device& dev, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.scalar_type() != type || t.device() != dev)
        refuse(PyExc_ValueError, what, "expected " + std::to_string(rows) + " x " + std::to_string(cols) + " " +
                                           type_name(type) + on(dev));
    return row_major(t, what);
}

Mat matrix_or_none(PyObject* o, int64_t rows, int64_t cols, at::ScalarType type, const at::Device& dev, const char* what)
{
    return o == Py_None ? Mat{} : matrix(o, rows, cols, type, dev, what);
}

const at::Tensor& matrix_input(PyObject* o, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != 2) refuse(PyExc_ValueError, what, "expected a matrix");
    return t;
}

const at::Tensor& vector(PyObject* o, int64_t n, const at::Device& dev, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != 1 || t.size(0) != n || t.device() != dev || !t.is_contiguous())
        refuse(PyExc_ValueError, what, "expected a contiguous vector of " + std::to_string(n) + " elements" + on(dev));
    return t;
}

float* vector32(PyObject* o, int64_t n, const at::Device& dev, const char* what)
{
    const at::Tensor& t = vector(o, n, dev, what);
    if (t.scalar_type() != at::kFloat) refuse(PyExc_ValueError, what, "expected fp32");
    return static_cast<float*>(t.data_ptr());
}

// A contiguous scratch buffer of any type.
void* buffer(PyObject* o, const at::Device& dev, const char* what, size_t& bytes)
{
    bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, what);
    if (t.device() != dev || !t.is_contiguous()) refuse(PyExc_ValueError, what, "expected a contiguous buffer" + on(dev));
    bytes = t.nbytes();
    return t.data_ptr();
}

uint8_t* tiles(PyObject* o, int64_t rows, int64_t cols, const at::Device& dev, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != at::kByte || t.device() != dev || !t.is_contiguous() ||
        t.numel() != (rows + 127) / 128 * ((cols + 127) / 128) * 512)
        refuse(PyExc_ValueError, what, "expected the fp4_scale_tiles of a " + std::to_string(rows) + " x " +
                                           std::to_string(cols) + " matrix" + on(dev));
    return static_cast<uint8_t*>(t.data_ptr());
}

// A column-major fp32 scale grid, rows x groups.
Mat grid(PyObject* o, int64_t rows, int64_t groups, const at::Device& dev, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != groups || t.scalar_type() != at::kFloat || t.device() != dev)
        refuse(PyExc_ValueError, what, "expected a " + std::to_string(rows) + " x " + std::to_string(groups) +
                                           " fp32 grid" + on(dev));
    if (t.stride(0) != 1 && rows != 1) refuse(PyExc_ValueError, what, "expected a column-major grid (stride (1, ld))");
    return {t.data_ptr(), groups != 1 ? t.stride(1) : (rows + 3) / 4 * 4};
}

// Packed 4-bit codes: rows x cols / 2 bytes.
const at::Tensor& packed(PyObject* o, const char* what)
{
    const at::Tensor& t = matrix_input(o, what);
    if (t.scalar_type() != at::kByte) refuse(PyExc_TypeError, what, "packed 4-bit codes are uint8");
    return t;
}

// Calls `f(stream)` with dev current, on its current stream, without the
// interpreter's lock.
template <typename F>
PyObject* call(const at::Device& dev, F&& f)
{
    if (!dev.is_cuda()) refuse(PyExc_ValueError, "device", "expected CUDA tensors, got " + dev.str());
    const c10::cuda::CUDAGuard guard(dev);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    fp8bs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f(stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// Runs f, turning refusals and C++ exceptions into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

long integer(PyObject* o, const char* what)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, what, "expected an integer");
    }
    return v;
}

// (bits, rule, x, weight, residual, eps, q, scale, h, rstd, y)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const long bits = integer(a[0], "bits"), rule = integer(a[1], "rule");
        const at::Tensor& x = matrix_input(a[2], "x");
        const int64_t rows = x.size(0), cols = x.size(1);
        const at::ScalarType type = x.scalar_type();
        const at::Device dev = x.device();
        const fp8bs_dtype xt = code(x, "x");
        if ((a[4] == Py_None) != (a[8] == Py_None)) refuse(PyExc_ValueError, "out", "h exactly where there is a residual");
        const Mat mx = row_major(x, "x"), mr = matrix_or_none(a[4], rows, cols, type, dev, "residual"),
                  mh = matrix_or_none(a[8], rows, cols, type, dev, "h"),
                  my = matrix_or_none(a[10], rows, cols, type, dev, "y"),
                  mq = matrix(a[6], rows, cols * bits / 8, at::kByte, dev, "q");
        const at::Tensor& w = vector(a[3], cols, dev, "weight");
        const fp8bs_dtype wt = code(w, "weight");
        const void* wp = w.data_ptr();
        float* rstd = vector32(a[9], rows, dev, "rstd");
        const double e = PyFloat_AsDouble(a[5]);
        if (e == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse(PyExc_TypeError, "eps", "expected a number");
        }
        const float eps = (float)e;
        uint8_t* q = static_cast<uint8_t*>(mq.p);
        if (bits == 8) {
            const Mat ms = grid(a[7], rows, (cols + 127) / 128, dev, "scale_inv");
            return call(dev, [&](cudaStream_t s) {
                return fp8_rmsnorm_quant_1x128(mx.p, mx.ld, mr.p, mr.ld, xt, rows, cols, wp, wt, eps, mh.p, mh.ld, rstd,
                                               my.p, my.ld, q, mq.ld, static_cast<float*>(ms.p), ms.ld,
                                               (fp8bs_scale_rule)rule, s);
            });
        }
        uint8_t* st = tiles(a[7], rows, cols, dev, "scale");
        return call(dev, [&](cudaStream_t s) {
            return fp4_rmsnorm_quant_1x32(mx.p, mx.ld, mr.p, mr.ld, xt, rows, cols, wp, wt, eps, mh.p, mh.ld, rstd, my.p,
                                          my.ld, q, mq.ld, st, s);
        });
    });
}

// (dy, h, weight, rstd, dh, dx, dweight, workspace)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor& h = matrix_input(a[1], "h");
        const int64_t rows = h.size(0), cols = h.size(1);
        const at::ScalarType type = h.scalar_type();
        const at::Device dev = h.device();
        const fp8bs_dtype xt = code(h, "h");
        const Mat mh = row_major(h, "h"), my = matrix(a[0], rows, cols, type, dev, "dy"),
                  mg = matrix_or_none(a[4], rows, cols, type, dev, "dh"), mx = matrix(a[5], rows, cols, type, dev, "dx");
        const at::Tensor& w = vector(a[2], cols, dev, "weight");
        const fp8bs_dtype wt = code(w, "weight");
        const void* wp = w.data_ptr();
        const float* rstd = vector32(a[3], rows, dev, "rstd");
        float* dw = vector32(a[6], cols, dev, "dweight");
        size_t bytes;
        void* ws = buffer(a[7], dev, "workspace", bytes);
        return call(dev, [&](cudaStream_t s) {
            return fp8bs_rmsnorm_backward(my.p, my.ld, mh.p, mh.ld, mg.p, mg.ld, xt, rows, cols, wp, wt, rstd, mx.p, mx.ld,
                                          dw, ws, bytes, s);
        });
    });
}

// (x, transpose, q, scale)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        const at::Tensor& x = matrix_input(a[0], "x");
        const int t = integer(a[1], "transpose_out") != 0;
        const int64_t rows = x.size(0), cols = x.size(1), R = t ? cols : rows, C = t ? rows : cols;
        const at::Device dev = x.device();
        const fp8bs_dtype xt = code(x, "x");
        const Mat mx = row_major(x, "x"), mq = matrix(a[2], R, C / 2, at::kByte, dev, "q");
        uint8_t* st = tiles(a[3], R, C, dev, "scale");
        return call(dev, [&](cudaStream_t s) {
            return fp4_quant_1x32(mx.p, xt, rows, cols, mx.ld, static_cast<uint8_t*>(mq.p), mq.ld, st, t, s);
        });
    });
}

// (q, scale, out)
PyObject* dequant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 3, [&] {
        const at::Tensor& q = packed(a[0], "q");
        const int64_t rows = q.size(0), cols = 2 * q.size(1);
        const at::Device dev = q.device();
        const Mat mq = row_major(q, "q");
        const at::Tensor& o = tensor(a[2], "out");
        const fp8bs_dtype ot = code(o, "out");
        const Mat mo = matrix(a[2], rows, cols, o.scalar_type(), dev, "out");
        const uint8_t* st = tiles(a[1], rows, cols, dev, "scale");
        return call(dev, [&](cudaStream_t s) {
            return fp4_dequant_1x32(static_cast<const uint8_t*>(mq.p), mq.ld, st, rows, cols, mo.p, ot, mo.ld, s);
        });
    });
}

// (A, Bt, scale_a, scale_b, out, workspace)
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const at::Tensor &A = packed(a[0], "A"), &B = packed(a[1], "Bt");
        const int64_t M = A.size(0), N = B.size(0), K = 2 * A.size(1);
        const at::Device dev = A.device();
        if (2 * B.size(1) != K || B.device() != dev) refuse(PyExc_ValueError, "A and Bt", "must share K and the device");
        const Mat ma = row_major(A, "A"), mb = row_major(B, "Bt");
        const at::Tensor& o = tensor(a[4], "out");
        const fp8bs_dtype ot = code(o, "out");
        const Mat mo = matrix(a[4], M, N, o.scalar_type(), dev, "out");
        const uint8_t *sa = tiles(a[2], M, K, dev, "scale_a"), *sb = tiles(a[3], N, K, dev, "scale_b");
        size_t bytes;
        void* ws = buffer(a[5], dev, "workspace", bytes);
        return call(dev, [&](cudaStream_t s) {
            return fp4_scaled_gemm(M, N, K, static_cast<const uint8_t*>(ma.p), ma.ld, static_cast<const uint8_t*>(mb.p),
                                   mb.ld, sa, sb, mo.p, mo.ld, ot, ws, bytes, s);
        });
    });
}

// Makes the CUDA device of that index current, as the calls do (-1: none does).
void make_current(c10::cuda::OptionalCUDAGuard& guard, PyObject* index)
{
    const long i = integer(index, "device");
    if (i >= 0) guard.set_index((c10::DeviceIndex)i);
}

// (M, N, K, device) -> bytes
PyObject* product_workspace(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        c10::cuda::OptionalCUDAGuard guard;
        make_current(guard, a[3]);
        return PyLong_FromSize_t(fp4_scaled_gemm_workspace_size(integer(a[0], "M"), integer(a[1], "N"), integer(a[2], "K")));
    });
}

// (rows, cols, device) -> bytes
PyObject* norm_backward_workspace(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 3, [&] {
        c10::cuda::OptionalCUDAGuard guard;
        make_current(guard, a[2]);
        return PyLong_FromSize_t(fp8bs_rmsnorm_backward_workspace_size(integer(a[0], "rows"), integer(a[1], "cols")));
    });
}

template <typename F>
PyMethodDef method(const char* name, F f)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    static PyMethodDef methods[] = {method("norm", norm), method("norm_backward", norm_backward), method("quant", quant),
                                    method("dequant", dequant), method("product", product),
                                    method("product_workspace", product_workspace),
                                    method("norm_backward_workspace", norm_backward_workspace), {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&def);
}
