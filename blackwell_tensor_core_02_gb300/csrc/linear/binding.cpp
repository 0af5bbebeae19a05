// binding.cpp -- the calls of linear.py, grouped.py and checkpoint.py below their
// keyword handling: checks of the tensors, outputs and workspaces from torch's
// allocator, the current stream, and the C entry points of linear_ops.h, grouped_ops.h
// and checkpoint_ops.h.
//
// The smallest calls (one token) run for two to four microseconds on the GPU, far
// less than the same checks, allocations and conversions take in Python (a layer
// norm of one row: 16.5 us a call with them there).
// Positional arguments only; every value a caller may pass is checked here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "checkpoint_ops.h"
#include "grouped_ops.h"
#include "linear_ops.h"

namespace {

PyObject *g_gemm_error = nullptr;  // the package's GemmError

// A Python exception is set.
struct Refused {};

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... args) {
    PyErr_Format(type, format, args...);
    throw Refused{};
}

void check_status(int64_t rc, const char *where) {
    if (rc >= 0) return;
    PyObject *e = PyObject_CallFunction(g_gemm_error, "Ls", static_cast<long long>(rc), where);
    if (e) {
        PyErr_SetObject(g_gemm_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

bool given(PyObject *o) { return o != Py_None; }

int dtype_code(at::ScalarType t) {
    return t == at::kHalf ? LINEAR_F16 : t == at::kBFloat16 ? LINEAR_BF16 : t == at::kFloat ? LINEAR_F32 : -1;
}

int dtype_of(const at::Tensor &t, const char *name) {
    const int code = dtype_code(t.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "%s must be float16, bfloat16 or float32", name);
    return code;
}

at::ScalarType dtype_arg(PyObject *o, const char *name) {
    if (!THPDtype_Check(o) || dtype_code(reinterpret_cast<THPDtype *>(o)->scalar_type) < 0) {
        refuse(PyExc_TypeError, "%s must be float16, bfloat16 or float32", name);
    }
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

struct Rows {
    int64_t rows, cols, step;
};

// A tensor whose last axis is contiguous and whose other axes step evenly.
Rows rows_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
    const int64_t dims = t.dim();
    if (dims == 0) refuse(PyExc_ValueError, "%s must have at least one axis", name);
    Rows r{1, t.size(dims - 1), t.size(dims - 1)};
    if (r.cols > 1 && t.stride(dims - 1) != 1) refuse(PyExc_ValueError, "%s: its last axis must be contiguous", name);
    bool first = true;
    int64_t next = 0;  // the stride of the axis above, if the rows step evenly
    for (int64_t i = dims - 2; i >= 0; --i) {
        const int64_t n = t.size(i);
        r.rows *= n;
        if (n <= 1) continue;
        if (first) {
            r.step = t.stride(i);
            first = false;
        } else if (t.stride(i) != next && t.numel() > 0) {
            refuse(PyExc_ValueError, "%s: its rows do not step evenly; make it contiguous", name);
        }
        next = t.stride(i) * n;
    }
    return r;
}

void same_kind(const at::Tensor &t, const at::Tensor &x, const char *name, const char *of) {
    if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes() || t.device() != x.device()) {
        refuse(PyExc_ValueError, "%s must have the dtype, shape and device of %s", name, of);
    }
}

// A vector of the last axis, x's dtype or float32.
const void *weights(const at::Tensor &t, const at::Tensor &x, int64_t cols, const char *name) {
    if (t.dim() != 1 || t.size(0) != cols || (cols > 1 && t.stride(0) != 1) || t.device() != x.device()) {
        refuse(PyExc_ValueError, "%s must be a contiguous vector of the last axis, on x's device", name);
    }
    if (t.scalar_type() != x.scalar_type() && t.scalar_type() != at::kFloat) {
        refuse(PyExc_TypeError, "%s must have x's dtype or float32", name);
    }
    return t.data_ptr();
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

void *stream_of(const at::Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// Memory for the length of a call, from torch's allocator and in the stream's order, without the
// tensor around it.
struct Workspace {
    void *p = nullptr;
    Workspace() = default;
    Workspace(const Workspace &) = delete;
    Workspace &operator=(const Workspace &) = delete;
    ~Workspace() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
    void *take(int64_t bytes, void *stream) {
        if (bytes > 0) {
            p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(static_cast<size_t>(bytes), static_cast<cudaStream_t>(stream));
        }
        return p;
    }
};

PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) throw Refused{};
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

// ------------------------------------------------------------- layer norm --

PyObject *norm(PyObject *const *args, Py_ssize_t n) {  // x, weight, bias, eps, out
    count(n, 5);
    const at::Tensor &x = tensor(args[0], "x");
    const int code = dtype_of(x, "x");
    const Rows r = rows_of(x, "x");
    if (r.cols == 0) refuse(PyExc_ValueError, "x: rows of no elements have no norm");
    int wcode = code;
    const void *w = nullptr, *b = nullptr;
    if (given(args[1])) {
        const at::Tensor &t = tensor(args[1], "weight");
        w = weights(t, x, r.cols, "weight");
        wcode = dtype_code(t.scalar_type());
    }
    if (given(args[2])) {
        const at::Tensor &t = tensor(args[2], "bias");
        b = weights(t, x, r.cols, "bias");
        const int bcode = dtype_code(t.scalar_type());
        if (w && bcode != wcode) refuse(PyExc_TypeError, "weight and bias must have one dtype");
        wcode = bcode;
    }
    const double eps = PyFloat_AsDouble(args[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{};
    const c10::cuda::CUDAGuard guard(x.device());
    Rows yr{r.rows, r.cols, r.cols};
    at::Tensor y;
    if (given(args[4])) {
        y = tensor(args[4], "out");
        same_kind(y, x, "out", "x");
        yr = rows_of(y, "out");
    } else {
        y = empty(x.sizes(), x.scalar_type(), x);
    }
    const at::IntArrayRef lead = x.sizes().slice(0, static_cast<size_t>(x.dim() - 1));
    at::Tensor mean = empty(lead, at::kFloat, x), rstd = empty(lead, at::kFloat, x);
    check_status(layer_norm_forward(x.data_ptr(), r.step, w, b, y.data_ptr(), yr.step, mean.data_ptr<float>(),
                                    rstd.data_ptr<float>(), r.rows, r.cols, static_cast<float>(eps), code, wcode,
                                    stream_of(x)),
                 "layer_norm");
    return tuple_of({y, mean, rstd});
}

const float *statistic(const at::Tensor &t, const at::Tensor &x, int64_t rows, const char *name) {
    if (t.scalar_type() != at::kFloat || t.numel() != rows || !t.is_contiguous() || t.device() != x.device()) {
        refuse(PyExc_ValueError, "%s must be contiguous float32, one for each row of x, on its device", name);
    }
    return t.data_ptr<float>();
}

PyObject *norm_backward(PyObject *const *args, Py_ssize_t n) {  // dy, x, weight, mean, rstd, dx, grad_dtype
    count(n, 7);
    const at::Tensor &dy = tensor(args[0], "dy"), &x = tensor(args[1], "x");
    const int code = dtype_of(x, "x");
    const Rows r = rows_of(x, "x");
    if (r.cols == 0) refuse(PyExc_ValueError, "x: rows of no elements have no norm");
    same_kind(dy, x, "dy", "x");
    const Rows dr = rows_of(dy, "dy");
    const float *mean = statistic(tensor(args[3], "mean"), x, r.rows, "mean");
    const float *rstd = statistic(tensor(args[4], "rstd"), x, r.rows, "rstd");
    const void *w = nullptr;
    at::ScalarType wtype = x.scalar_type();
    if (given(args[2])) {
        const at::Tensor &t = tensor(args[2], "weight");
        w = weights(t, x, r.cols, "weight");
        wtype = t.scalar_type();
    }
    const bool parameters = w || given(args[6]);  // their gradients are wanted
    if (given(args[6])) {
        const at::ScalarType want = dtype_arg(args[6], "grad_dtype");
        if (w ? want != wtype : (want != wtype && want != at::kFloat)) {
            refuse(PyExc_TypeError, "grad_dtype must be weight's dtype or, without a weight, x's or float32");
        }
        wtype = want;
    }
    const c10::cuda::CUDAGuard guard(x.device());
    Rows gr{r.rows, r.cols, r.cols};
    at::Tensor dx, dweight, dbias, space;
    if (given(args[5])) {
        dx = tensor(args[5], "dx");
        same_kind(dx, x, "dx", "x");
        gr = rows_of(dx, "dx");
    } else {
        dx = empty(x.sizes(), x.scalar_type(), x);
    }
    int64_t need = 0;
    if (parameters) {
        dweight = empty({r.cols}, wtype, x);
        dbias = empty({r.cols}, wtype, x);
        need = layer_norm_backward_workspace_size(r.rows, r.cols);
        check_status(need, "layer_norm_backward");
        space = empty({need}, at::kByte, x);
    }
    check_status(layer_norm_backward(dy.data_ptr(), dr.step, x.data_ptr(), r.step, w, mean, rstd, dx.data_ptr(), gr.step,
                                     parameters ? dweight.data_ptr() : nullptr, parameters ? dbias.data_ptr() : nullptr,
                                     r.rows, r.cols, code, dtype_code(wtype), parameters ? space.data_ptr() : nullptr, need,
                                     stream_of(x)),
                 "layer_norm_backward");
    return tuple_of({dx, dweight, dbias});
}

// -------------------------------------------------------------------- fp4 --

long whole(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s must be an int", name);
    }
    return v;
}

struct Format {
    int code;
    int exponent;
};

Format format_of(PyObject *name, PyObject *exponent) {
    Format f{-1, 0};
    if (PyUnicode_Check(name)) {
        f.code = PyUnicode_CompareWithASCIIString(name, "mx") == 0   ? FP4_MX
                 : PyUnicode_CompareWithASCIIString(name, "nv") == 0 ? FP4_NV
                                                                     : -1;
    }
    if (f.code < 0) refuse(PyExc_ValueError, "format must be \"mx\" or \"nv\", not %R", name);
    const long e = whole(exponent, "exponent");
    if (e < -100 || e > 100 || (e != 0 && f.code == FP4_MX)) {
        refuse(PyExc_ValueError, "exponent must be in [-100, 100], and 0 for format \"mx\"");
    }
    f.exponent = static_cast<int>(e);
    return f;
}

struct Sizes {
    int64_t data[2], scales[5];
};

Sizes sizes_of(int64_t rows, int64_t cols, int code) {
    const int64_t units = (cols + 31) / 32, per = code == FP4_NV ? 2 : 4;
    return {{rows, units * 16}, {(rows + 127) / 128, (units + per - 1) / per, 32, 4, 4}};
}

// The parts of an Fp4Tensor (a tuple: data, scales, cols, format, exponent) that fit together.
struct Fp4 {
    const at::Tensor *data, *scales;
    int64_t rows, cols;
    Format format;
};

Fp4 fp4_of(PyObject *o, const char *name) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) refuse(PyExc_TypeError, "%s must be an Fp4Tensor", name);
    Fp4 q;
    q.data = &tensor(PyTuple_GET_ITEM(o, 0), "data");
    q.scales = &tensor(PyTuple_GET_ITEM(o, 1), "scales");
    q.cols = whole(PyTuple_GET_ITEM(o, 2), "cols");
    q.format = format_of(PyTuple_GET_ITEM(o, 3), PyTuple_GET_ITEM(o, 4));
    if (q.data->dim() != 2 || q.cols < 0) refuse(PyExc_ValueError, "%s: data must be [rows, bytes] and cols not negative", name);
    q.rows = q.data->size(0);
    const Sizes want = sizes_of(q.rows, q.cols, q.format.code);
    if (q.data->sizes() != at::IntArrayRef(want.data, 2) || q.scales->sizes() != at::IntArrayRef(want.scales, 5)) {
        refuse(PyExc_ValueError,
               "%s: data of %lld x %lld in its format is [%lld, %lld], and scales [%lld, %lld, 32, 4, 4]", name,
               static_cast<long long>(q.rows), static_cast<long long>(q.cols), static_cast<long long>(want.data[0]),
               static_cast<long long>(want.data[1]), static_cast<long long>(want.scales[0]),
               static_cast<long long>(want.scales[1]));
    }
    if (q.data->scalar_type() != at::kByte || q.scales->scalar_type() != at::kByte) {
        refuse(PyExc_TypeError, "%s: data and scales must be uint8", name);
    }
    if (!q.data->is_cuda() || q.scales->device() != q.data->device() || !q.data->is_contiguous() ||
        !q.scales->is_contiguous()) {
        refuse(PyExc_ValueError, "%s: data and scales must be contiguous tensors of one CUDA device", name);
    }
    return q;
}

PyObject *quantize(PyObject *const *args, Py_ssize_t n) {  // x, format, exponent, out -> (data, scales)
    count(n, 4);
    const at::Tensor &x = tensor(args[0], "x");
    const int code = dtype_of(x, "x");
    const Format f = format_of(args[1], args[2]);
    if (x.dim() != 2) refuse(PyExc_ValueError, "x must be a matrix");
    const Rows r = rows_of(x, "x");
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor data, scales;
    if (given(args[3])) {
        const Fp4 q = fp4_of(args[3], "out");
        if (q.rows != r.rows || q.cols != r.cols || q.format.code != f.code || q.format.exponent != f.exponent ||
            q.data->device() != x.device()) {
            refuse(PyExc_ValueError, "out must have x's shape and device, and the format and exponent asked for");
        }
        data = *q.data;
        scales = *q.scales;
    } else {
        const Sizes s = sizes_of(r.rows, r.cols, f.code);
        data = empty(at::IntArrayRef(s.data, 2), at::kByte, x);
        scales = empty(at::IntArrayRef(s.scales, 5), at::kByte, x);
    }
    check_status(fp4_quantize(x.data_ptr(), r.step, r.rows, r.cols, code, f.code, f.exponent, data.data_ptr(),
                              scales.data_ptr(), stream_of(x)),
                 "quantize_fp4");
    return tuple_of({data, scales});
}

PyObject *dequantize(PyObject *const *args, Py_ssize_t n) {  // q, dtype, out
    count(n, 3);
    const Fp4 q = fp4_of(args[0], "q");
    const c10::cuda::CUDAGuard guard(q.data->device());
    at::Tensor y;
    int64_t step = q.cols;
    if (given(args[2])) {
        y = tensor(args[2], "out");
        if (y.dim() != 2 || y.size(0) != q.rows || y.size(1) != q.cols || y.device() != q.data->device()) {
            refuse(PyExc_ValueError, "out must have q's rows and columns, on its device");
        }
        step = rows_of(y, "out").step;
    } else {
        y = empty({q.rows, q.cols}, given(args[1]) ? dtype_arg(args[1], "dtype") : at::kFloat, *q.data);
    }
    check_status(fp4_dequantize(q.data->data_ptr(), q.scales->data_ptr(), q.rows, q.cols, q.format.code,
                                q.format.exponent, y.data_ptr(), step, dtype_of(y, "out"), stream_of(y)),
                 "dequantize_fp4");
    return THPVariable_Wrap(y);
}

PyObject *product(PyObject *const *args, Py_ssize_t n) {  // A, B, D, dtype, alpha, address of the options or 0
    count(n, 6);
    const Fp4 a = fp4_of(args[0], "A"), b = fp4_of(args[1], "B");
    if (a.format.code != b.format.code) refuse(PyExc_ValueError, "A and B must have one format");
    if (a.cols != b.cols) {
        refuse(PyExc_ValueError, "expected A (M x K) and B (N x K), got %lld x %lld and %lld x %lld",
               static_cast<long long>(a.rows), static_cast<long long>(a.cols), static_cast<long long>(b.rows),
               static_cast<long long>(b.cols));
    }
    if (a.data->device() != b.data->device()) refuse(PyExc_ValueError, "A and B must be on one device");
    double alpha = PyFloat_AsDouble(args[4]);
    if (alpha == -1.0 && PyErr_Occurred()) throw Refused{};
    const void *options = PyLong_AsVoidPtr(args[5]);
    if (!options && PyErr_Occurred()) throw Refused{};
    gemm_fp4_options o = {};
    if (options) o = *static_cast<const gemm_fp4_options *>(options);
    if (a.format.code == FP4_NV) {
        // 24 bits of alpha, and its power of two with the matrices' (past 700 either way the
        // result is an infinity or 0; an exponent of the options' own that is out of range
        // stays so)
        int e = 0;
        alpha = std::frexp(alpha, &e);
        const int64_t sum = static_cast<int64_t>(o.exponent) + std::max(-700, std::min(700, e)) + a.format.exponent +
                            b.format.exponent;
        o.exponent = static_cast<int32_t>(std::max<int64_t>(-2000, std::min<int64_t>(2000, sum)));
    } else if (std::isfinite(alpha) && !std::isfinite(static_cast<float>(alpha))) {
        refuse(PyExc_ValueError, "alpha must be in float32's range");
    }
    const c10::cuda::CUDAGuard guard(a.data->device());
    at::Tensor d;
    if (given(args[2])) {
        d = tensor(args[2], "D");
        if (d.dim() != 2 || d.size(0) != a.rows || d.size(1) != b.rows || !d.is_contiguous() ||
            d.device() != a.data->device()) {
            refuse(PyExc_ValueError, "D must be a contiguous %lld x %lld matrix on A's device",
                   static_cast<long long>(a.rows), static_cast<long long>(b.rows));
        }
    } else {
        d = empty({a.rows, b.rows}, given(args[3]) ? dtype_arg(args[3], "dtype") : at::kHalf, *a.data);
    }
    check_status(gemm_fp4_nt(a.data->data_ptr(), a.scales->data_ptr(), b.data->data_ptr(), b.scales->data_ptr(),
                             d.data_ptr(), a.rows, b.rows, a.cols, a.format.code, dtype_of(d, "D"),
                             static_cast<float>(alpha), stream_of(d), &o),
                 "gemm_fp4_nt");
    return THPVariable_Wrap(d);
}

// ---------------------------------------------------------------- grouped --

int half_type(const at::Tensor &t, const char *name) {
    const int code = dtype_code(t.scalar_type());
    if (code != LINEAR_F16 && code != LINEAR_BF16) refuse(PyExc_TypeError, "%s must be float16 or bfloat16", name);
    return code;
}

// A tensor of `dims` axes, the last contiguous, of like's type on its device.
void operand(const at::Tensor &t, const char *name, int64_t dims, const at::Tensor &like) {
    if (t.scalar_type() != like.scalar_type()) refuse(PyExc_TypeError, "%s must have the first operand's dtype", name);
    if (!t.is_cuda() || t.device() != like.device()) {
        refuse(PyExc_ValueError, "%s must be a CUDA tensor, all on one device", name);
    }
    if (t.dim() != dims) refuse(PyExc_ValueError, "%s must have %lld axes", name, static_cast<long long>(dims));
    if (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1) {
        refuse(PyExc_ValueError, "%s: its last axis must be contiguous", name);
    }
}

// Whole numbers in device memory; whether they are 64-bit.
int whole_numbers(const at::Tensor &t, const char *name, int64_t count, const at::Tensor &like) {
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong) refuse(PyExc_TypeError, "%s must be int32 or int64", name);
    if (t.device() != like.device() || t.dim() != 1 || t.size(0) != count || !t.is_contiguous()) {
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %lld on the operands' device", name,
               static_cast<long long>(count));
    }
    return t.scalar_type() == at::kLong;
}

const grouped_options *grouped_opts(PyObject *o) {
    const void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused{};
    return static_cast<const grouped_options *>(p);
}

// The rows of a result, `like`'s or given, and whether they are new.
at::Tensor grouped_rows(PyObject *o, const char *name, int64_t rows, int64_t cols, const at::Tensor &like, bool *made) {
    *made = !given(o);
    if (*made) return empty({rows, cols}, like.scalar_type(), like);
    const at::Tensor &t = tensor(o, name);
    operand(t, name, 2, like);
    if (t.size(0) != rows || t.size(1) != cols) {
        refuse(PyExc_ValueError, "%s must be %lld x %lld", name, static_cast<long long>(rows), static_cast<long long>(cols));
    }
    return t;
}

// The two products whose results have the ragged rows: NT (x is A, the result D) and NN (x is dD, the result dA).
template <bool NT>
PyObject *grouped_rows_product(PyObject *const *args, Py_ssize_t n) {  // x, B, offsets, out, address of the options or 0
    count(n, 5);
    const at::Tensor &x = tensor(args[0], NT ? "A" : "dD"), &B = tensor(args[1], "B"), &offsets = tensor(args[2], "offsets");
    const int code = half_type(x, NT ? "A" : "dD");
    operand(x, NT ? "A" : "dD", 2, x);
    operand(B, "B", 3, x);
    const int64_t rows = x.size(0), groups = B.size(0), N = B.size(1), K = B.size(2);
    if (x.size(1) != (NT ? K : N)) {
        refuse(PyExc_ValueError, NT ? "expected A (rows x K) and B (groups x N x K), got rows of %lld and of %lld"
                                    : "expected dD (rows x N) and B (groups x N x K), got rows of %lld and N %lld",
               static_cast<long long>(x.size(1)), static_cast<long long>(NT ? K : N));
    }
    const int wide = whole_numbers(offsets, "offsets", groups + 1, x);
    const grouped_options *opts = grouped_opts(args[4]);
    const c10::cuda::CUDAGuard guard(x.device());
    bool made = false;
    at::Tensor out = grouped_rows(args[3], NT ? "D" : "dA", rows, NT ? N : K, x, &made);
    const auto call = NT ? grouped_gemm_nt : grouped_gemm_nn;
    check_status(call(x.data_ptr(), x.stride(0), B.data_ptr(), B.stride(1), B.stride(0), offsets.data_ptr(), wide,
                      out.data_ptr(), out.stride(0), rows, groups, N, K, code, made, stream_of(x), opts),
                 NT ? "grouped_gemm_nt" : "grouped_gemm_nn");
    return THPVariable_Wrap(out);
}

PyObject *grouped_matrices(PyObject *const *args, Py_ssize_t n) {  // dD, A, offsets, dB, address of the options or 0
    count(n, 5);
    const at::Tensor &dD = tensor(args[0], "dD"), &A = tensor(args[1], "A"), &offsets = tensor(args[2], "offsets");
    const int code = half_type(dD, "dD");
    operand(dD, "dD", 2, dD);
    operand(A, "A", 2, dD);
    const int64_t rows = dD.size(0), N = dD.size(1), K = A.size(1);
    if (A.size(0) != rows) refuse(PyExc_ValueError, "expected dD (rows x N) and A (rows x K) of the same rows");
    const int64_t groups = offsets.numel() - 1;
    if (groups < 0) refuse(PyExc_ValueError, "offsets must be a vector of at least one");
    const int wide = whole_numbers(offsets, "offsets", groups + 1, dD);
    const grouped_options *opts = grouped_opts(args[4]);
    const c10::cuda::CUDAGuard guard(dD.device());
    at::Tensor dB;
    if (given(args[3])) {
        dB = tensor(args[3], "dB");
        operand(dB, "dB", 3, dD);
        if (dB.size(0) != groups || dB.size(1) != N || dB.size(2) != K) {
            refuse(PyExc_ValueError, "dB must be %lld x %lld x %lld", static_cast<long long>(groups),
                   static_cast<long long>(N), static_cast<long long>(K));
        }
    } else {
        dB = empty({groups, N, K}, dD.scalar_type(), dD);
    }
    check_status(grouped_gemm_tn(dD.data_ptr(), dD.stride(0), A.data_ptr(), A.stride(0), offsets.data_ptr(), wide,
                                 dB.data_ptr(), dB.stride(1), dB.stride(0), rows, groups, N, K, code, stream_of(dD), opts),
                 "grouped_gemm_tn");
    return THPVariable_Wrap(dB);
}

PyObject *lora(PyObject *const *args, Py_ssize_t n) {  // x, W, down, up, offsets, adapters, D, scales, options or 0
    count(n, 9);
    const at::Tensor &x = tensor(args[0], "x"), &W = tensor(args[1], "W"), &down = tensor(args[2], "down"),
                     &up = tensor(args[3], "up"), &offsets = tensor(args[4], "offsets"), &adapters = tensor(args[5], "adapters");
    const int code = half_type(x, "x");
    operand(x, "x", 2, x);
    operand(W, "W", 2, x);
    operand(down, "down", 3, x);
    operand(up, "up", 3, x);
    const int64_t rows = x.size(0), K = x.size(1), N = W.size(0), many = down.size(0), rank = down.size(1);
    if (W.size(1) != K || down.size(2) != K || up.size(0) != many || up.size(1) != N || up.size(2) != rank) {
        refuse(PyExc_ValueError,
               "expected x (rows x K), W (N x K), down (adapters x rank x K) and up (adapters x N x rank)");
    }
    if (adapters.scalar_type() != at::kInt) refuse(PyExc_TypeError, "adapters must be int32");
    const int64_t requests = adapters.numel();
    whole_numbers(adapters, "adapters", requests, x);
    const int wide = whole_numbers(offsets, "offsets", requests + 1, x);
    const float *scales = nullptr;
    if (given(args[7])) {
        const at::Tensor &t = tensor(args[7], "scales");
        if (t.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "scales must be float32");
        if (t.device() != x.device() || t.dim() != 1 || t.size(0) != many || !t.is_contiguous()) {
            refuse(PyExc_ValueError, "scales must be a contiguous vector of one for each adapter, on x's device");
        }
        scales = t.data_ptr<float>();
    }
    const grouped_options *opts = grouped_opts(args[8]);
    const c10::cuda::CUDAGuard guard(x.device());
    bool made = false;
    at::Tensor D = grouped_rows(args[6], "D", rows, N, x, &made);
    const int64_t need = gemm_lora_workspace_size(rows, rank);
    check_status(need, "gemm_lora_nt");
    Workspace space;
    void *workspace = space.take(need, stream_of(x));
    check_status(gemm_lora_nt(x.data_ptr(), x.stride(0), W.data_ptr(), W.stride(0), down.data_ptr(), down.stride(1),
                              down.stride(0), up.data_ptr(), up.stride(1), up.stride(0), scales, offsets.data_ptr(), wide,
                              adapters.data_ptr<int32_t>(), D.data_ptr(), D.stride(0), rows, requests, many, N, K, rank, code,
                              workspace, need, stream_of(x), opts),
                 "gemm_lora_nt");
    return THPVariable_Wrap(D);
}

// ------------------------------------------------------------ checkpoints --

// The parts of an Fp8Rows (a tuple: codes, scales) that fit together.
struct Fp8 {
    const at::Tensor *codes, *scales;
    int64_t rows, cols;
};

Fp8 fp8_of(PyObject *o, const char *name) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse(PyExc_TypeError, "%s must be an Fp8Rows", name);
    Fp8 q;
    q.codes = &tensor(PyTuple_GET_ITEM(o, 0), "codes");
    q.scales = &tensor(PyTuple_GET_ITEM(o, 1), "scales");
    if (q.codes->scalar_type() != at::kFloat8_e4m3fn || q.scales->scalar_type() != at::kByte) {
        refuse(PyExc_TypeError, "%s: codes must be float8_e4m3fn and scales uint8", name);
    }
    const int64_t dims = q.codes->dim();
    if (dims == 0) refuse(PyExc_ValueError, "%s: codes must have at least one axis", name);
    q.cols = q.codes->size(dims - 1);
    q.rows = 1;
    bool fits = q.scales->dim() == dims && q.scales->size(dims - 1) == (q.cols + 31) / 32;
    for (int64_t i = 0; i < dims - 1; ++i) {
        q.rows *= q.codes->size(i);
        fits = fits && q.scales->size(i) == q.codes->size(i);
    }
    if (!fits) refuse(PyExc_ValueError, "%s: scales must be one for each 32 codes of a row", name);
    if (!q.codes->is_cuda() || q.scales->device() != q.codes->device() || !q.codes->is_contiguous() ||
        !q.scales->is_contiguous()) {
        refuse(PyExc_ValueError, "%s: codes and scales must be contiguous tensors of one CUDA device", name);
    }
    if (q.cols == 0) refuse(PyExc_ValueError, "%s: rows of no elements have no norm", name);
    return q;
}

at::DimVector blocks_of(at::IntArrayRef sizes) {
    at::DimVector s(sizes.begin(), sizes.end());
    s.back() = (s.back() + 31) / 32;
    return s;
}

// weight and bias (either may be None), vectors of `cols` of one dtype, `type` or float32, on like's device.
struct Affine {
    const void *weight = nullptr, *bias = nullptr;
    at::ScalarType type;
};

Affine affine_of(PyObject *weight, PyObject *bias, int64_t cols, at::ScalarType type, const at::Tensor &like) {
    Affine a;
    a.type = type;
    bool first = true;
    for (int i = 0; i < 2; ++i) {
        PyObject *o = i == 0 ? weight : bias;
        if (!given(o)) continue;
        const char *name = i == 0 ? "weight" : "bias";
        const at::Tensor &t = tensor(o, name);
        if (t.dim() != 1 || t.size(0) != cols || (cols > 1 && t.stride(0) != 1) || t.device() != like.device()) {
            refuse(PyExc_ValueError, "%s must be a contiguous vector of the last axis, on the rows' device", name);
        }
        if (t.scalar_type() != type && t.scalar_type() != at::kFloat) {
            refuse(PyExc_TypeError, "%s must have the rows' dtype or float32", name);
        }
        if (!first && t.scalar_type() != a.type) refuse(PyExc_TypeError, "weight and bias must have one dtype");
        a.type = t.scalar_type();
        first = false;
        (i == 0 ? a.weight : a.bias) = t.data_ptr();
    }
    return a;
}

PyObject *keep(PyObject *const *args, Py_ssize_t n) {  // x, weight, bias, eps, out -> (y, codes, scales, rstd)
    count(n, 5);
    const at::Tensor &x = tensor(args[0], "x");
    const int code = dtype_of(x, "x");
    const Rows r = rows_of(x, "x");
    if (r.cols == 0) refuse(PyExc_ValueError, "x: rows of no elements have no norm");
    const Affine a = affine_of(args[1], args[2], r.cols, x.scalar_type(), x);
    const double eps = PyFloat_AsDouble(args[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{};
    const c10::cuda::CUDAGuard guard(x.device());
    Rows yr{r.rows, r.cols, r.cols};
    at::Tensor y;
    if (given(args[4])) {
        y = tensor(args[4], "out");
        same_kind(y, x, "out", "x");
        yr = rows_of(y, "out");
    } else {
        y = empty(x.sizes(), x.scalar_type(), x);
    }
    at::Tensor codes = empty(x.sizes(), at::kFloat8_e4m3fn, x), scales = empty(blocks_of(x.sizes()), at::kByte, x);
    at::Tensor rstd = empty(x.sizes().slice(0, static_cast<size_t>(x.dim() - 1)), at::kFloat, x);
    check_status(norm_checkpoint_forward(x.data_ptr(), r.step, a.weight, a.bias, y.data_ptr(), yr.step, codes.data_ptr(),
                                         scales.data_ptr(), rstd.data_ptr<float>(), r.rows, r.cols, static_cast<float>(eps),
                                         code, dtype_code(a.type), stream_of(x)),
                 "layer_norm_checkpoint");
    return tuple_of({y, codes, scales, rstd});
}

PyObject *restore(PyObject *const *args, Py_ssize_t n) {  // kept, weight, bias, dtype, out
    count(n, 5);
    const Fp8 q = fp8_of(args[0], "kept");
    const at::Tensor &codes = *q.codes;
    const c10::cuda::CUDAGuard guard(codes.device());
    at::Tensor y;
    int64_t step = q.cols;
    if (given(args[4])) {
        y = tensor(args[4], "out");
        dtype_of(y, "out");
        if (y.sizes() != codes.sizes() || y.device() != codes.device()) {
            refuse(PyExc_ValueError, "out must have the kept rows' shape and device");
        }
        if (given(args[3]) && dtype_arg(args[3], "dtype") != y.scalar_type()) {
            refuse(PyExc_TypeError, "dtype must be out's");
        }
        step = rows_of(y, "out").step;
    } else {
        at::ScalarType type = at::kFloat;
        if (given(args[3])) {
            type = dtype_arg(args[3], "dtype");
        } else if (given(args[1]) || given(args[2])) {  // the weights'
            const at::Tensor &t = given(args[1]) ? tensor(args[1], "weight") : tensor(args[2], "bias");
            dtype_of(t, given(args[1]) ? "weight" : "bias");
            type = t.scalar_type();
        }
        y = empty(codes.sizes(), type, codes);
    }
    const Affine a = affine_of(args[1], args[2], q.cols, y.scalar_type(), codes);
    check_status(norm_checkpoint_restore(codes.data_ptr(), q.scales->data_ptr(), a.weight, a.bias, y.data_ptr(), step, q.rows,
                                         q.cols, dtype_code(y.scalar_type()), dtype_code(a.type), stream_of(y)),
                 "layer_norm_restore");
    return THPVariable_Wrap(y);
}

PyObject *keep_backward(PyObject *const *args, Py_ssize_t n) {  // dy, kept, weight, rstd, dx, grad_dtype
    count(n, 6);
    const at::Tensor &dy = tensor(args[0], "dy");
    const int code = dtype_of(dy, "dy");
    const Rows r = rows_of(dy, "dy");
    const Fp8 q = fp8_of(args[1], "kept");
    if (q.codes->sizes() != dy.sizes() || q.codes->device() != dy.device()) {
        refuse(PyExc_ValueError, "kept must have dy's shape and device");
    }
    const float *rstd = statistic(tensor(args[3], "rstd"), dy, r.rows, "rstd");
    const Affine a = affine_of(args[2], Py_None, r.cols, dy.scalar_type(), dy);
    at::ScalarType wtype = a.type;
    const bool parameters = a.weight || given(args[5]);  // their gradients are wanted
    if (given(args[5])) {
        const at::ScalarType want = dtype_arg(args[5], "grad_dtype");
        if (a.weight ? want != wtype : (want != wtype && want != at::kFloat)) {
            refuse(PyExc_TypeError, "grad_dtype must be weight's dtype or, without a weight, dy's or float32");
        }
        wtype = want;
    }
    const c10::cuda::CUDAGuard guard(dy.device());
    Rows gr{r.rows, r.cols, r.cols};
    at::Tensor dx, dweight, dbias;
    Workspace space;
    if (given(args[4])) {
        dx = tensor(args[4], "dx");
        same_kind(dx, dy, "dx", "dy");
        gr = rows_of(dx, "dx");
    } else {
        dx = empty(dy.sizes(), dy.scalar_type(), dy);
    }
    int64_t need = 0;
    if (parameters) {
        dweight = empty({r.cols}, wtype, dy);
        dbias = empty({r.cols}, wtype, dy);
        need = layer_norm_backward_workspace_size(r.rows, r.cols);
        check_status(need, "layer_norm_backward_checkpoint");
    }
    check_status(norm_checkpoint_backward(dy.data_ptr(), r.step, q.codes->data_ptr(), q.scales->data_ptr(), a.weight, rstd,
                                          dx.data_ptr(), gr.step, parameters ? dweight.data_ptr() : nullptr,
                                          parameters ? dbias.data_ptr() : nullptr, r.rows, r.cols, code, dtype_code(wtype),
                                          space.take(need, stream_of(dy)), need, stream_of(dy)),
                 "layer_norm_backward_checkpoint");
    return tuple_of({dx, dweight, dbias});
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XDECREF(g_gemm_error);
    g_gemm_error = Py_NewRef(cls);
    Py_RETURN_NONE;
}

#define LINEAR_METHOD(name, fn) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<fn>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {LINEAR_METHOD("layer_norm", norm),
                           LINEAR_METHOD("layer_norm_backward", norm_backward),
                           LINEAR_METHOD("quantize_fp4", quantize),
                           LINEAR_METHOD("dequantize_fp4", dequantize),
                           LINEAR_METHOD("gemm_fp4_nt", product),
                           LINEAR_METHOD("grouped_gemm_nt", grouped_rows_product<true>),
                           LINEAR_METHOD("grouped_gemm_nn", grouped_rows_product<false>),
                           LINEAR_METHOD("grouped_gemm_tn", grouped_matrices),
                           LINEAR_METHOD("gemm_lora_nt", lora),
                           LINEAR_METHOD("layer_norm_checkpoint", keep),
                           LINEAR_METHOD("layer_norm_restore", restore),
                           LINEAR_METHOD("layer_norm_backward_checkpoint", keep_backward),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_linear_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__linear_binding() { return PyModule_Create(&g_module); }
