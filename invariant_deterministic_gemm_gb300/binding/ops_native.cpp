// The native half of _ops.py and _attn.py: argument marshalling of the
// mixture-of-experts and attention operators. Each function reads its tensors'
// types, shapes, strides and pointers, allocates the outputs with PyTorch's
// allocator and calls the C function of det_ops.h or det_attn.h on the current
// stream; all arithmetic is the library's. A decode-sized call is bound by this work: through ctypes it
// took 11 to 18 us of host time, most of it Python attribute look-ups and
// argument conversions.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <string>

#include "det_attn.h"
#include "det_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;
constexpr ScalarType kBF16 = ScalarType::BFloat16, kF32 = ScalarType::Float, kI32 = ScalarType::Int, kI64 = ScalarType::Long,
                     kE4M3 = ScalarType::Float8_e4m3fn;
constexpr int64_t kBlock = DET_FP8_BLOCK;

// Thrown once a Python error has been set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *format, ...)
{
    va_list v;
    va_start(v, format);
    PyErr_FormatV(type, format, v);
    va_end(v);
    throw Raised{};
}

const char *type_name(ScalarType t)
{
    switch (t) {
    case kBF16: return "torch.bfloat16";
    case kF32: return "torch.float32";
    case kI32: return "torch.int32";
    case kI64: return "torch.int64";
    case kE4M3: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
    }
}

std::string shape_of(const Tensor &t)
{
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}

// ---- arguments

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

const Tensor &cuda_tensor(PyObject *o, const char *name, ScalarType dtype)
{
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != dtype)
        raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(dtype), type_name(t.scalar_type()));
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return t;
}

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, "%s must be an integer", name);
    }
    return v;
}

int small(PyObject *o, const char *name)
{
    return static_cast<int>(std::clamp<int64_t>(integer(o, name), INT32_MIN, INT32_MAX));
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

float real(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, "%s must be a number", name);
    }
    return static_cast<float>(v);
}

// The CUDA tensors among a call's arguments lie on the device that the work is
// enqueued on, the current one: a kernel would follow another device's addresses,
// in no order with that device's streams.
thread_local c10::DeviceIndex g_device = 0;      // the current device of this call

void on_current_device(PyObject *const *a, Py_ssize_t n)
{
    const Tensor *first = nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        // (asking of a plain number whether it is a tensor takes a tenth of a microsecond)
        PyTypeObject *type = Py_TYPE(a[i]);
        if (type == &PyLong_Type || type == &PyBool_Type || type == &PyFloat_Type || a[i] == Py_None || !THPVariable_Check(a[i])) continue;
        const Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda()) continue;
        if (!first) first = &t;
        else if (t.device() != first->device())
            raise(PyExc_ValueError, "the tensors lie on different devices: %s and %s", first->device().str().c_str(),
                  t.device().str().c_str());
    }
    if (!first) return;
    g_device = c10::cuda::current_device();
    if (first->device().index() != g_device)
        raise(PyExc_ValueError, "the tensors lie on %s, the current device is cuda:%d", first->device().str().c_str(),
              static_cast<int>(g_device));
}

// `stack` row-major matrices; a plain matrix is a stack of one.
struct Mat {
    void *p;
    int64_t mats, rows, cols, ld, gap;
};

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

Mat matrix_of(const Tensor &t, const char *name, int64_t es, bool stack)
{
    const int64_t d = stack ? 3 : 2;
    if (t.dim() != d) raise(PyExc_ValueError, "%s must be %d-D, got shape %s", name, static_cast<int>(d), shape_of(t).c_str());
    Mat m{t.data_ptr(), stack ? t.size(0) : 1, t.size(d - 2), t.size(d - 1), t.stride(d - 2), 0};
    if (m.cols > 1 && t.stride(d - 1) != 1) raise(PyExc_ValueError, "%s must be row-major with unit column stride", name);
    // One row: its pitch addresses nothing, so any value that meets the 16-byte rule will do.
    if (m.rows <= 1) m.ld = round_up(std::max({m.cols, m.ld, int64_t{1}}), 16 / es);
    m.gap = stack && m.mats > 1 ? t.stride(0) : m.rows * m.ld;
    return m;
}

Mat matrix(PyObject *o, const char *name, ScalarType dtype, bool stack = false)
{
    const Tensor &t = cuda_tensor(o, name, dtype);
    return matrix_of(t, name, t.element_size(), stack);
}

// A contiguous tensor of this shape.
void *flat(PyObject *o, const char *name, ScalarType dtype, at::IntArrayRef shape)
{
    const Tensor &t = cuda_tensor(o, name, dtype);
    if (t.sizes() != shape) {
        std::string s = "(";
        for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
        raise(PyExc_ValueError, "%s must have shape %s, got %s", name, (s + (shape.size() == 1 ? ",)" : ")")).c_str(),
              shape_of(t).c_str());
    }
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

void *flat_or_null(PyObject *o, const char *name, ScalarType dtype, at::IntArrayRef shape)
{
    return o == Py_None ? nullptr : flat(o, name, dtype, shape);
}

// A contiguous int32 tensor of `dim` dimensions.
const Tensor &index(PyObject *o, const char *name, int dim)
{
    const Tensor &t = tensor(o, name);
    if (t.dim() != dim) raise(PyExc_ValueError, "%s must be a %d-D tensor", name, dim);
    cuda_tensor(o, name, kI32);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

struct Logits {
    void *p;
    int64_t T, E, ld;
    int fp32;
    ScalarType dtype;
    at::Device device;
};
Logits logits(PyObject *o)
{
    const Tensor &t = tensor(o, "logits");
    const ScalarType dt = t.scalar_type();
    if (dt != kF32 && dt != kBF16) raise(PyExc_TypeError, "logits must be torch.float32 or torch.bfloat16, got %s", type_name(dt));
    cuda_tensor(o, "logits", dt);
    if (t.dim() != 2) raise(PyExc_ValueError, "logits must be 2-D, got shape %s", shape_of(t).c_str());
    const int64_t T = t.size(0), E = t.size(1);
    if (E > 1 && t.stride(1) != 1) raise(PyExc_ValueError, "logits must be row-major with unit column stride");
    return Logits{t.data_ptr(), T, E, T > 1 ? t.stride(0) : std::max(E, t.stride(0)), dt == kF32, dt, t.device()};
}

struct Tokens {
    void *p;
    int64_t n;
    int is64;
};
Tokens tokens(PyObject *o)
{
    if (!THPVariable_Check(o) || (THPVariable_Unpack(o).scalar_type() != kI64 && THPVariable_Unpack(o).scalar_type() != kI32))
        raise(PyExc_TypeError, "tokens must be an int64 or int32 tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 1) raise(PyExc_ValueError, "tokens must be 1-D, got shape %s", shape_of(t).c_str());
    const bool is64 = t.scalar_type() == kI64;
    return Tokens{flat(o, "tokens", t.scalar_type(), t.sizes()), t.size(0), is64};
}

// ---- outputs

Tensor empty(at::IntArrayRef shape, ScalarType dtype, at::Device device)
{
    return Tensor(at::detail::empty_cuda(shape, dtype, device, std::nullopt));
}

// [rows, cols], or [mats, rows, cols], with 16-byte row pitches.
Tensor empty_mat(int64_t rows, int64_t cols, ScalarType dtype, at::Device device, int64_t mats = -1)
{
    const int64_t ld = std::max<int64_t>(1, round_up(cols, 16 / static_cast<int64_t>(c10::elementSize(dtype))));
    if (mats < 0) return Tensor(at::detail::empty_strided_cuda({rows, cols}, {ld, 1}, dtype, device));
    return Tensor(at::detail::empty_strided_cuda({mats, rows, cols}, {rows * ld, ld, 1}, dtype, device));
}

// The output given as `o`, of this shape and type, or a new one.
Tensor output(PyObject *o, int64_t rows, int64_t cols, ScalarType dtype, at::Device device, int64_t mats = -1)
{
    if (o == Py_None) return empty_mat(rows, cols, dtype, device, mats);
    const Tensor &t = tensor(o, "out");
    const bool same = mats < 0 ? t.dim() == 2 && t.size(0) == rows && t.size(1) == cols
                               : t.dim() == 3 && t.size(0) == mats && t.size(1) == rows && t.size(2) == cols;
    if (!same) raise(PyExc_ValueError, "out has shape %s, which is not the result's", shape_of(t).c_str());
    return cuda_tensor(o, "out", dtype);
}

// The type of a product's or gradient's output: out's, or `dtype` ("bf16" or "fp32" as a number).
ScalarType out_type(PyObject *out, PyObject *fp32)
{
    if (out == Py_None) return integer(fp32, "out_dtype") ? kF32 : kBF16;
    const ScalarType t = tensor(out, "out").scalar_type();
    if (t != kF32 && t != kBF16) raise(PyExc_TypeError, "out_dtype must be torch.bfloat16 or torch.float32, got %s", type_name(t));
    return t;
}

det_gemm_stream stream() { return reinterpret_cast<det_gemm_stream>(c10::cuda::getCurrentCUDAStream(g_device).stream()); }

// Raises DetGemmError for a status that is not OK.
void check(det_gemm_status st, const char *name)
{
    if (st == DET_GEMM_OK) return;
    PyObject *m = PyImport_ImportModule("invariant_deterministic_gemm_gb300");
    PyObject *type = m ? PyObject_GetAttrString(m, "DetGemmError") : nullptr;
    PyObject *err = type ? PyObject_CallFunction(type, "is", static_cast<int>(st), name) : nullptr;
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_XDECREF(type);
    Py_XDECREF(m);
    throw Raised{};
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap(const Tensor &a, const Tensor &b)
{
    PyObject *r = PyTuple_New(2);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
    return r;
}

template <typename T = void>
T *ptr(const Tensor &t)
{
    return static_cast<T *>(t.data_ptr());
}
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
int64_t pitch(const Tensor &t, int64_t es)       // of an output made by empty_mat, any number of rows
{
    return std::max(t.stride(t.dim() - 2), 16 / es);
}

using bf16 = det_gemm_bf16;
using Argv = PyObject *const *;

// ---- the operators

PyObject *route(Argv a)
{
    const Logits l = logits(a[0]);
    const int k = small(a[1], "top_k");
    const float *bias = static_cast<float *>(flat_or_null(a[3], "bias", kF32, {l.E}));
    const int64_t room = std::clamp(k, 0, DET_MOE_MAX_TOP_K);          // the library refuses any other
    const Tensor w = empty({l.T, room}, kF32, l.device), ids = empty({l.T, room}, kI32, l.device);
    check(det_moe_route(l.p, l.fp32, bias, ptr<float>(w), ptr<int32_t>(ids), l.T, l.E, l.ld, k, small(a[2], "score"),
                        small(a[4], "n_groups"), small(a[5], "top_groups"), small(a[6], "group_best"),
                        truth(a[7]), real(a[8], "scale"), stream()),
          "det_moe_route");
    return wrap(w, ids);
}

PyObject *route_bwd(Argv a)
{
    const Logits l = logits(a[1]);
    const Tensor &ids = index(a[2], "ids", 2);
    if (ids.size(0) != l.T)
        raise(PyExc_ValueError, "logits and ids disagree on the tokens: %lld vs %lld", static_cast<long long>(l.T),
              static_cast<long long>(ids.size(0)));
    const int k = static_cast<int>(ids.size(1));
    const float *dw = static_cast<float *>(flat(a[0], "dweights", kF32, {l.T, k}));
    const Tensor d = empty({l.T, l.E}, l.dtype, l.device);
    check(det_moe_route_bwd(dw, l.p, l.fp32, ptr<int32_t>(ids), ptr(d), l.T, l.E, l.ld, l.E, k, small(a[3], "score"),
                            truth(a[4]), real(a[5], "scale"), stream()),
          "det_moe_route_bwd");
    return wrap(d);
}

PyObject *dispatch(Argv a)
{
    const Tensor &ids = index(a[0], "ids", 2);
    const int64_t E = integer(a[1], "num_experts"), T = ids.size(0), k = ids.size(1);
    const Tensor off = empty({std::clamp<int64_t>(E, -1, DET_MOE_MAX_EXPERTS) + 1}, kI32, ids.device()), rows = empty({T * k}, kI32, ids.device()),
                 slots = empty({T, k}, kI32, ids.device());
    check(det_moe_dispatch(ptr<int32_t>(ids), ptr<int32_t>(off), ptr<int32_t>(rows), ptr<int32_t>(slots), T, E,
                           static_cast<int>(std::min<int64_t>(k, INT32_MAX)), stream()),
          "det_moe_dispatch");
    PyObject *r = PyTuple_New(3);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(off));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(rows));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(slots));
    return r;
}

PyObject *gather(Argv a)
{
    const Mat x = matrix(a[0], "x", kBF16);
    const Tensor &rows = index(a[1], "rows", 1);
    const Tensor out = output(a[3], rows.size(0), x.cols, kBF16, rows.device());
    const Mat o = matrix_of(out, "out", 2, false);
    check(det_moe_gather(static_cast<bf16 *>(x.p), ptr<int32_t>(rows), static_cast<bf16 *>(o.p), x.rows, rows.size(0), x.cols,
                         small(a[2], "top_k"), x.ld, o.ld, stream()),
          "det_moe_gather");
    return wrap(out);
}

PyObject *combine(Argv a)
{
    const Mat ys = matrix(a[0], "ys", kBF16);
    const Tensor &slots = index(a[1], "slots", 2);
    const int64_t T = slots.size(0), k = slots.size(1);
    const float *w = static_cast<float *>(flat_or_null(a[2], "weights", kF32, {T, k}));
    const Tensor out = output(a[3], T, ys.cols, kBF16, slots.device());
    const Mat o = matrix_of(out, "out", 2, false);
    check(det_moe_combine(static_cast<bf16 *>(ys.p), ptr<int32_t>(slots), w, static_cast<bf16 *>(o.p), T, ys.rows, ys.cols,
                          static_cast<int>(std::min<int64_t>(k, INT32_MAX)), ys.ld, o.ld, stream()),
          "det_moe_combine");
    return wrap(out);
}

PyObject *combine_bwd(Argv a)
{
    const Mat dy = matrix(a[0], "dy", kBF16), ys = matrix(a[1], "ys", kBF16);
    const Tensor &slots = index(a[3], "slots", 2);
    const int64_t T = dy.rows, k = slots.size(1);
    if (slots.size(0) != T)
        raise(PyExc_ValueError, "dy and slots disagree on the tokens: %lld vs %lld", static_cast<long long>(T),
              static_cast<long long>(slots.size(0)));
    const int32_t *rows = static_cast<int32_t *>(flat(a[2], "rows", kI32, {T * k}));
    const float *w = static_cast<float *>(flat(a[4], "weights", kF32, {T, k}));
    if (ys.rows != T * k || ys.cols != dy.cols)
        raise(PyExc_ValueError, "ys must have shape (%lld, %lld), got (%lld, %lld)", static_cast<long long>(T * k),
              static_cast<long long>(dy.cols), static_cast<long long>(ys.rows), static_cast<long long>(ys.cols));
    const Tensor dys = empty_mat(T * k, dy.cols, kBF16, slots.device()), dw = empty({T, k}, kF32, slots.device());
    check(det_moe_combine_bwd(static_cast<bf16 *>(dy.p), static_cast<bf16 *>(ys.p), rows, ptr<int32_t>(slots), w,
                              ptr<bf16>(dys), ptr<float>(dw), T, dy.cols, static_cast<int>(std::min<int64_t>(k, INT32_MAX)),
                              dy.ld, ys.ld, pitch(dys, 2), stream()),
          "det_moe_combine_bwd");
    return wrap(dys, dw);
}

PyObject *quantize_rows(Argv a)
{
    const Mat x = matrix(a[0], "x", kBF16);
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    int64_t M = x.rows;
    const int32_t *rows = nullptr;
    if (a[1] != Py_None) {
        const Tensor &r = index(a[1], "rows", 1);
        rows = ptr<int32_t>(r);
        M = r.size(0);
    }
    const Tensor q = empty_mat(M, x.cols, kE4M3, dev);
    const int64_t lds = std::max<int64_t>(M, 1);
    const Tensor s(at::detail::empty_strided_cuda({M, blocks_of(x.cols)}, {1, lds}, kF32, dev));
    check(det_fp8_quantize_rows(static_cast<bf16 *>(x.p), rows, ptr<uint8_t>(q), ptr<float>(s), x.rows, M, x.cols,
                                small(a[2], "top_k"), x.ld, pitch(q, 1), lds, stream()),
          "det_fp8_quantize_rows");
    return wrap(q, s);
}

PyObject *quantize_cols(Argv a)
{
    const Mat x = matrix(a[0], "x", kBF16);
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    int64_t G = 0;
    const int32_t *off = nullptr;
    if (a[1] != Py_None) {
        const Tensor &o = index(a[1], "offsets", 1);
        off = ptr<int32_t>(o);
        G = std::max<int64_t>(o.size(0) - 1, 0);
    }
    const int64_t nb = blocks_of(x.rows) + G;
    const Tensor q = empty({x.cols, nb * kBlock}, kE4M3, dev), s = empty_mat(nb, x.cols, kF32, dev);
    check(det_fp8_quantize_cols(static_cast<bf16 *>(x.p), off, ptr<uint8_t>(q), ptr<float>(s), x.rows, x.cols, G, nb, x.ld,
                                nb * kBlock, pitch(s, 4), stream()),
          "det_fp8_quantize_cols");
    return wrap(q, s);
}

PyObject *quantize_tiles(Argv a)
{
    const Tensor &t = tensor(a[0], "w");
    if (t.dim() != 2 && t.dim() != 3) raise(PyExc_ValueError, "w must be a 2-D or 3-D tensor");
    const bool stack = t.dim() == 3, flip = truth(a[1]);
    const Mat w = matrix(a[0], "w", kBF16, stack);
    const int64_t rt = blocks_of(w.rows), ct = blocks_of(w.cols), mats = stack ? w.mats : -1;
    const Tensor q = flip ? empty_mat(w.cols, w.rows, kE4M3, t.device(), mats) : empty_mat(w.rows, w.cols, kE4M3, t.device(), mats);
    const int64_t s0 = flip ? ct : rt, s1 = flip ? rt : ct;
    const Tensor s = stack ? empty({w.mats, s0, s1}, kF32, t.device()) : empty({s0, s1}, kF32, t.device());
    const int64_t ld = pitch(q, 1), gap = std::max<int64_t>((flip ? w.cols : w.rows) * ld, 16);
    uint8_t *qp = ptr<uint8_t>(q);
    float *sp = ptr<float>(s);
    check(det_fp8_quantize_tiles(static_cast<bf16 *>(w.p), flip ? nullptr : qp, flip ? nullptr : sp, flip ? qp : nullptr,
                                 flip ? sp : nullptr, w.mats, w.rows, w.cols, w.ld, w.gap, ld, gap, ld, gap, stream()),
          "det_fp8_quantize_tiles");
    return wrap(q, s);
}

// A's scales: [rows, blocks] FP32 with any strides.
const Tensor &row_scales(PyObject *o, const char *name, int64_t rows, int64_t blocks)
{
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != kF32 || !t.is_cuda()) raise(PyExc_TypeError, "%s must be a float32 CUDA tensor", name);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != blocks)
        raise(PyExc_ValueError, "%s must have shape (%lld, %lld), got %s", name, static_cast<long long>(rows),
              static_cast<long long>(blocks), shape_of(t).c_str());
    return t;
}

void same_inner(int64_t a, int64_t b)
{
    if (a != b) raise(PyExc_ValueError, "inner dimensions differ: %lld vs %lld", static_cast<long long>(a), static_cast<long long>(b));
}

PyObject *gemm(Argv a)
{
    const Mat A = matrix(a[0], "A", kE4M3), W = matrix(a[2], "W", kE4M3);
    same_inner(A.cols, W.cols);
    const int64_t kb = blocks_of(A.cols);
    const Tensor &sa = row_scales(a[1], "a_scale", A.rows, kb);
    const float *sw = static_cast<float *>(flat(a[3], "w_scale", kF32, {blocks_of(W.rows), kb}));
    const ScalarType dt = out_type(a[5], a[4]);
    const Tensor out = output(a[5], A.rows, W.rows, dt, sa.device());
    const Mat c = matrix_of(out, "out", out.element_size(), false);
    check(det_fp8_gemm(static_cast<uint8_t *>(A.p), ptr<float>(sa), static_cast<uint8_t *>(W.p), sw, c.p, dt == kF32, A.rows,
                       W.rows, A.cols, A.ld, sa.stride(0), sa.stride(1), W.ld, kb, c.ld, stream()),
          "det_fp8_gemm");
    return wrap(out);
}

PyObject *gemm_grouped(Argv a)
{
    const Mat A = matrix(a[0], "A", kE4M3), W = matrix(a[2], "W", kE4M3, true);
    same_inner(A.cols, W.cols);
    const int64_t kb = blocks_of(A.cols), nb = blocks_of(W.rows);
    const Tensor &sa = row_scales(a[1], "a_scale", A.rows, kb);
    const float *sw = static_cast<float *>(flat(a[3], "w_scale", kF32, {W.mats, nb, kb}));
    const int32_t *off = static_cast<int32_t *>(flat(a[4], "offsets", kI32, {W.mats + 1}));
    const ScalarType dt = out_type(a[6], a[5]);
    const Tensor out = output(a[6], A.rows, W.rows, dt, sa.device());
    const Mat c = matrix_of(out, "out", out.element_size(), false);
    check(det_fp8_gemm_grouped(static_cast<uint8_t *>(A.p), ptr<float>(sa), static_cast<uint8_t *>(W.p), sw, off, c.p,
                               dt == kF32, W.mats, A.rows, W.rows, A.cols, A.ld, sa.stride(0), sa.stride(1), W.ld, W.gap, kb,
                               nb * kb, c.ld, stream()),
          "det_fp8_gemm_grouped");
    return wrap(out);
}

PyObject *gemm_wgrad(Argv a)
{
    const Mat Y = matrix(a[0], "Yt", kE4M3), X = matrix(a[2], "Xt", kE4M3);
    if (Y.cols != X.cols || Y.cols % kBlock)
        raise(PyExc_ValueError, "Yt and Xt must have the same whole number of blocks: %lld vs %lld columns",
              static_cast<long long>(Y.cols), static_cast<long long>(X.cols));
    const int64_t nb = Y.cols / kBlock;
    const Mat sy = matrix(a[1], "y_scale", kF32), sx = matrix(a[3], "x_scale", kF32);
    if (sy.rows != nb || sy.cols != Y.rows || sx.rows != nb || sx.cols != X.rows)
        raise(PyExc_ValueError, "y_scale and x_scale must have shapes (%lld, %lld) and (%lld, %lld)", static_cast<long long>(nb),
              static_cast<long long>(Y.rows), static_cast<long long>(nb), static_cast<long long>(X.rows));
    int64_t G = 1, M = Y.cols;
    const int32_t *off = nullptr;
    if (a[4] != Py_None) {
        const Tensor &o = index(a[4], "offsets", 1);
        off = ptr<int32_t>(o);
        G = o.size(0) - 1;
        M = (nb - G) * kBlock;                       // at least the tokens' number
        if (G < 0 || M < 0) raise(PyExc_ValueError, "offsets does not match the blocks of Yt and Xt");
    }
    const ScalarType dt = out_type(a[6], a[5]);
    const Tensor out = output(a[6], Y.rows, X.rows, dt, THPVariable_Unpack(a[0]).device(), off || a[4] != Py_None ? G : -1);
    const Mat d = matrix_of(out, "out", out.element_size(), out.dim() == 3);
    check(det_fp8_gemm_wgrad(static_cast<uint8_t *>(Y.p), static_cast<float *>(sy.p), static_cast<uint8_t *>(X.p),
                             static_cast<float *>(sx.p), off, d.p, dt == kF32, G, M, Y.rows, X.rows, nb, Y.ld, sy.ld, X.ld,
                             sx.ld, d.ld, d.gap, stream()),
          "det_fp8_gemm_wgrad");
    return wrap(out);
}

PyObject *embedding(Argv a)
{
    const Tokens t = tokens(a[0]);
    const Mat w = matrix(a[1], "table", kBF16);
    const Tensor out = output(a[3], t.n, w.cols, kBF16, THPVariable_Unpack(a[1]).device());
    const Mat o = matrix_of(out, "out", 2, false);
    check(det_embedding(t.p, t.is64, static_cast<bf16 *>(w.p), static_cast<bf16 *>(o.p), t.n, w.rows, w.cols,
                        real(a[2], "scale"), w.ld, o.ld, stream()),
          "det_embedding");
    return wrap(out);
}

PyObject *embedding_grad(Argv a)
{
    const Mat dy = matrix(a[0], "dy", kBF16);
    const Tokens t = tokens(a[1]);
    if (t.n != dy.rows)
        raise(PyExc_ValueError, "dy and tokens disagree on the tokens: %lld vs %lld", static_cast<long long>(dy.rows),
              static_cast<long long>(t.n));
    const int64_t V = integer(a[2], "vocab");
    const bool accumulate = truth(a[7]);
    if (accumulate && a[6] == Py_None) raise(PyExc_ValueError, "accumulate needs out");
    int64_t pad = -1;
    if (a[4] != Py_None) {
        pad = integer(a[4], "padding_idx");
        if (pad < 0 || pad >= V) raise(PyExc_ValueError, "padding_idx must be in [0, vocab)");
    }
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    const ScalarType dt = out_type(a[6], a[5]);
    const int64_t size = std::max<int64_t>(det_embedding_grad_workspace(t.n, V, dy.cols), 256);
    const Tensor ws = empty({size}, ScalarType::Byte, dev);
    const Tensor out = output(a[6], std::max<int64_t>(V, 0), dy.cols, dt, dev);
    const Mat o = matrix_of(out, "out", out.element_size(), false);
    check(det_embedding_grad(static_cast<bf16 *>(dy.p), t.p, t.is64, o.p, dt == kF32, t.n, V, dy.cols, real(a[3], "scale"),
                             pad, accumulate, dy.ld, o.ld, ptr(ws), size, stream()),
          "det_embedding_grad");
    return wrap(out);
}

// ---- attention

// [tokens, heads, D] with any strides but D's.
struct Rows {
    bf16 *p;
    int64_t T, H, D, t, h;
};

Rows rows_of(const Tensor &t, const char *name)
{
    if (t.dim() != 3) raise(PyExc_ValueError, "%s must be 3-D, got shape %s", name, shape_of(t).c_str());
    if (t.size(2) > 1 && t.stride(2) != 1) raise(PyExc_ValueError, "%s must have unit stride in its last dimension", name);
    return Rows{static_cast<bf16 *>(t.data_ptr()), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
}
Rows rows(PyObject *o, const char *name) { return rows_of(cuda_tensor(o, name, kBF16), name); }

// The output given as `o`, or a new one.
Tensor rows_out(PyObject *o, int64_t T, int64_t H, int64_t D, at::Device device)
{
    if (o == Py_None) return empty({T, H, D}, kBF16, device);
    const Tensor &t = cuda_tensor(o, "out", kBF16);
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D)
        raise(PyExc_ValueError, "out has shape %s, which is not the result's", shape_of(t).c_str());
    return t;
}

void same(const Rows &a, const char *an, const Rows &b, const char *bn, bool tokens, bool heads)
{
    if (a.D != b.D || (tokens && a.T != b.T) || (heads && a.H != b.H))
        raise(PyExc_ValueError, "%s and %s disagree: (%lld, %lld, %lld) vs (%lld, %lld, %lld)", an, bn, static_cast<long long>(a.T),
              static_cast<long long>(a.H), static_cast<long long>(a.D), static_cast<long long>(b.T), static_cast<long long>(b.H),
              static_cast<long long>(b.D));
}

// cos and sin [P, rot / 2].
struct Turn {
    const float *c, *s;
    int64_t P, rot, ld;
};
Turn turn_of(PyObject *co, PyObject *si)
{
    const Tensor &c = cuda_tensor(co, "cos", kF32), &s = cuda_tensor(si, "sin", kF32);
    if (c.dim() != 2 || s.sizes() != c.sizes() || s.strides() != c.strides() || (c.size(1) > 1 && c.stride(1) != 1))
        raise(PyExc_ValueError, "cos and sin must be 2-D, of one shape and layout, with unit column stride");
    return Turn{ptr<float>(c), ptr<float>(s), c.size(0), 2 * c.size(1), c.size(0) > 1 ? c.stride(0) : std::max<int64_t>(c.size(1), 1)};
}

struct Pages {
    bf16 *p;
    int64_t pages, size, heads, D, sp, ss, sh;
};
Pages pages_of(PyObject *o, const char *name)
{
    const Tensor &t = cuda_tensor(o, name, kBF16);
    if (t.dim() != 4) raise(PyExc_ValueError, "%s must be 4-D, got shape %s", name, shape_of(t).c_str());
    if (t.size(3) > 1 && t.stride(3) != 1) raise(PyExc_ValueError, "%s must have unit stride in its last dimension", name);
    return Pages{static_cast<bf16 *>(t.data_ptr()), t.size(0), t.size(1), t.size(2), t.size(3), t.stride(0), t.stride(1), t.stride(2)};
}
void same(const Pages &k, const Pages &v)
{
    if (k.pages != v.pages || k.size != v.size || k.heads != v.heads || k.D != v.D)
        raise(PyExc_ValueError, "k_cache and v_cache must have one shape");
}

float scale_of(PyObject *o, int64_t D) { return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(std::max<int64_t>(D, 1)))) : real(o, "scale"); }
int64_t window_of(PyObject *o)
{
    if (o == Py_None) return 0;
    const int64_t w = integer(o, "window");
    if (w < 1) raise(PyExc_ValueError, "window must be at least 1 (None: no window)");
    return w;
}

PyObject *rope(Argv a)
{
    const Rows x = rows(a[0], "x");
    const Turn c = turn_of(a[1], a[2]);
    const int32_t *pos = static_cast<int32_t *>(flat(a[3], "positions", kI32, {x.T}));
    const Tensor out = rows_out(a[6], x.T, x.H, x.D, THPVariable_Unpack(a[0]).device());
    const Rows y = rows_of(out, "out");
    check(det_rope(x.p, c.c, c.s, pos, y.p, x.T, x.H, x.D, c.rot, c.P, truth(a[4]), truth(a[5]), x.t, x.h, c.ld, y.t, y.h, stream()),
          "det_rope");
    return wrap(out);
}

PyObject *kv_append(Argv a)
{
    const Rows k = rows(a[1], "k"), v = rows(a[2], "v");
    same(k, "k", v, "v", true, true);
    const Turn c = turn_of(a[3], a[4]);
    const int32_t *pos = static_cast<int32_t *>(flat(a[5], "positions", kI32, {k.T})),
                  *slots = static_cast<int32_t *>(flat(a[6], "slots", kI32, {k.T}));
    const Pages kc = pages_of(a[7], "k_cache"), vc = pages_of(a[8], "v_cache");
    same(kc, vc);
    if (kc.heads != k.H || kc.D != k.D)
        raise(PyExc_ValueError, "k and k_cache disagree on the heads: (%lld, %lld) vs (%lld, %lld)", static_cast<long long>(k.H),
              static_cast<long long>(k.D), static_cast<long long>(kc.heads), static_cast<long long>(kc.D));
    Rows q{}, y{};
    Tensor out;
    if (a[0] != Py_None) {
        q = rows(a[0], "q");
        same(q, "q", k, "k", true, false);
        out = rows_out(a[10], q.T, q.H, q.D, THPVariable_Unpack(a[0]).device());
        y = rows_of(out, "out");
    } else if (a[10] != Py_None) {
        raise(PyExc_ValueError, "out needs q");
    }
    check(det_kv_append(q.p, k.p, v.p, c.c, c.s, pos, slots, y.p, kc.p, vc.p, k.T, q.H, k.H, k.D, c.rot, c.P, kc.pages, kc.size,
                        truth(a[9]), q.t, q.h, k.t, k.h, v.t, v.h, c.ld, y.t, y.h, kc.sp, kc.ss, kc.sh, vc.sp, vc.ss, vc.sh,
                        stream()),
          "det_kv_append");
    if (a[0] == Py_None) Py_RETURN_NONE;
    return wrap(out);
}

PyObject *attn_decode(Argv a)
{
    const Rows q = rows(a[0], "q");
    const Pages kc = pages_of(a[1], "k_cache"), vc = pages_of(a[2], "v_cache");
    same(kc, vc);
    if (kc.D != q.D) raise(PyExc_ValueError, "q and k_cache disagree on the head's columns: %lld vs %lld", static_cast<long long>(q.D), static_cast<long long>(kc.D));
    const Tensor &table = cuda_tensor(a[3], "table", kI32);
    if (table.dim() != 2 || table.size(0) != q.T) raise(PyExc_ValueError, "table must have a row for each query, got shape %s", shape_of(table).c_str());
    const int64_t most = table.size(1);
    if (most > 1 && table.stride(1) != 1) raise(PyExc_ValueError, "table must be row-major with unit column stride");
    const int32_t *lengths = static_cast<int32_t *>(flat(a[4], "lengths", kI32, {q.T}));
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    const int64_t tokens = kc.size > 0 && most <= INT32_MAX / kc.size ? most * kc.size : 0;     // the library refuses more
    const int64_t size = std::max<int64_t>(det_attn_decode_workspace(q.T, q.H, kc.heads, q.D, tokens), 256);
    const Tensor ws = empty({size}, ScalarType::Byte, dev);
    const Tensor out = rows_out(a[8], q.T, q.H, q.D, dev);
    const Rows y = rows_of(out, "out");
    check(det_attn_decode(q.p, kc.p, vc.p, ptr<int32_t>(table), lengths, y.p, q.T, q.H, kc.heads, q.D, kc.pages, kc.size, most,
                          scale_of(a[5], q.D), window_of(a[6]), integer(a[7], "sinks"), q.t, q.h, kc.sp, kc.ss, kc.sh, vc.sp, vc.ss,
                          vc.sh, q.T > 1 ? table.stride(0) : std::max<int64_t>(most, 1), y.t, y.h, ptr(ws), size, stream()),
          "det_attn_decode");
    return wrap(out);
}

// The bounds of packed sequences: queries' and keys', either may be None.
struct Packed {
    const int32_t *q, *k;
    int64_t N;
};
Packed packed(PyObject *qb, PyObject *kb, int64_t T, int64_t S)
{
    if (qb == Py_None) {
        if (kb != Py_None) raise(PyExc_ValueError, "k_bounds needs bounds");
        return Packed{nullptr, nullptr, 1};
    }
    const Tensor &q = index(qb, "bounds", 1);
    if (q.size(0) < 1) raise(PyExc_ValueError, "bounds must have an element more than there are sequences");
    Packed r{ptr<int32_t>(q), nullptr, q.size(0) - 1};
    if (kb != Py_None) r.k = static_cast<int32_t *>(flat(kb, "k_bounds", kI32, q.sizes()));
    else if (T != S) raise(PyExc_ValueError, "q and k have %lld and %lld rows: k_bounds is needed", static_cast<long long>(T), static_cast<long long>(S));
    return r;
}

PyObject *attn(Argv a)
{
    const Rows q = rows(a[0], "q"), k = rows(a[1], "k"), v = rows(a[2], "v");
    same(q, "q", k, "k", false, false);
    same(k, "k", v, "v", true, true);
    const Packed b = packed(a[3], a[4], q.T, k.T);
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    const Tensor out = rows_out(a[8], q.T, q.H, q.D, dev), lse = empty({q.H, q.T}, kF32, dev);
    const Rows y = rows_of(out, "out");
    check(det_attn(q.p, k.p, v.p, b.q, b.k, y.p, ptr<float>(lse), b.N, q.T, k.T, q.H, k.H, q.D, scale_of(a[5], q.D), window_of(a[6]),
                   integer(a[7], "sinks"), q.t, q.h, k.t, k.h, v.t, v.h, y.t, y.h, stream()),
          "det_attn");
    return wrap(out, lse);
}

PyObject *attn_bwd(Argv a)
{
    const Rows d = rows(a[0], "dout"), q = rows(a[1], "q"), k = rows(a[2], "k"), v = rows(a[3], "v"), y = rows(a[4], "out");
    same(q, "q", k, "k", false, false);
    same(k, "k", v, "v", true, true);
    same(d, "dout", q, "q", true, true);
    same(y, "out", q, "q", true, true);
    const float *lse = static_cast<float *>(flat(a[5], "lse", kF32, {q.H, q.T}));
    const Packed b = packed(a[6], a[7], q.T, k.T);
    const at::Device dev = THPVariable_Unpack(a[0]).device();
    const int64_t window = window_of(a[9]), sinks = integer(a[10], "sinks");
    const int64_t size = std::max<int64_t>(det_attn_bwd_workspace(b.N, q.T, k.T, q.H, k.H, q.D, window, sinks), 256);
    const Tensor ws = empty({size}, ScalarType::Byte, dev);
    const Tensor dq = empty({q.T, q.H, q.D}, kBF16, dev), dk = empty({k.T, k.H, k.D}, kBF16, dev), dv = empty({k.T, k.H, k.D}, kBF16, dev);
    const int64_t qt = q.H * q.D, kt = k.H * k.D;
    check(det_attn_bwd(d.p, q.p, k.p, v.p, y.p, lse, b.q, b.k, ptr<bf16>(dq), ptr<bf16>(dk), ptr<bf16>(dv), b.N, q.T, k.T, q.H, k.H, q.D,
                       scale_of(a[8], q.D), window, sinks, d.t, d.h, q.t, q.h, k.t, k.h, v.t, v.h, y.t, y.h,
                       qt, q.D, kt, k.D, kt, k.D, ptr(ws), size, stream()),
          "det_attn_bwd");
    PyObject *r = PyTuple_New(3);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dq));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dk));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(dv));
    return r;
}

PyObject *force_timeout(Argv a)
{
    det_ops_debug_force_timeout(truth(a[0]));
    Py_RETURN_NONE;
}

// The Python-visible form of `F`, which takes exactly N positional arguments.
template <PyObject *(*F)(Argv), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        on_current_device(args, n);
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(Argv), int N>
PyMethodDef method(const char *name)
{
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<route, 9>("route"),
    method<route_bwd, 6>("route_bwd"),
    method<dispatch, 2>("dispatch"),
    method<gather, 4>("gather"),
    method<combine, 4>("combine"),
    method<combine_bwd, 5>("combine_bwd"),
    method<quantize_rows, 3>("quantize_rows"),
    method<quantize_cols, 2>("quantize_cols"),
    method<quantize_tiles, 2>("quantize_tiles"),
    method<gemm, 6>("gemm"),
    method<gemm_grouped, 7>("gemm_grouped"),
    method<gemm_wgrad, 7>("gemm_wgrad"),
    method<embedding, 4>("embedding"),
    method<embedding_grad, 8>("embedding_grad"),
    method<rope, 7>("rope"),
    method<kv_append, 11>("kv_append"),
    method<attn_decode, 9>("attn_decode"),
    method<attn, 9>("attn"),
    method<attn_bwd, 11>("attn_bwd"),
    method<force_timeout, 1>("force_timeout"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_native(void) { return PyModule_Create(&g_module); }
