// Python module between expert_ops.py and the entry points of expert_ops.h:
// checks tensors, allocates results and workspaces from PyTorch's allocator and
// makes the call.  In C++ because most calls of a decoding step are as short
// as their marshalling: through ctypes and Python's torch.empty a routing
// call cost 14.7 us, of which its kernel takes 4.
//
// Every function takes the stream last and returns its results, or an int:
// the status of a call that failed.  Wrong arguments raise TypeError or
// ValueError.  The library is already loaded; bind() takes the addresses of
// its entry points.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>

#include "expert_ops.h"

namespace {

enum { LINEAR, WEIGHT_GRAD, QUANTIZE, DEQUANTIZE, MX4_SPACE, MX4_LINEAR, ROUTE_SPACE, ROUTE, ROUTE_GRAD,
       BALANCE_SPACE, BALANCE, BALANCE_GRAD, QUANTIZE8, DEQUANTIZE8, INT8_SPACE, INT8_LINEAR, ORTHO_SPACE, ORTHO, COUNT };
const char *const kNames[COUNT] = {
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize",   "expert_mx4_dequantize",
    "expert_mx4_workspace",  "expert_mx4_linear",          "expert_route_workspace", "expert_route",
    "expert_route_grad",     "expert_route_balanced_workspace", "expert_route_balanced", "expert_route_balanced_grad",
    "expert_int8_quantize",  "expert_int8_dequantize",     "expert_int8_workspace",  "expert_int8_linear",
    "expert_orthogonalize_workspace", "expert_orthogonalize"};
void *g_entry[COUNT];

#define ENTRY(which, function) reinterpret_cast<decltype(&function)>(g_entry[which])

using at::Tensor;

struct Wrong {
    PyObject *type;
    std::string what;
};

[[noreturn]] void wrong_value(std::string what) { throw Wrong{PyExc_ValueError, std::move(what)}; }
[[noreturn]] void wrong_type(std::string what) { throw Wrong{PyExc_TypeError, std::move(what)}; }

const Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) wrong_type(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// NULL for None.
const Tensor *optional(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

void *stream_of(PyObject *o)
{
    void *s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw python_error();
    return s;
}

std::string shape_of(const Tensor &t)
{
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

int dtype_of(const Tensor &t, const char *what)
{
    if (t.scalar_type() == at::kFloat) return EXPERT_F32;
    if (t.scalar_type() == at::kBFloat16) return EXPERT_BF16;
    wrong_type(std::string(what) + " must be float32 or bfloat16");
}

void on_gpu(const Tensor &t, const char *what)
{
    if (!t.is_cuda()) wrong_value(std::string(what) + " must be on a GPU");
}

void on(const at::Device &device, const Tensor &t, const char *what)
{
    if (t.device() != device) wrong_value(std::string(what) + " must be on " + device.str());
}

// Distance between the rows of a matrix with unit stride along its columns.
int64_t rows_of(const Tensor &t, const char *what)
{
    if (t.dim() != 2) wrong_value(std::string(what) + " must be 2-D");
    const int64_t cols = t.size(1);
    if (cols > 1 && t.stride(1) != 1) wrong_value(std::string(what) + " needs unit stride along its rows");
    if (t.size(0) <= 1) return cols;
    if (t.stride(0) < cols) wrong_value(std::string(what) + " has overlapping rows");
    return t.stride(0);
}

const int *offsets_of(const Tensor &t, int64_t groups, const at::Device &device)
{
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.numel() != groups + 1 || !t.is_contiguous())
        wrong_value("offsets must be " + std::to_string(groups + 1) + " contiguous int32 values");
    on(device, t, "offsets");
    return static_cast<const int *>(t.const_data_ptr());
}

// bias (groups, n), or (n) for one matrix.
const float *bias_of(const Tensor *t, int64_t groups, int64_t n, bool flat, const at::Device &device)
{
    if (!t) return nullptr;
    const bool fits = t->dim() == 2 ? t->size(0) == groups && t->size(1) == n : flat && t->dim() == 1 && t->size(0) == n;
    if (t->scalar_type() != at::kFloat || !fits || !t->is_contiguous())
        wrong_value("bias must be a contiguous float32 (" + std::to_string(groups) + ", " + std::to_string(n) + ") tensor");
    on(device, *t, "bias");
    return static_cast<const float *>(t->const_data_ptr());
}

Tensor result(const Tensor *out, at::IntArrayRef shape, at::ScalarType dtype, const at::Device &device)
{
    if (!out) return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
    if (out->sizes() != shape || out->scalar_type() != dtype || out->device() != device) {
        std::string s;
        for (int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
        wrong_value(std::string("out must be a ") + at::toString(dtype) + " (" + s + ") tensor on " + device.str());
    }
    return *out;
}

PyObject *status(int st) { return PyLong_FromLong(st); }

// Calls f() on the device with the GIL released.
template <class F>
int call(const at::Device &device, F f)
{
    pybind11::gil_scoped_release release;
    const c10::DeviceGuard guard(device);
    return f();
}

PyObject *grouped_linear(PyObject *const *args)
{
    const Tensor &a = tensor(args[0], "a"), &b = tensor(args[1], "b"), &offsets = tensor(args[2], "offsets");
    const Tensor *bias = optional(args[3], "bias"), *out = optional(args[5], "out");
    const int act = (int)integer(args[4]);
    void *const stream = stream_of(args[6]);
    const int dt = dtype_of(a, "a");
    on_gpu(a, "a");
    const int64_t lda = rows_of(a, "a");
    if (b.dim() != 3) wrong_value("b must be 3-D");
    if (b.scalar_type() != a.scalar_type()) wrong_type("a and b must have the same type");
    const int64_t m = a.size(0), k = a.size(1), groups = b.size(0), n = b.size(2);
    if (b.size(1) != k) wrong_value("inner dimensions differ: a is " + shape_of(a) + ", b is " + shape_of(b));
    const int64_t se = b.stride(0), sk = b.stride(1), sn = b.stride(2);
    int layout;
    int64_t ldb;
    if (sn == 1 || (n == 1 && sk != 1)) {
        layout = GEMM_F32_ROW_MAJOR;
        ldb = k > 1 ? sk : n;
        if (ldb < n) wrong_value("b has overlapping rows");
    } else if (sk == 1 || k == 1) {
        layout = GEMM_F32_COL_MAJOR;
        ldb = n > 1 ? sn : k;
        if (ldb < k) wrong_value("b has overlapping rows");
    } else {
        wrong_value("b needs unit stride along n or along k");
    }
    const at::Device device = a.device();
    on(device, b, "b");
    const int *const off = offsets_of(offsets, groups, device);
    const float *const bias_p = bias_of(bias, groups, n, false, device);
    const Tensor c = result(out, {m, n}, a.scalar_type(), device);
    const int64_t ldc = rows_of(c, "out");
    const int st = call(device, [&] {
        return ENTRY(LINEAR, expert_grouped_linear)(dt, m, n, k, groups, a.const_data_ptr(), lda, b.const_data_ptr(),
                                                    layout, ldb, se, off, bias_p, act, c.mutable_data_ptr(), ldc, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(c) : status(st);
}

PyObject *grouped_weight_grad(PyObject *const *args)
{
    const Tensor &a = tensor(args[0], "a"), &grad = tensor(args[1], "grad"), &offsets = tensor(args[2], "offsets");
    const Tensor *out = optional(args[3], "out");
    void *const stream = stream_of(args[4]);
    const int dt = dtype_of(a, "a");
    on_gpu(a, "a");
    const int64_t lda = rows_of(a, "a"), ldg = rows_of(grad, "grad");
    if (grad.scalar_type() != a.scalar_type()) wrong_type("a and grad must have the same type");
    if (grad.size(0) != a.size(0)) wrong_value("row counts differ: a is " + shape_of(a) + ", grad is " + shape_of(grad));
    const at::Device device = a.device();
    on(device, grad, "grad");
    const int64_t groups = offsets.numel() - 1, m = a.size(0), k = a.size(1), n = grad.size(1);
    if (groups < 1) wrong_value("offsets must be groups + 1 contiguous int32 values");
    const int *const off = offsets_of(offsets, groups, device);
    const Tensor c = result(out, {groups, k, n}, a.scalar_type(), device);
    const int64_t ldd = k > 1 ? c.stride(1) : n;
    if ((n > 1 && c.stride(2) != 1) || ldd < n) wrong_value("out needs unit stride along its rows");
    const int64_t se = c.stride(0);
    if (groups > 1 && se < (k - 1) * ldd + n && (se < n || ldd < (groups - 1) * se + n))
        wrong_value("out has overlapping experts");
    const int st = call(device, [&] {
        return ENTRY(WEIGHT_GRAD, expert_grouped_weight_grad)(dt, m, n, k, groups, a.const_data_ptr(), lda,
                                                              grad.const_data_ptr(), ldg, off, c.mutable_data_ptr(), ldd,
                                                              c.stride(0), stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(c) : status(st);
}

// The results of a call, in order.
PyObject *results(std::initializer_list<Tensor> all)
{
    PyObject *const tuple = PyTuple_New((Py_ssize_t)all.size());
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor &t : all) PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(t));
    return tuple;
}

// A matrix to quantise, with unit stride along either axis.
struct Source {
    int dt, layout;
    int64_t r, k, ld;

    explicit Source(const Tensor &x) : dt(dtype_of(x, "x")), layout(GEMM_F32_ROW_MAJOR)
    {
        on_gpu(x, "x");
        if (x.dim() != 2) wrong_value("x must be 2-D");
        r = x.size(0);
        k = x.size(1);
        if (k < 1) wrong_value("x needs at least one column");
        ld = r > 1 ? x.stride(0) : k;
        if (!(k == 1 || x.stride(1) == 1 || r == 0)) {
            if (!(r == 1 || x.stride(0) == 1)) wrong_value("x needs unit stride along one axis");
            layout = GEMM_F32_COL_MAJOR;
            ld = x.stride(1);
        }
        if (r > 0 && ld < (layout == GEMM_F32_COL_MAJOR ? r : k)) wrong_value("x has overlapping rows");
        if (r == 0) ld = k;
    }
};

PyObject *mx4_quantize(PyObject *const *args)
{
    const Tensor &x = tensor(args[0], "x");
    void *const stream = stream_of(args[1]);
    const Source s(x);
    const int64_t kb = (s.k + 127) / 128;
    const auto bytes = at::TensorOptions().dtype(at::kByte).device(x.device());
    const Tensor codes = at::empty({s.r, kb * 64}, bytes), scales = at::empty({kb, s.r, 4}, bytes);
    const int st = call(x.device(), [&] {
        return ENTRY(QUANTIZE, expert_mx4_quantize)(s.dt, s.r, s.k, x.const_data_ptr(), s.layout, s.ld,
                                                    codes.mutable_data_ptr(), scales.mutable_data_ptr(), stream);
    });
    return st == GEMM_F32_SUCCESS ? results({codes, scales}) : status(st);
}

PyObject *int8_quantize(PyObject *const *args)
{
    const Tensor &x = tensor(args[0], "x");
    void *const stream = stream_of(args[1]);
    const Source s(x);
    const auto options = at::TensorOptions().device(x.device());
    const Tensor codes = at::empty({s.r, (s.k + 15) / 16 * 16}, options.dtype(at::kChar));
    const Tensor scales = at::empty({s.r}, options.dtype(at::kFloat));
    const int st = call(x.device(), [&] {
        return ENTRY(QUANTIZE8, expert_int8_quantize)(s.dt, s.r, s.k, x.const_data_ptr(), s.layout, s.ld,
                                                      codes.mutable_data_ptr(), static_cast<float *>(scales.mutable_data_ptr()),
                                                      stream);
    });
    return st == GEMM_F32_SUCCESS ? results({codes, scales}) : status(st);
}

PyObject *int8_dequantize(PyObject *const *args)
{
    const Tensor &codes = tensor(args[0], "codes"), &scales = tensor(args[1], "scales");
    const int64_t k = integer(args[2]);
    const int dt = (int)integer(args[3]);
    const Tensor *out = optional(args[4], "out");
    void *const stream = stream_of(args[5]);
    if (codes.dim() != 2) wrong_value("q must hold one matrix");
    on_gpu(codes, "q");
    const int64_t r = codes.size(0);
    const Tensor x = result(out, {r, k}, dt == EXPERT_BF16 ? at::kBFloat16 : at::kFloat, codes.device());
    const int64_t ld = rows_of(x, "out");
    const int st = call(codes.device(), [&] {
        return ENTRY(DEQUANTIZE8, expert_int8_dequantize)(dt, r, k, codes.const_data_ptr(),
                                                          static_cast<const float *>(scales.const_data_ptr()),
                                                          x.mutable_data_ptr(), ld, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(x) : status(st);
}

// x and the 8-bit or 4-bit matrices of a product, and its result.
struct Product {
    const Tensor &x, &codes, &scales;
    const Tensor *offsets, *bias, *out;
    int dt, act;
    void *stream;
    int64_t ldx, m, k, groups, n, ldy;
    at::Device device;
    bool many;
    const int *off;
    const float *bias_p;
    Tensor y;

    explicit Product(PyObject *const *args)
        : x(tensor(args[0], "x")), codes(tensor(args[1], "w")), scales(tensor(args[2], "w")),
          offsets(optional(args[4], "offsets")), bias(optional(args[5], "bias")), out(optional(args[7], "out")),
          device(x.device())
    {
        const int64_t wk = integer(args[3]);
        act = (int)integer(args[6]);
        stream = stream_of(args[8]);
        dt = dtype_of(x, "x");
        on_gpu(x, "x");
        ldx = rows_of(x, "x");
        m = x.size(0);
        k = x.size(1);
        if (k != wk) wrong_value("inner dimensions differ: x is " + shape_of(x) + ", w has " + std::to_string(wk) + " columns");
        on(device, codes, "w");
        many = codes.dim() == 3;
        groups = many ? codes.size(0) : 1;
        n = codes.size(-2);
        if (many && !offsets) wrong_value("one matrix an expert needs offsets");
        if (!many && offsets) wrong_value("offsets need one matrix an expert");
        off = many ? offsets_of(*offsets, groups, device) : nullptr;
        bias_p = bias_of(bias, groups, n, !many, device);
        y = result(out, {m, n}, x.scalar_type(), device);
        ldy = rows_of(y, "out");
    }
};

PyObject *int8_linear(PyObject *const *args)
{
    const Product p(args);
    const int64_t need = ENTRY(INT8_SPACE, expert_int8_workspace)(p.m, p.k);
    Tensor space;
    if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(p.device));
    const int st = call(p.device, [&] {
        return ENTRY(INT8_LINEAR, expert_int8_linear)(p.dt, p.m, p.n, p.k, p.groups, p.x.const_data_ptr(), p.ldx,
                                                      p.codes.const_data_ptr(),
                                                      static_cast<const float *>(p.scales.const_data_ptr()), p.off, p.bias_p,
                                                      p.act, p.y.mutable_data_ptr(), p.ldy,
                                                      need ? space.mutable_data_ptr() : nullptr, need, p.stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(p.y) : status(st);
}

PyObject *mx4_dequantize(PyObject *const *args)
{
    const Tensor &codes = tensor(args[0], "codes"), &scales = tensor(args[1], "scales");
    const int64_t k = integer(args[2]);
    const int dt = (int)integer(args[3]);
    const Tensor *out = optional(args[4], "out");
    void *const stream = stream_of(args[5]);
    if (codes.dim() != 2) wrong_value("q must hold one matrix");
    on_gpu(codes, "q");
    const int64_t r = codes.size(0);
    const Tensor x = result(out, {r, k}, dt == EXPERT_BF16 ? at::kBFloat16 : at::kFloat, codes.device());
    const int64_t ld = rows_of(x, "out");
    const int st = call(codes.device(), [&] {
        return ENTRY(DEQUANTIZE, expert_mx4_dequantize)(dt, r, k, codes.const_data_ptr(), scales.const_data_ptr(),
                                                        x.mutable_data_ptr(), ld, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(x) : status(st);
}

PyObject *mx4_linear(PyObject *const *args)
{
    const Product p(args);
    const int64_t need = ENTRY(MX4_SPACE, expert_mx4_workspace)(p.m, p.n, p.k, p.groups);
    Tensor space;
    if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(p.device));
    const int st = call(p.device, [&] {
        return ENTRY(MX4_LINEAR, expert_mx4_linear)(p.dt, p.m, p.n, p.k, p.groups, p.x.const_data_ptr(), p.ldx,
                                                    p.codes.const_data_ptr(), p.scales.const_data_ptr(), p.off, p.bias_p, p.act,
                                                    p.y.mutable_data_ptr(), p.ldy, need ? space.mutable_data_ptr() : nullptr,
                                                    need, p.stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(p.y) : status(st);
}

// What a routing call writes.
struct Routed {
    Tensor weights, experts, offsets, order, space;

    Routed(const at::Device &device, int64_t tokens, int64_t groups, int64_t choices, int64_t need)
    {
        const auto floats = at::TensorOptions().dtype(at::kFloat).device(device);
        const auto ints = at::TensorOptions().dtype(at::kInt).device(device);
        weights = at::empty({tokens, choices}, floats);
        experts = at::empty({tokens, choices}, ints);
        offsets = at::empty({groups + 1}, ints);
        order = at::empty({tokens * choices}, ints);
        if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(device));
    }
    float *w() const { return static_cast<float *>(weights.mutable_data_ptr()); }
    int *e() const { return static_cast<int *>(experts.mutable_data_ptr()); }
    int *off() const { return static_cast<int *>(offsets.mutable_data_ptr()); }
    int *ord() const { return static_cast<int *>(order.mutable_data_ptr()); }
    void *work() const { return space.defined() ? space.mutable_data_ptr() : nullptr; }
};

PyObject *route(PyObject *const *args)
{
    const Tensor &logits = tensor(args[0], "logits");
    const int64_t choices = integer(args[1]);
    const int normalize = (int)integer(args[2]);
    void *const stream = stream_of(args[3]);
    const int dt = dtype_of(logits, "logits");
    on_gpu(logits, "logits");
    const int64_t ld = rows_of(logits, "logits"), tokens = logits.size(0), groups = logits.size(1);
    if (choices < 1 || choices > groups)
        wrong_value("choices must be from 1 to the " + std::to_string(groups) + " experts");
    const at::Device device = logits.device();
    const int64_t need = ENTRY(ROUTE_SPACE, expert_route_workspace)(tokens, groups);
    const Routed r(device, tokens, groups, choices, need);
    const int st = call(device, [&] {
        return ENTRY(ROUTE, expert_route)(dt, tokens, groups, choices, normalize, logits.const_data_ptr(), ld, r.w(), r.e(),
                                          r.off(), r.ord(), r.work(), need, stream);
    });
    return st == GEMM_F32_SUCCESS ? results({r.weights, r.experts, r.offsets, r.order}) : status(st);
}

PyObject *route_balanced(PyObject *const *args)
{
    const Tensor &logits = tensor(args[0], "logits");
    const int64_t choices = integer(args[1]);
    const Tensor *bias = optional(args[2], "bias");
    const int scores = (int)integer(args[3]);
    const int64_t sets = integer(args[4]), kept = integer(args[5]);
    const int normalize = (int)integer(args[6]);
    const double scale = number(args[7]);
    void *const stream = stream_of(args[8]);
    const int dt = dtype_of(logits, "logits");
    on_gpu(logits, "logits");
    const int64_t ld = rows_of(logits, "logits"), tokens = logits.size(0), groups = logits.size(1);
    if (sets < 1 || groups % sets != 0) wrong_value("the " + std::to_string(groups) + " experts must be whole sets");
    if (kept < 1 || kept > sets) wrong_value("kept_sets must be from 1 to the " + std::to_string(sets) + " sets");
    const int64_t left = groups / sets * kept;
    if (choices < 1 || choices > left)
        wrong_value("choices must be from 1 to the " + std::to_string(left) + " experts of the sets that are kept");
    if (!(scale > 0.0 && scale <= 3.4028234663852886e38)) wrong_value("scale must be above 0 and finite");
    const at::Device device = logits.device();
    const float *bias_p = nullptr;
    if (bias) {
        if (bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != groups || !bias->is_contiguous())
            wrong_value("bias must be " + std::to_string(groups) + " contiguous float32 values");
        on(device, *bias, "bias");
        bias_p = static_cast<const float *>(bias->const_data_ptr());
    }
    const int64_t need = ENTRY(BALANCE_SPACE, expert_route_balanced_workspace)(tokens, groups);
    const Routed r(device, tokens, groups, choices, need);
    const int st = call(device, [&] {
        return ENTRY(BALANCE, expert_route_balanced)(dt, tokens, groups, choices, scores, sets, kept, normalize, (float)scale,
                                                     logits.const_data_ptr(), ld, bias_p, r.w(), r.e(), r.off(), r.ord(),
                                                     r.work(), need, stream);
    });
    return st == GEMM_F32_SUCCESS ? results({r.weights, r.experts, r.offsets, r.order}) : status(st);
}

// What the gradient of a routing reads: the logits, the routing's weights and
// experts, and the weights' gradient.
struct Routing {
    const Tensor &logits, &weights, &experts, &grad;
    int dt;
    int64_t ld, tokens, groups;
    at::Device device;
    Tensor d;

    Routing(PyObject *of_logits, PyObject *of_weights, PyObject *of_experts, PyObject *of_grad)
        : logits(tensor(of_logits, "logits")), weights(tensor(of_weights, "r.weights")),
          experts(tensor(of_experts, "r.experts")), grad(tensor(of_grad, "grad")), device(logits.device())
    {
        dt = dtype_of(logits, "logits");
        on_gpu(logits, "logits");
        ld = rows_of(logits, "logits");
        tokens = logits.size(0);
        groups = logits.size(1);
        if (weights.dim() != 2 || weights.size(0) != tokens || experts.sizes() != weights.sizes())
            wrong_value("r is not the routing of these logits");
        if (weights.scalar_type() != at::kFloat || experts.scalar_type() != at::kInt || !weights.is_contiguous() ||
            !experts.is_contiguous())
            wrong_value("r must hold contiguous float32 weights and int32 experts");
        if (grad.scalar_type() != at::kFloat || grad.sizes() != weights.sizes() || !grad.is_contiguous())
            wrong_value("grad must be a contiguous float32 " + shape_of(weights) + " tensor");
        on(device, weights, "r.weights");
        on(device, experts, "r.experts");
        on(device, grad, "grad");
        d = at::empty({tokens, groups}, logits.options());
    }
    const float *w() const { return static_cast<const float *>(weights.const_data_ptr()); }
    const int *e() const { return static_cast<const int *>(experts.const_data_ptr()); }
    const float *g() const { return static_cast<const float *>(grad.const_data_ptr()); }
};

PyObject *route_grad(PyObject *const *args)
{
    const int normalize = (int)integer(args[3]);
    void *const stream = stream_of(args[5]);
    const Routing r(args[0], args[1], args[2], args[4]);
    const int st = call(r.device, [&] {
        return ENTRY(ROUTE_GRAD, expert_route_grad)(r.dt, r.tokens, r.groups, r.weights.size(1), normalize,
                                                    r.logits.const_data_ptr(), r.ld, r.w(), r.e(), r.g(),
                                                    r.d.mutable_data_ptr(), r.groups, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(r.d) : status(st);
}

PyObject *route_balanced_grad(PyObject *const *args)
{
    const int scores = (int)integer(args[3]), normalize = (int)integer(args[4]);
    const double scale = number(args[5]);
    void *const stream = stream_of(args[7]);
    const Routing r(args[0], args[1], args[2], args[6]);
    const int st = call(r.device, [&] {
        return ENTRY(BALANCE_GRAD, expert_route_balanced_grad)(r.dt, r.tokens, r.groups, r.weights.size(1), scores, normalize,
                                                               (float)scale, r.logits.const_data_ptr(), r.ld, r.w(), r.e(),
                                                               r.g(), r.d.mutable_data_ptr(), r.groups, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(r.d) : status(st);
}

// A stack of matrices (batch, rows, cols), or one (rows, cols).
struct Stack {
    int64_t batch, rows, cols, ld, stride;

    Stack(const Tensor &t, const char *what, bool apart)
    {
        const int64_t d = t.dim();
        if (d != 2 && d != 3) wrong_value(std::string(what) + " must be 2-D or 3-D");
        batch = d == 3 ? t.size(0) : 1;
        rows = t.size(d - 2);
        cols = t.size(d - 1);
        if (rows < 1 || cols < 1) wrong_value(std::string(what) + " needs at least one row and column");
        if (cols > 1 && t.stride(d - 1) != 1) wrong_value(std::string(what) + " needs unit stride along its rows");
        ld = rows > 1 ? t.stride(d - 2) : cols;
        if (ld < cols) wrong_value(std::string(what) + " has overlapping rows");
        stride = batch > 1 ? t.stride(0) : 0;
        if (apart && batch > 1 && stride < (rows - 1) * ld + cols) wrong_value(std::string(what) + " has overlapping matrices");
    }
};

PyObject *orthogonalize(PyObject *const *args)
{
    const Tensor &x = tensor(args[0], "x");
    const int64_t steps = integer(args[1]);
    const double scale = number(args[3]);
    const Tensor *out = optional(args[4], "out");
    void *const stream = stream_of(args[5]);
    const int dt = dtype_of(x, "x");
    on_gpu(x, "x");
    const Stack s(x, "x", false);
    if (steps < 1 || steps > 64) wrong_value("steps must be from 1 to 64");
    if (!PyTuple_Check(args[2]) || PyTuple_GET_SIZE(args[2]) != 3 * steps) wrong_value("a step has three coefficients");
    float f[192];
    for (int64_t i = 0; i < 3 * steps; ++i) f[i] = (float)number(PyTuple_GET_ITEM(args[2], i));
    const Tensor y = result(out, x.sizes(), x.scalar_type(), x.device());
    const Stack t(y, "out", true);
    const int64_t need = ENTRY(ORTHO_SPACE, expert_orthogonalize_workspace)(dt, s.batch, s.rows, s.cols);
    Tensor space;
    if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(x.device()));
    const int st = call(x.device(), [&] {
        return ENTRY(ORTHO, expert_orthogonalize)(dt, s.batch, s.rows, s.cols, x.const_data_ptr(), s.ld, s.stride, (int)steps, f,
                                                  (float)scale, y.mutable_data_ptr(), t.ld, t.stride,
                                                  need ? space.mutable_data_ptr() : nullptr, need, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(y) : status(st);
}

// A function of `want` arguments, with its exceptions as Python's.
template <PyObject *(*F)(PyObject *const *), int WANT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != WANT) {
        PyErr_Format(PyExc_TypeError, "%d arguments are wanted, %zd given", WANT, n);
        return nullptr;
    }
    if (!g_entry[0]) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Wrong &w) {
        PyErr_SetString(w.type, w.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *bind(PyObject *, PyObject *addresses)
{
    void *found[COUNT];
    for (int i = 0; i < COUNT; ++i) {
        PyObject *const a = PyMapping_GetItemString(addresses, kNames[i]);
        if (!a) return nullptr;
        found[i] = PyLong_AsVoidPtr(a);
        Py_DECREF(a);
        if (PyErr_Occurred()) return nullptr;
    }
    std::copy(found, found + COUNT, g_entry);
    Py_RETURN_NONE;
}

#define FAST(name, want)                                                                            \
    {                                                                                               \
#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<&name, want>)), METH_FASTCALL, nullptr \
    }
PyMethodDef g_methods[] = {
    {"bind", bind, METH_O, "bind({name: address}) for every entry point of expert_ops.h"},
    FAST(grouped_linear, 7),
    FAST(grouped_weight_grad, 5),
    FAST(mx4_quantize, 2),
    FAST(mx4_dequantize, 6),
    FAST(mx4_linear, 9),
    FAST(route, 4),
    FAST(route_grad, 6),
    FAST(route_balanced, 9),
    FAST(route_balanced_grad, 8),
    FAST(int8_quantize, 2),
    FAST(int8_dequantize, 6),
    FAST(int8_linear, 9),
    FAST(orthogonalize, 6),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_expert_binding", "The expert-layer entry points, on tensors.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__expert_binding(void) { return PyModule_Create(&g_module); }
