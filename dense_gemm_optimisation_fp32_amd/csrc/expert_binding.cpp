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

enum { LINEAR, WEIGHT_GRAD, QUANTIZE, DEQUANTIZE, MX4_SPACE, MX4_LINEAR, ROUTE_SPACE, ROUTE, ROUTE_GRAD, COUNT };
const char *const kNames[COUNT] = {
    "expert_grouped_linear", "expert_grouped_weight_grad", "expert_mx4_quantize",   "expert_mx4_dequantize",
    "expert_mx4_workspace",  "expert_mx4_linear",          "expert_route_workspace", "expert_route",
    "expert_route_grad"};
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

PyObject *mx4_quantize(PyObject *const *args)
{
    const Tensor &x = tensor(args[0], "x");
    void *const stream = stream_of(args[1]);
    const int dt = dtype_of(x, "x");
    on_gpu(x, "x");
    if (x.dim() != 2) wrong_value("x must be 2-D");
    const int64_t r = x.size(0), k = x.size(1);
    if (k < 1) wrong_value("x needs at least one column");
    int layout = GEMM_F32_ROW_MAJOR;
    int64_t ld = r > 1 ? x.stride(0) : k;
    if (!(k == 1 || x.stride(1) == 1 || r == 0)) {
        if (!(r == 1 || x.stride(0) == 1)) wrong_value("x needs unit stride along one axis");
        layout = GEMM_F32_COL_MAJOR;
        ld = x.stride(1);
    }
    if (r > 0 && ld < (layout == GEMM_F32_COL_MAJOR ? r : k)) wrong_value("x has overlapping rows");
    const int64_t kb = (k + 127) / 128;
    const auto bytes = at::TensorOptions().dtype(at::kByte).device(x.device());
    const Tensor codes = at::empty({r, kb * 64}, bytes), scales = at::empty({kb, r, 4}, bytes);
    const int st = call(x.device(), [&] {
        return ENTRY(QUANTIZE, expert_mx4_quantize)(dt, r, k, x.const_data_ptr(), layout, r > 0 ? ld : k,
                                                    codes.mutable_data_ptr(), scales.mutable_data_ptr(), stream);
    });
    if (st != GEMM_F32_SUCCESS) return status(st);
    PyObject *const pair = PyTuple_New(2);
    if (!pair) throw python_error();
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(codes));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(scales));
    return pair;
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
    const Tensor &x = tensor(args[0], "x"), &codes = tensor(args[1], "w"), &scales = tensor(args[2], "w");
    const int64_t wk = integer(args[3]);
    const Tensor *offsets = optional(args[4], "offsets"), *bias = optional(args[5], "bias"), *out = optional(args[7], "out");
    const int act = (int)integer(args[6]);
    void *const stream = stream_of(args[8]);
    const int dt = dtype_of(x, "x");
    on_gpu(x, "x");
    const int64_t ldx = rows_of(x, "x"), m = x.size(0), k = x.size(1);
    if (k != wk) wrong_value("inner dimensions differ: x is " + shape_of(x) + ", w has " + std::to_string(wk) + " columns");
    const at::Device device = x.device();
    on(device, codes, "w");
    const bool many = codes.dim() == 3;
    const int64_t groups = many ? codes.size(0) : 1, n = codes.size(-2);
    if (many && !offsets) wrong_value("one matrix an expert needs offsets");
    if (!many && offsets) wrong_value("offsets need one matrix an expert");
    const int *const off = many ? offsets_of(*offsets, groups, device) : nullptr;
    const float *const bias_p = bias_of(bias, groups, n, !many, device);
    const Tensor y = result(out, {m, n}, x.scalar_type(), device);
    const int64_t ldy = rows_of(y, "out");
    const int64_t need = ENTRY(MX4_SPACE, expert_mx4_workspace)(m, n, k, groups);
    Tensor space;
    if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(device));
    const int st = call(device, [&] {
        return ENTRY(MX4_LINEAR, expert_mx4_linear)(dt, m, n, k, groups, x.const_data_ptr(), ldx, codes.const_data_ptr(),
                                                    scales.const_data_ptr(), off, bias_p, act, y.mutable_data_ptr(), ldy,
                                                    need ? space.mutable_data_ptr() : nullptr, need, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(y) : status(st);
}

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
    const auto floats = at::TensorOptions().dtype(at::kFloat).device(device);
    const auto ints = at::TensorOptions().dtype(at::kInt).device(device);
    const Tensor weights = at::empty({tokens, choices}, floats), experts = at::empty({tokens, choices}, ints);
    const Tensor offsets = at::empty({groups + 1}, ints), order = at::empty({tokens * choices}, ints);
    const int64_t need = ENTRY(ROUTE_SPACE, expert_route_workspace)(tokens, groups);
    Tensor space;
    if (need) space = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(device));
    const int st = call(device, [&] {
        return ENTRY(ROUTE, expert_route)(dt, tokens, groups, choices, normalize, logits.const_data_ptr(), ld,
                                          static_cast<float *>(weights.mutable_data_ptr()),
                                          static_cast<int *>(experts.mutable_data_ptr()),
                                          static_cast<int *>(offsets.mutable_data_ptr()),
                                          static_cast<int *>(order.mutable_data_ptr()),
                                          need ? space.mutable_data_ptr() : nullptr, need, stream);
    });
    if (st != GEMM_F32_SUCCESS) return status(st);
    PyObject *const all = PyTuple_New(4);
    if (!all) throw python_error();
    PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(weights));
    PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(experts));
    PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(offsets));
    PyTuple_SET_ITEM(all, 3, THPVariable_Wrap(order));
    return all;
}

PyObject *route_grad(PyObject *const *args)
{
    const Tensor &logits = tensor(args[0], "logits"), &weights = tensor(args[1], "r.weights");
    const Tensor &experts = tensor(args[2], "r.experts"), &grad = tensor(args[4], "grad");
    const int normalize = (int)integer(args[3]);
    void *const stream = stream_of(args[5]);
    const int dt = dtype_of(logits, "logits");
    on_gpu(logits, "logits");
    const int64_t ld = rows_of(logits, "logits"), tokens = logits.size(0), groups = logits.size(1);
    if (weights.dim() != 2 || weights.size(0) != tokens || experts.sizes() != weights.sizes())
        wrong_value("r is not the routing of these logits");
    if (weights.scalar_type() != at::kFloat || experts.scalar_type() != at::kInt || !weights.is_contiguous() ||
        !experts.is_contiguous())
        wrong_value("r must hold contiguous float32 weights and int32 experts");
    if (grad.scalar_type() != at::kFloat || grad.sizes() != weights.sizes() || !grad.is_contiguous())
        wrong_value("grad must be a contiguous float32 " + shape_of(weights) + " tensor");
    const at::Device device = logits.device();
    on(device, weights, "r.weights");
    on(device, experts, "r.experts");
    on(device, grad, "grad");
    const Tensor d = at::empty({tokens, groups}, logits.options());
    const int st = call(device, [&] {
        return ENTRY(ROUTE_GRAD, expert_route_grad)(dt, tokens, groups, weights.size(1), normalize, logits.const_data_ptr(),
                                                    ld, static_cast<const float *>(weights.const_data_ptr()),
                                                    static_cast<const int *>(experts.const_data_ptr()),
                                                    static_cast<const float *>(grad.const_data_ptr()),
                                                    d.mutable_data_ptr(), groups, stream);
    });
    return st == GEMM_F32_SUCCESS ? THPVariable_Wrap(d) : status(st);
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
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_expert_binding", "The expert-layer entry points, on tensors.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__expert_binding(void) { return PyModule_Create(&g_module); }
