// kt_ops_py.cpp -- the Python side of include/kt_ops.h for torch tensors: checks each tensor's
// device, type, shape and strides, and calls the C entry point with its address and pitch.
//
// A small call's time on the GPU (2 to 8 us) is below what the same checks take in Python: with
// them there, and ctypes, a layer norm call took its caller 6.4 us, of which the launch is 1.9.
// Compiled against torch's headers into a module of its own; the library itself knows no torch.
//
// Every function returns None, a status code other than KT_OK, or a text where a tensor does not
// fit (a KT_ERR_INVALID of its own).  No C++ exception leaves it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdio>
#include <string>

#include "kt_ops.h"

namespace {

struct Refusal {
    std::string text;
};
[[noreturn]] void refuse(const char* name, const char* what) { throw Refusal{std::string(name) + ": " + what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, "a torch tensor expected");
    return THPVariable_Unpack(o);
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

[[noreturn]] void misfit(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, c10::Device dev) {
    throw Refusal{std::string(name) + ": expected " + c10::toString(dtype) + " " + shape_text(shape) + " on " + dev.str() +
                  ", got " + c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " + t.device().str() +
                  ", strides " + shape_text(t.strides())};
}

struct Rows {
    void* p;
    int64_t ld;
};
// A matrix with consecutive elements in a row, and its pitch (a single row's is never used: it is
// rounded up to `unit` elements).
Rows rows(const at::Tensor& t, const char* name, int64_t m, int64_t n, at::ScalarType dtype, c10::Device dev, int64_t unit = 1) {
    if (t.dim() != 2 || t.size(0) != m || t.size(1) != n || t.scalar_type() != dtype || t.device() != dev)
        misfit(name, t, {m, n}, dtype, dev);
    if (n > 1 && t.stride(1) != 1) refuse(name, "the elements of a row must be consecutive");
    int64_t ld = t.stride(0);
    if (m > 1 && ld < n) refuse(name, "rows overlap");
    if (m <= 1) ld = (std::max(ld, n) + unit - 1) / unit * unit;
    return {t.data_ptr(), ld};
}

// A contiguous tensor's address; None: null.
void* whole(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::Device dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.sizes() != shape || t.scalar_type() != dtype || t.device() != dev || !t.is_contiguous()) misfit(name, t, shape, dtype, dev);
    return t.data_ptr();
}

kt_dtype code(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kHalf) return KT_F16;
    if (t.scalar_type() == at::kBFloat16) return KT_BF16;
    refuse(name, "float16 or bfloat16 expected");
}

const at::Tensor& matrix(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) refuse(name, "a matrix expected");
    return t;
}

// The stream to launch on: torch's current one of the tensors' device, which has to be the current
// device, unless the caller names another (an address, or an object with a cuda_stream).
void* stream_of(PyObject* o, c10::Device dev) {
    if (!dev.is_cuda()) throw Refusal{"CUDA tensors expected, got " + dev.str()};
    if (dev.index() != c10::cuda::current_device())
        throw Refusal{"the tensors are on " + dev.str() + ", the current device is cuda:" + std::to_string((int)c10::cuda::current_device())};
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    PyObject* n = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    void* s = n ? PyLong_AsVoidPtr(n) : nullptr;
    Py_XDECREF(n);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Refusal{"stream: None, an address or a torch stream expected"};
    }
    return s;
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(name, "an integer expected");
    }
    return v;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    std::string text;
    try {
        if (n != want) throw Refusal{std::to_string(want) + " arguments expected, got " + std::to_string(n)};
        const kt_status s = f();
        if (s == KT_OK) Py_RETURN_NONE;
        return PyLong_FromLong(s);
    } catch (const Refusal& r) {
        text = r.text;
    } catch (const std::exception& e) {
        text = e.what();
    } catch (...) {
        text = "unknown exception";
    }
    return PyUnicode_FromStringAndSize(text.data(), (Py_ssize_t)text.size());
}

// layernorm_forward(X, gamma, beta, eps, Y, mean, rstd, stream)
PyObject* layernorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const at::Tensor& X = matrix(a[0], "X");
        const int64_t M = X.size(0), D = X.size(1);
        const c10::Device dev = X.device();
        const at::ScalarType dt = X.scalar_type();
        const kt_dtype c = code(X, "X");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("eps", "a number expected");
        }
        const Rows x = rows(X, "X", M, D, dt, dev), y = rows(tensor(a[4], "Y"), "Y", M, D, dt, dev);
        void* gamma = whole(a[1], "gamma", {D}, dt, dev);
        void* beta = whole(a[2], "beta", {D}, dt, dev);
        void* mean = whole(a[5], "mean", {M}, at::kFloat, dev);
        void* rstd = whole(a[6], "rstd", {M}, at::kFloat, dev);
        void* s = stream_of(a[7], dev);
        return kt_layernorm_forward(M, D, c, x.p, x.ld, gamma, beta, (float)eps, y.p, y.ld, (float*)mean, (float*)rstd, s);
    });
}

// layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace, stream)
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor& X = matrix(a[1], "X");
        const int64_t M = X.size(0), D = X.size(1);
        const c10::Device dev = X.device();
        const at::ScalarType dt = X.scalar_type();
        const kt_dtype c = code(X, "X");
        const Rows x = rows(X, "X", M, D, dt, dev), dy = rows(tensor(a[0], "dY"), "dY", M, D, dt, dev),
                   dx = rows(tensor(a[5], "dX"), "dX", M, D, dt, dev);
        void* gamma = whole(a[2], "gamma", {D}, dt, dev);
        void* mean = whole(a[3], "mean", {M}, at::kFloat, dev);
        void* rstd = whole(a[4], "rstd", {M}, at::kFloat, dev);
        void* dgamma = whole(a[6], "dgamma", {D}, at::kFloat, dev);
        void* dbeta = whole(a[7], "dbeta", {D}, at::kFloat, dev);
        void* ws = nullptr;
        size_t bytes = 0;
        if (a[8] != Py_None) {
            const at::Tensor& w = tensor(a[8], "workspace");
            if (w.device() != dev || !w.is_contiguous()) refuse("workspace", "a contiguous tensor on the other tensors' device expected");
            ws = w.data_ptr();
            bytes = w.nbytes();
        }
        void* s = stream_of(a[9], dev);
        return kt_layernorm_backward(M, D, c, dy.p, dy.ld, x.p, x.ld, gamma, (const float*)mean, (const float*)rstd, dx.p, dx.ld,
                                     (float*)dgamma, (float*)dbeta, ws, bytes, s);
    });
}

// quantize_rows(X, Q, scale, act, stream)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const at::Tensor &X = matrix(a[0], "X"), &Q = matrix(a[1], "Q");
        const int64_t M = Q.size(0), K = Q.size(1), act = integer(a[3], "act");
        const c10::Device dev = Q.device();
        const kt_dtype c = code(X, "X");
        const Rows x = rows(X, "X", M, act == KT_ACT_GEGLU ? 2 * K : K, X.scalar_type(), dev), q = rows(Q, "Q", M, K, at::kChar, dev);
        void* scale = whole(a[2], "scale", {M}, at::kFloat, dev);
        void* s = stream_of(a[4], dev);
        return kt_quantize_rows(M, K, c, (kt_act)act, x.p, x.ld, (int8_t*)q.p, q.ld, (float*)scale, s);
    });
}

// linear_i8(Q, scale_x, W, scale_w, bias, Y, stream)
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const at::Tensor &Q = matrix(a[0], "Q"), &W = matrix(a[2], "W"), &Y = matrix(a[5], "Y");
        const int64_t M = Q.size(0), K = Q.size(1), N = W.size(0);
        const c10::Device dev = Q.device();
        const kt_dtype c = code(Y, "Y");
        const Rows q = rows(Q, "Q", M, K, at::kChar, dev, 16), w = rows(W, "W", N, K, at::kChar, dev, 16),
                   y = rows(Y, "Y", M, N, Y.scalar_type(), dev);
        void* sx = whole(a[1], "scale_x", {M}, at::kFloat, dev);
        void* sw = whole(a[3], "scale_w", {N}, at::kFloat, dev);
        void* bias = whole(a[4], "bias", {N}, Y.scalar_type(), dev);
        void* s = stream_of(a[6], dev);
        return kt_linear_i8(M, N, K, c, (const int8_t*)q.p, q.ld, (const int8_t*)w.p, w.ld, (const float*)sx, (const float*)sw, bias,
                            y.p, y.ld, s);
    });
}

// moe_run(plan, (dtype, D, F, F_up, E, top_k), X, W_router, W_up, W_down, Y, b_up, b_down, R, ids, weights, stream)
PyObject* moe_run(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        void* plan = PyLong_AsVoidPtr(a[0]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            refuse("plan", "a handle expected");
        }
        if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 6) refuse("sizes", "a tuple of six expected");
        int64_t z[6];
        for (int i = 0; i < 6; ++i) z[i] = integer(PyTuple_GET_ITEM(a[1], i), "sizes");
        const at::ScalarType dt = z[0] == KT_BF16 ? at::kBFloat16 : at::kHalf;
        const int64_t D = z[1], F = z[2], F_up = z[3], E = z[4], k = z[5];
        const at::Tensor& X = matrix(a[2], "X");
        const int64_t T = X.size(0);
        const c10::Device dev = X.device();
        kt_moe_tensors t = {};
        const Rows x = rows(X, "X", T, D, dt, dev, 8);
        t.tokens = T;
        t.X = x.p;
        t.ldx = x.ld;
        t.W_router = whole(a[3], "W_router", {E, D}, dt, dev);
        t.W_up = whole(a[4], "W_up", {E, F_up, D}, dt, dev);
        t.W_down = whole(a[5], "W_down", {E, D, F}, dt, dev);
        t.Y = whole(a[6], "Y", {T, D}, dt, dev);
        t.b_up = whole(a[7], "b_up", {E, F_up}, dt, dev);
        t.b_down = whole(a[8], "b_down", {E, D}, dt, dev);
        t.R = whole(a[9], "R", {T, D}, dt, dev);
        t.ids = (int32_t*)whole(a[10], "ids", {T, k}, at::kInt, dev);
        t.weights = (float*)whole(a[11], "weights", {T, k}, at::kFloat, dev);
        void* s = stream_of(a[12], dev);
        return kt_moe_run((kt_moe_plan_t)plan, &t, s);
    });
}

PyMethodDef kMethods[] = {
    {"layernorm_forward", (PyCFunction)(void*)layernorm_forward, METH_FASTCALL, nullptr},
    {"layernorm_backward", (PyCFunction)(void*)layernorm_backward, METH_FASTCALL, nullptr},
    {"quantize_rows", (PyCFunction)(void*)quantize_rows, METH_FASTCALL, nullptr},
    {"linear_i8", (PyCFunction)(void*)linear_i8, METH_FASTCALL, nullptr},
    {"moe_run", (PyCFunction)(void*)moe_run, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kt_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kt_ops(void) { return PyModule_Create(&kModule); }
