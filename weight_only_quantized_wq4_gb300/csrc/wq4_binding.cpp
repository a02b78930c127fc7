// Argument checks and marshalling of the 8-bit row operators' Python calls. A decode step makes such a
// call every few microseconds and its kernels take one or two, so the call itself decides: read
// through Python, a tensor's type, device, sizes, strides and pointer take about half a microsecond,
// and a call has five to seven tensors (norm: 8.0 us a call in Python, 2.3 us here, of which 1.9 us are the
// launch). Nothing is computed here: each function checks its tensors, passes pointers, sizes and
// torch's current stream on to the C ABI and returns its status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include <cstdio>

#include "wq4.h"

namespace {

decltype(&wq4_add_rmsnorm_quant) g_norm = nullptr;
decltype(&wq4_silu_mul_quant) g_gated = nullptr;
decltype(&wq4_block_mm) g_mm = nullptr;
decltype(&wq4_token_logprobs) g_logprobs = nullptr;

bool refuse(const char* name, const char* what) {
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, what);
    return false;
}

// The tensor in `o`, of type `type`, on CUDA device `dev` (-1: any, and dev becomes its own).
const at::Tensor* tensor(PyObject* o, const char* name, at::ScalarType type, int* dev) {
    if (!THPVariable_Check(o)) return refuse(name, "a tensor"), nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type) {
        char text[96];
        std::snprintf(text, sizeof(text), "of type %s", c10::toString(type));
        return refuse(name, text), nullptr;
    }
    if (!t.is_cuda() || (*dev >= 0 && t.get_device() != *dev))
        return refuse(name, "a CUDA tensor on the device of the others"), nullptr;
    *dev = static_cast<int>(t.get_device());
    return &t;
}

bool shaped(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
    if (t.dim() == 2 && t.size(0) == rows && t.size(1) == cols) return true;
    char text[96];
    std::snprintf(text, sizeof(text), "of shape [%lld][%lld]", static_cast<long long>(rows), static_cast<long long>(cols));
    return refuse(name, text);
}

struct Rows {
    void* p = nullptr;
    long long ld = 0;       // row stride in elements
};

// The rows of a 2-D tensor, each contiguous.
bool rows_of(const at::Tensor& t, const char* name, Rows* r) {
    if (t.size(1) > 1 && t.stride(1) != 1) return refuse(name, "contiguous along its rows");
    r->p = t.data_ptr();
    r->ld = t.size(0) > 1 ? t.stride(0) : (t.size(1) + 15) / 16 * 16;   // (a single row's stride is never used)
    return true;
}

bool rows(PyObject* o, const char* name, int64_t n, int64_t cols, at::ScalarType type, int dev, Rows* r) {
    const at::Tensor* t = tensor(o, name, type, &dev);
    return t && shaped(*t, name, n, cols) && rows_of(*t, name, r);
}

// A contiguous tensor of n elements (null for None).
bool vector(PyObject* o, const char* name, int64_t n, at::ScalarType type, int dev, void** p) {
    if (o == Py_None) return true;
    const at::Tensor* t = tensor(o, name, type, &dev);
    if (!t) return false;
    if (t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1)) {
        char text[96];
        std::snprintf(text, sizeof(text), "a contiguous tensor of %lld elements", static_cast<long long>(n));
        return refuse(name, text);
    }
    *p = t->data_ptr();
    return true;
}

// The first argument of a call: a 2-D CUDA tensor, which sets the device and (one of three) the type.
const at::Tensor* leading(PyObject* o, const char* name, bool fp32, int* dtype, int* dev) {
    if (!THPVariable_Check(o)) return refuse(name, "a tensor"), nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    switch (t.scalar_type()) {
        case at::kBFloat16: *dtype = WQ4_BF16; break;
        case at::kHalf: *dtype = WQ4_FP16; break;
        case at::kFloat:
            *dtype = WQ4_FP32;
            if (fp32) break;
            [[fallthrough]];
        default: return refuse(name, fp32 ? "bfloat16, float16 or float32" : "bfloat16 or float16"), nullptr;
    }
    if (t.dim() != 2 || !t.is_cuda()) return refuse(name, "a 2-D CUDA tensor"), nullptr;
    *dev = static_cast<int>(t.get_device());
    return &t;
}

bool fits(const char* name, int64_t n) {
    return (n >= -0x7fffffff && n <= 0x7fffffff) || refuse(name, "smaller than 2^31 in each dimension");
}

wq4_stream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

bool count(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return false;
}

// add_rmsnorm_quant(x, weight, residual | None, eps, q, scales, residual_out | None, y | None) -> status
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 8)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* x = leading(a[0], "x", false, &dtype, &dev);
    if (!x) return nullptr;
    const int64_t T = x->size(0), D = x->size(1);
    const at::ScalarType half = x->scalar_type();
    Rows rx, rr, ro, ry, rq, rs;
    void* w = nullptr;
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (a[1] == Py_None) return refuse("weight", "a tensor"), nullptr;
    if (!fits("x", T) || !fits("x", D) || !rows_of(*x, "x", &rx) || !vector(a[1], "weight", D, half, dev, &w) ||
        (a[2] != Py_None && !rows(a[2], "residual", T, D, half, dev, &rr)) ||
        !rows(a[4], "q", T, D, at::kFloat8_e4m3fn, dev, &rq) || !rows(a[5], "scales", blocks(D), T, at::kFloat, dev, &rs) ||
        (a[6] != Py_None && !rows(a[6], "residual_out", T, D, half, dev, &ro)) ||
        (a[7] != Py_None && !rows(a[7], "y", T, D, half, dev, &ry)))
        return nullptr;
    return PyLong_FromLong(g_norm(rx.p, rx.ld, rr.p, rr.ld, w, static_cast<int>(T), static_cast<int>(D),
                                  static_cast<float>(eps), dtype, ro.p, ro.ld, ry.p, ry.ld, rq.p, rq.ld,
                                  static_cast<float*>(rs.p), rs.ld, stream(dev)));
}

// silu_mul_quant(x, q, scales) -> status
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 3)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* x = leading(a[0], "x", false, &dtype, &dev);
    if (!x) return nullptr;
    const int64_t T = x->size(0), D = x->size(1) / 2;
    Rows rx, rq, rs;
    if (x->size(1) % 2) return refuse("x", "of two halves, gate and up"), nullptr;
    if (!fits("x", T) || !fits("x", D) || !rows_of(*x, "x", &rx) || !rows(a[1], "q", T, D, at::kFloat8_e4m3fn, dev, &rq) ||
        !rows(a[2], "scales", blocks(D), T, at::kFloat, dev, &rs))
        return nullptr;
    return PyLong_FromLong(g_gated(rx.p, rx.ld, static_cast<int>(T), static_cast<int>(D), dtype, rq.p, rq.ld,
                                   static_cast<float*>(rs.p), rs.ld, stream(dev)));
}

// block_mm(q, scales, W, W_scales, out) -> status
PyObject* mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 5)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* y = leading(a[4], "out", true, &dtype, &dev);
    const at::Tensor* q = y ? tensor(a[0], "q", at::kFloat8_e4m3fn, &dev) : nullptr;
    const at::Tensor* w = q ? tensor(a[2], "W", at::kFloat8_e4m3fn, &dev) : nullptr;
    if (!w) return nullptr;
    if (q->dim() != 2 || w->dim() != 2) return refuse("q and W", "2-D"), nullptr;
    const int64_t M = q->size(0), K = q->size(1), N = w->size(0);
    Rows rq, rs, rw, rws, ry;
    if (!fits("q", M) || !fits("q", K) || !fits("W", N) || !rows_of(*q, "q", &rq) ||
        !rows(a[1], "scales", blocks(K), M, at::kFloat, dev, &rs) || !shaped(*w, "W", N, K) || !rows_of(*w, "W", &rw) ||
        !rows(a[3], "W_scales", blocks(N), blocks(K), at::kFloat, dev, &rws) || !shaped(*y, "out", M, N) ||
        !rows_of(*y, "out", &ry))
        return nullptr;
    return PyLong_FromLong(g_mm(rq.p, rq.ld, static_cast<const float*>(rs.p), rs.ld, rw.p, rw.ld,
                                static_cast<const float*>(rws.p), rws.ld, ry.p, ry.ld, static_cast<int>(M),
                                static_cast<int>(N), static_cast<int>(K), dtype, stream(dev)));
}

// token_logprobs(logits, tokens | None, top_k, logprobs | None, entropy, top_ids | None, top_logprobs | None) -> status
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 7)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* x = leading(a[0], "logits", true, &dtype, &dev);
    if (!x) return nullptr;
    const int64_t T = x->size(0), V = x->size(1);
    const long k = PyLong_AsLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Rows rx, ri, rl;
    void *tok = nullptr, *lp = nullptr, *ent = nullptr;
    if (!fits("logits", T) || !fits("logits", V) || !fits("top_k", k) || !rows_of(*x, "logits", &rx) ||
        !vector(a[1], "tokens", T, at::kLong, dev, &tok) || !vector(a[3], "logprobs", T, at::kFloat, dev, &lp) ||
        !vector(a[4], "entropy", T, at::kFloat, dev, &ent) ||
        (a[5] != Py_None && !rows(a[5], "top_ids", T, k, at::kInt, dev, &ri)) ||
        (a[6] != Py_None && !rows(a[6], "top_logprobs", T, k, at::kFloat, dev, &rl)))
        return nullptr;
    if (T > 1 && ((ri.p && ri.ld != k) || (rl.p && rl.ld != k)))
        return refuse("top_ids and top_logprobs", "contiguous"), nullptr;
    return PyLong_FromLong(g_logprobs(rx.p, T > 1 ? rx.ld : V, static_cast<const long long*>(tok), static_cast<int>(T),
                                      static_cast<int>(V), dtype, static_cast<int>(k), static_cast<float*>(lp),
                                      static_cast<float*>(ent), static_cast<int*>(ri.p), static_cast<float*>(rl.p),
                                      stream(dev)));
}

// bind(norm, gated, mm, logprobs): the addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 4)) return nullptr;
    void* p[4];
    for (int i = 0; i < 4; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) refuse("each address", "non-zero");
            return nullptr;
        }
    g_norm = reinterpret_cast<decltype(g_norm)>(p[0]);
    g_gated = reinterpret_cast<decltype(g_gated)>(p[1]);
    g_mm = reinterpret_cast<decltype(g_mm)>(p[2]);
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(p[3]);
    Py_RETURN_NONE;
}

// A C++ exception (torch's accessors throw on misuse) becomes a Python one.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<norm>("add_rmsnorm_quant"), method<gated>("silu_mul_quant"), method<mm>("block_mm"),
                           method<logprobs>("token_logprobs"), method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_wq4_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wq4_binding(void) { return PyModule_Create(&g_module); }
