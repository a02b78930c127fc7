// Argument checks and marshalling of the 8-bit row operators' and the attention operators' Python calls. A decode step makes such a
// call every few microseconds and its kernels take one or two, so the call itself decides: read
// through Python, a tensor's type, device, sizes, strides and pointer take about half a microsecond,
// and a call has five to seven tensors (norm: 8.0 us a call in Python, 2.3 us here, of which 1.9 us are the
// launch). Nothing is computed here: each function checks its tensors, passes pointers, sizes and
// torch's current stream on to the C ABI and returns its status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdio>

#include "wq4.h"

namespace {

decltype(&wq4_add_rmsnorm_quant) g_norm = nullptr;
decltype(&wq4_silu_mul_quant) g_gated = nullptr;
decltype(&wq4_block_mm) g_mm = nullptr;
decltype(&wq4_token_logprobs) g_logprobs = nullptr;
decltype(&wq4_rope_append) g_append = nullptr;
decltype(&wq4_tree_attention) g_attention = nullptr;
decltype(&wq4_verify_drafts) g_verify = nullptr;

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

// A [tokens][heads][D] tensor whose heads are contiguous rows.
struct Heads {
    void* p = nullptr;
    long long ts = 0, hs = 0;
};
bool heads_of(PyObject* o, const char* name, int64_t T, int64_t H, int64_t D, at::ScalarType type, int dev, Heads* r) {
    const at::Tensor* t = tensor(o, name, type, &dev);
    if (!t) return false;
    if (t->dim() != 3 || t->size(0) != T || t->size(1) != H || t->size(2) != D) {
        char text[96];
        std::snprintf(text, sizeof(text), "of shape [%lld][%lld][%lld]", static_cast<long long>(T), static_cast<long long>(H),
                      static_cast<long long>(D));
        return refuse(name, text);
    }
    if (D > 1 && t->stride(2) != 1) return refuse(name, "contiguous along its heads");
    *r = {t->data_ptr(), t->stride(0), t->stride(1)};
    return true;
}

// The caches, [pages][page_size][heads][D] each.
bool cache_of(PyObject* ko, PyObject* vo, int64_t H, int64_t D, at::ScalarType type, int dev, wq4_kv_cache* c) {
    const at::Tensor* k = tensor(ko, "k_cache", type, &dev);
    const at::Tensor* v = k ? tensor(vo, "v_cache", type, &dev) : nullptr;
    if (!v) return false;
    if (k->dim() != 4 || k->size(2) != H || k->size(3) != D || v->sizes() != k->sizes())
        return refuse("k_cache and v_cache", "of shape [pages][page_size][kv heads][D]");
    if (D > 1 && (k->stride(3) != 1 || v->stride(3) != 1)) return refuse("k_cache and v_cache", "contiguous along their heads");
    if (!fits("k_cache", k->size(0)) || !fits("k_cache", k->size(1))) return false;
    *c = {k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), k->stride(2), v->stride(0), v->stride(1), v->stride(2),
          static_cast<int>(k->size(0)), static_cast<int>(k->size(1))};
    return true;
}

// The first argument of a call: a 3-D CUDA tensor, which sets the device and the type.
const at::Tensor* leading_heads(PyObject* o, const char* name, int* dtype, int* dev) {
    if (!THPVariable_Check(o)) return refuse(name, "a tensor"), nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf) return refuse(name, "bfloat16 or float16"), nullptr;
    *dtype = t.scalar_type() == at::kBFloat16 ? WQ4_BF16 : WQ4_FP16;
    if (t.dim() != 3 || !t.is_cuda()) return refuse(name, "a 3-D CUDA tensor"), nullptr;
    *dev = static_cast<int>(t.get_device());
    for (int i = 0; i < 3; ++i)
        if (!fits(name, t.size(i))) return nullptr;
    return &t;
}

// The tensors' device is made the current one for the call.
using Guard = c10::cuda::CUDAGuard;

// rope_append(q | None, k, v, k_cache, v_cache, slots, positions | None, inv_freq | None, q_weight | None, k_weight | None, eps,
// interleaved, q_out | None) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 13)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* k = leading_heads(a[1], "k", &dtype, &dev);
    if (!k) return nullptr;
    const int64_t T = k->size(0), Hk = k->size(1), D = k->size(2);
    const at::ScalarType half = k->scalar_type();
    int64_t Hq = 0, pairs = 0;
    Heads q, kh, v, qo;
    wq4_kv_cache cache;
    void *slots = nullptr, *pos = nullptr, *freq = nullptr, *qw = nullptr, *kw = nullptr;
    const double eps = PyFloat_AsDouble(a[10]);
    const int interleaved = eps == -1.0 && PyErr_Occurred() ? -1 : PyObject_IsTrue(a[11]);
    if (interleaved < 0) return nullptr;
    if (a[0] != Py_None) {
        if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 3) return refuse("q", "a 3-D tensor"), nullptr;
        Hq = THPVariable_Unpack(a[0]).size(1);
    }
    if (a[7] != Py_None) {
        if (!THPVariable_Check(a[7]) || THPVariable_Unpack(a[7]).dim() != 1) return refuse("inv_freq", "a 1-D tensor"), nullptr;
        pairs = THPVariable_Unpack(a[7]).size(0);
    }
    if ((a[6] != Py_None) != (a[7] != Py_None)) return refuse("positions and inv_freq", "given together"), nullptr;
    if (a[5] == Py_None) return refuse("slots", "a tensor"), nullptr;
    if (!heads_of(a[1], "k", T, Hk, D, half, dev, &kh) || !heads_of(a[2], "v", T, Hk, D, half, dev, &v) ||
        (a[0] != Py_None && (!fits("q", Hq) || !heads_of(a[0], "q", T, Hq, D, half, dev, &q) ||
                             !heads_of(a[12], "q_out", T, Hq, D, half, dev, &qo))) ||
        !cache_of(a[3], a[4], Hk, D, half, dev, &cache) || !vector(a[5], "slots", T, at::kLong, dev, &slots) ||
        !vector(a[6], "positions", T, at::kLong, dev, &pos) || !fits("inv_freq", 2 * pairs) ||
        !vector(a[7], "inv_freq", pairs, at::kFloat, dev, &freq) || !vector(a[8], "q_weight", D, half, dev, &qw) ||
        !vector(a[9], "k_weight", D, half, dev, &kw))
        return nullptr;
    const Guard guard(static_cast<c10::DeviceIndex>(dev));
    return PyLong_FromLong(g_append(q.p, q.ts, q.hs, kh.p, kh.ts, kh.hs, v.p, v.ts, v.hs, static_cast<int>(T), static_cast<int>(Hq),
                                    static_cast<int>(Hk), static_cast<int>(D), dtype, qw, kw, static_cast<float>(eps),
                                    static_cast<const long long*>(pos), static_cast<const float*>(freq), static_cast<int>(2 * pairs),
                                    interleaved, qo.p, qo.ts, qo.hs, &cache, static_cast<const long long*>(slots), stream(dev)));
}

// tree_attention(q, k_cache, v_cache, page_table, starts, context, max_tokens, mask | None, scale, out, lse | None, workspace) -> status
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 12)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* q = leading_heads(a[0], "q", &dtype, &dev);
    const at::Tensor* table = q ? tensor(a[3], "page_table", at::kInt, &dev) : nullptr;
    const at::Tensor* k = table ? tensor(a[1], "k_cache", q->scalar_type(), &dev) : nullptr;
    if (!k) return nullptr;
    if (k->dim() != 4) return refuse("k_cache", "4-D"), nullptr;
    if (table->dim() != 2) return refuse("page_table", "2-D"), nullptr;
    const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hk = k->size(2), B = table->size(0);
    const at::ScalarType half = q->scalar_type();
    const long most = PyLong_AsLong(a[6]);
    const double scale = PyErr_Occurred() ? 0 : PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) return nullptr;
    Heads qh, oh;
    Rows rt, rm;
    int64_t words = 0;
    void *starts = nullptr, *context = nullptr, *lse = nullptr, *space = nullptr;
    wq4_kv_cache cache;
    if (a[4] == Py_None || a[5] == Py_None) return refuse("starts and context", "tensors"), nullptr;
    if (!fits("max_tokens", most) || !fits("page_table", B) || !fits("page_table", table->size(1)) || !rows_of(*table, "page_table", &rt) ||
        !heads_of(a[0], "q", T, Hq, D, half, dev, &qh) || !heads_of(a[9], "out", T, Hq, D, half, dev, &oh) ||
        !cache_of(a[1], a[2], Hk, D, half, dev, &cache) || !vector(a[4], "starts", B + 1, at::kInt, dev, &starts) ||
        !vector(a[5], "context", B, at::kInt, dev, &context))
        return nullptr;
    if (B <= 1) rt.ld = table->size(1);
    if (!fits("page_table", rt.ld)) return nullptr;
    if (a[7] != Py_None) {
        const at::Tensor* m = tensor(a[7], "mask", at::kLong, &dev);
        if (!m) return nullptr;
        if (m->dim() != 2 || m->size(0) != T || !m->is_contiguous()) return refuse("mask", "contiguous, of shape [tokens][words]"), nullptr;
        words = m->size(1);
        if (!fits("mask", words)) return nullptr;
        if (words * 64 < most) return refuse("mask", "of a word for each 64 of max_tokens"), nullptr;
        rm.p = m->data_ptr();
        if (!rm.p && T > 0) return refuse("mask", "a tensor"), nullptr;
    }
    if (a[10] != Py_None) {
        const at::Tensor* l = tensor(a[10], "lse", at::kFloat, &dev);
        if (!l) return nullptr;
        if (!shaped(*l, "lse", T, Hq)) return nullptr;
        if (!l->is_contiguous()) return refuse("lse", "contiguous"), nullptr;
        lse = l->data_ptr();
    }
    const at::Tensor* ws = tensor(a[11], "workspace", at::kByte, &dev);
    if (!ws) return nullptr;
    if (!ws->is_contiguous()) return refuse("workspace", "contiguous"), nullptr;
    space = ws->data_ptr();
    const Guard guard(static_cast<c10::DeviceIndex>(dev));
    return PyLong_FromLong(g_attention(qh.p, qh.ts, qh.hs, &cache, static_cast<const int*>(rt.p), static_cast<int>(rt.ld),
                                       static_cast<int>(table->size(1)), static_cast<const int*>(starts), static_cast<const int*>(context),
                                       static_cast<int>(B), static_cast<int>(T), static_cast<int>(most), static_cast<int>(Hq),
                                       static_cast<int>(Hk), static_cast<int>(D), dtype, static_cast<float>(scale),
                                       static_cast<const unsigned long long*>(rm.p), static_cast<int>(words), oh.p, oh.ts, oh.hs,
                                       static_cast<float*>(lse), space, static_cast<size_t>(ws->numel()), stream(dev)));
}

// verify_drafts(logits, tokens, parents, starts, uniforms, final_uniforms, max_tokens, draft_probs | None, temperature | None, accepted,
// path, next_tokens) -> status
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 12)) return nullptr;
    int dtype = 0, dev = -1;
    const at::Tensor* x = leading(a[0], "logits", true, &dtype, &dev);
    const at::Tensor* last = x ? tensor(a[11], "next_tokens", at::kLong, &dev) : nullptr;
    if (!last) return nullptr;
    if (last->dim() != 1) return refuse("next_tokens", "1-D"), nullptr;
    const int64_t T = x->size(0), V = x->size(1), B = last->size(0);
    const long most = PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return nullptr;
    if (!fits("max_tokens", most)) return nullptr;
    Rows rx, rq, rp;
    void *tokens = nullptr, *parents = nullptr, *starts = nullptr, *u = nullptr, *uf = nullptr, *heat = nullptr, *kept = nullptr, *next = nullptr;
    for (const int i : {1, 2, 3, 4, 5, 9})
        if (a[i] == Py_None) return refuse("tokens, parents, starts, uniforms, final_uniforms and accepted", "tensors"), nullptr;
    if (!fits("logits", T) || !fits("logits", V) || !fits("next_tokens", B) || !rows_of(*x, "logits", &rx) ||
        !vector(a[1], "tokens", T, at::kLong, dev, &tokens) || !vector(a[2], "parents", T, at::kInt, dev, &parents) ||
        !vector(a[3], "starts", B + 1, at::kInt, dev, &starts) || !vector(a[4], "uniforms", T, at::kFloat, dev, &u) ||
        !vector(a[5], "final_uniforms", B, at::kFloat, dev, &uf) ||
        (a[7] != Py_None && !rows(a[7], "draft_probs", T, V, at::kFloat, dev, &rq)) || !vector(a[8], "temperature", B, at::kFloat, dev, &heat) ||
        !vector(a[9], "accepted", B, at::kInt, dev, &kept) || !rows(a[10], "path", B, most > 1 ? most - 1 : 1, at::kInt, dev, &rp) ||
        !vector(a[11], "next_tokens", B, at::kLong, dev, &next))
        return nullptr;
    if (B <= 1) rp.ld = most > 1 ? most - 1 : 1;
    if (!fits("path", rp.ld)) return nullptr;
    const Guard guard(static_cast<c10::DeviceIndex>(dev));
    return PyLong_FromLong(g_verify(rx.p, T > 1 ? rx.ld : V, static_cast<const long long*>(tokens), static_cast<const int*>(parents),
                                    static_cast<const int*>(starts), static_cast<int>(B), static_cast<int>(T), static_cast<int>(most),
                                    static_cast<int>(V), dtype, static_cast<const float*>(rq.p), T > 1 ? rq.ld : V,
                                    static_cast<const float*>(heat), static_cast<const float*>(u), static_cast<const float*>(uf),
                                    static_cast<int*>(kept), static_cast<int*>(rp.p), static_cast<int>(rp.ld),
                                    static_cast<long long*>(next), stream(dev)));
}

// bind(norm, gated, mm, logprobs, append, attention, verify): the addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr int kFns = 7;
    if (!count(n, kFns)) return nullptr;
    void* p[kFns];
    for (int i = 0; i < kFns; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) refuse("each address", "non-zero");
            return nullptr;
        }
    g_norm = reinterpret_cast<decltype(g_norm)>(p[0]);
    g_gated = reinterpret_cast<decltype(g_gated)>(p[1]);
    g_mm = reinterpret_cast<decltype(g_mm)>(p[2]);
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(p[3]);
    g_append = reinterpret_cast<decltype(g_append)>(p[4]);
    g_attention = reinterpret_cast<decltype(g_attention)>(p[5]);
    g_verify = reinterpret_cast<decltype(g_verify)>(p[6]);
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
                           method<logprobs>("token_logprobs"), method<append>("rope_append"),
                           method<attention>("tree_attention"), method<verify>("verify_drafts"), method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_wq4_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wq4_binding(void) { return PyModule_Create(&g_module); }
