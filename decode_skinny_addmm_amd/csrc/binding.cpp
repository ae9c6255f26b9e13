// binding.cpp -- argument checks and marshalling of the latent attention operators between
// torch tensors and the C ABI of libskinny.so, as a CPython module (_latent).
//
// A call on one token's work takes the GPU a few microseconds, and reading shapes, strides and
// addresses of ten tensors through Python attributes takes forty; here it takes under one. The
// module computes nothing: every function checks its tensors (ValueError), fills the argument
// struct and calls the entry point whose address bind() was given.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <initializer_list>
#include <string>

#include "../../include/skinny.h"

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kHead = 128;    // what the kernels are built for
constexpr int64_t kDim = kLatent + kRope, kQuery = kHead + kRope;

typedef skinny_status (*append_fn)(const skinny_latent_append_args *, void *);
typedef skinny_status (*decode_fn)(const skinny_latent_decode_args *, void *);
typedef skinny_status (*prefill_fn)(const skinny_latent_prefill_args *, void *);
append_fn g_append = nullptr;
decode_fn g_decode = nullptr;
prefill_fn g_prefill = nullptr;

// A Python error has been set.
struct Refused {};

[[noreturn]] void refuse(const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    throw Refused();
}

std::string list(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

const char *type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "bfloat16";
        case at::kFloat: return "float32";
        case at::kDouble: return "float64";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kByte: return "uint8";
        default: return "another type";
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

// A tensor operand and the bytes it spans.
struct Operand {
    const char *name;
    const at::Tensor *t;
    uintptr_t begin = 0, end = 0;
    void *ptr() const { return reinterpret_cast<void *>(begin); }
    int64_t stride(int d) const { return t->stride(d); }
};

// Checks an operand's type, device and shape, and takes its span. One that is written gets memory of its
// own here if it still shares that of the tensor it was lazily cloned from; so the written operands of
// a call are taken first, and those that are views of the same storage find it where it is then.
enum Use { READ, WRITTEN };
Operand operand(PyObject *o, const char *name, at::ScalarType type, at::Device dev, std::initializer_list<int64_t> shape,
                Use use = READ) {
    Operand a{name, &tensor(o, name)};
    const at::Tensor &t = *a.t;
    if (t.layout() != at::kStrided) refuse("%s must be a dense tensor", name);
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape))
        refuse("%s must be %s %s, got %s %s", name, type_name(type), list(shape).c_str(), type_name(t.scalar_type()),
               list(t.sizes()).c_str());
    if (t.device() != dev)
        refuse("%s is on %s: all tensors must be on %s", name, t.device().str().c_str(), dev.str().c_str());
    a.begin = a.end = reinterpret_cast<uintptr_t>(use == WRITTEN ? t.mutable_data_ptr() : t.const_data_ptr());
    if (t.numel() > 0) {
        int64_t last = 0;
        for (int64_t d = 0; d < t.dim(); ++d) last += (t.size(d) - 1) * t.stride(d);
        a.end += (last + 1) * t.element_size();
    }
    return a;
}

void want_contiguous(const Operand &a) {
    if (!a.t->is_contiguous()) refuse("%s must be contiguous", a.name);
}

// Rows that are read or written in 16-byte vectors.
void want_rows(const Operand &a) {
    const at::Tensor &t = *a.t;
    const int64_t d = t.dim();
    if (t.numel() == 0) return;
    if (t.size(d - 1) > 1 && t.stride(d - 1) != 1) refuse("%s must be contiguous in its last dimension", a.name);
    for (int64_t i = 0; i + 1 < d; ++i)
        if (t.size(i) > 1 && (t.stride(i) % 8 || t.stride(i) < t.size(d - 1)))
            refuse("%s has strides %s: rows must not overlap and must start at multiples of 8 elements", a.name,
                   list(t.strides()).c_str());
    if (a.begin % 16) refuse("%s must be 16-byte aligned", a.name);
}

// Rows that are written: want_rows, and of two extents the larger stride steps over all rows of the
// smaller one, so that no two rows share numbers.
void want_apart_rows(const Operand &a) {
    want_rows(a);
    const at::Tensor &t = *a.t;
    if (t.numel() == 0 || t.dim() != 3 || t.size(0) <= 1 || t.size(1) <= 1) return;
    const int small = t.stride(0) < t.stride(1) ? 0 : 1;
    if ((t.stride(1 - small) - t.size(2)) / t.stride(small) < t.size(small) - 1)
        refuse("%s has shape %s and strides %s: its rows must not overlap", a.name, list(t.sizes()).c_str(),
               list(t.strides()).c_str());
}

// Judged on byte spans: views that interleave in one wider tensor count as overlapping.
void want_apart(const Operand &out, std::initializer_list<const Operand *> others) {
    for (const Operand *b : others)
        if (b && out.begin < b->end && b->begin < out.end) refuse("%s must not overlap %s", out.name, b->name);
}

at::Device device_of(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (!t.device().is_cuda()) refuse("%s must be on the GPU", name);
    return t.device();
}

int64_t whole(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be a whole number", name);
    }
    return v;
}

float number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be a number", name);
    }
    return static_cast<float>(v);
}

float positive_scale(PyObject *o) {
    const float s = number(o, "scale");      // as the library sees it, in 32 bits
    if (!(s > 0.0f && std::isfinite(s))) refuse("scale must be positive and finite, got %S", o);
    return s;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}

void *stream_of(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
}

const at::Tensor &paged_cache(PyObject *o) {
    const at::Tensor &t = tensor(o, "cache");
    if (t.dim() != 3 || t.size(1) < 1) refuse("cache must be a tensor [pages, page_size, %lld]", (long long)kDim);
    return t;
}

// None: no workspace
Operand workspace_operand(PyObject *o, at::Device dev) {
    if (o == Py_None) return Operand{"workspace", nullptr};
    const at::Tensor &t = tensor(o, "workspace");
    if (t.scalar_type() != at::kByte || t.device() != dev || !t.is_contiguous())
        refuse("workspace must be a contiguous uint8 tensor on the inputs' GPU");
    Operand w{"workspace", &t};
    w.begin = reinterpret_cast<uintptr_t>(t.mutable_data_ptr());
    w.end = w.begin + t.numel();
    return w;
}

PyObject *append(PyObject *const *x) {
    enum { KV, CACHE, SLOTS, POSITIONS, FREQ, WEIGHT, EPS, Q, Q_OUT, INTERLEAVED, STREAM };
    const at::Device dev = device_of(x[KV], "kv");
    if (tensor(x[KV], "kv").dim() != 2) refuse("kv must be 2-D");
    const int64_t n = tensor(x[KV], "kv").size(0);
    const at::Tensor &c = paged_cache(x[CACHE]);
    const Operand cache = operand(x[CACHE], "cache", at::kBFloat16, dev, {c.size(0), c.size(1), kDim}, WRITTEN);
    Operand weight{}, q{}, q_out{};
    const bool normed = x[WEIGHT] != Py_None, queries = x[Q] != Py_None;
    int64_t heads = 0;
    if (queries) {
        if (tensor(x[Q], "q").dim() != 3) refuse("q must be a tensor [n, heads, %lld]", (long long)kRope);
        heads = tensor(x[Q], "q").size(1);
        q_out = operand(x[Q_OUT], "q_out", at::kBFloat16, dev, {n, heads, kRope}, WRITTEN);
        q = operand(x[Q], "q", at::kBFloat16, dev, {n, heads, kRope});
        want_rows(q);
        want_apart_rows(q_out);
    } else if (x[Q_OUT] != Py_None) {
        refuse("q_out needs q");
    }
    const Operand kv = operand(x[KV], "kv", at::kBFloat16, dev, {n, kDim});
    const Operand slots = operand(x[SLOTS], "slots", at::kLong, dev, {n});
    const Operand positions = operand(x[POSITIONS], "positions", at::kLong, dev, {n});
    const Operand freq = operand(x[FREQ], "inv_freq", at::kDouble, dev, {kRope / 2});
    if (normed) {
        weight = operand(x[WEIGHT], "norm_weight", at::kBFloat16, dev, {kLatent});
        want_contiguous(weight);
        want_rows(weight);
    }
    const float eps = number(x[EPS], "eps");
    if (!(eps >= 0.0f)) refuse("eps must not be negative, got %S", x[EPS]);
    want_contiguous(slots);
    want_contiguous(positions);
    want_contiguous(freq);
    want_rows(kv);
    want_apart_rows(cache);
    want_apart(cache, {&kv, &slots, &positions, &freq, normed ? &weight : nullptr, queries ? &q : nullptr});
    if (queries) {
        const bool in_place = q.begin == q_out.begin && q.t->strides() == q_out.t->strides();
        want_apart(q_out, {&kv, &cache, &slots, &positions, &freq, normed ? &weight : nullptr, in_place ? nullptr : &q});
    }
    skinny_latent_append_args a{};
    a.kv = kv.ptr();
    a.cache = cache.ptr();
    a.slots = static_cast<const int64_t *>(slots.ptr());
    a.positions = static_cast<const int64_t *>(positions.ptr());
    a.inv_freq = static_cast<const double *>(freq.ptr());
    a.kv_stride = kv.stride(0);
    a.cache_page_stride = cache.stride(0);
    a.cache_row_stride = cache.stride(1);
    if (normed) a.norm_weight = weight.ptr();
    if (queries) {
        a.q = q.ptr();
        a.q_out = q_out.ptr();
        a.q_row_stride = q.stride(0);
        a.q_head_stride = q.stride(1);
        a.q_out_row_stride = q_out.stride(0);
        a.q_out_head_stride = q_out.stride(1);
    }
    a.n = n;
    a.heads = heads;
    a.pages = c.size(0);
    a.page = c.size(1);
    a.latent = kLatent;
    a.rope = kRope;
    a.eps = eps;
    a.interleaved = truth(x[INTERLEAVED]);
    return PyLong_FromLong(g_append(&a, stream_of(x[STREAM])));
}

PyObject *decode(PyObject *const *x) {
    enum { Q, CACHE, TABLE, LENS, SCALE, TOKENS, ROPE_DIM, OUT, LSE, WORK, STREAM };
    const at::Device dev = device_of(x[Q], "q");
    if (whole(x[ROPE_DIM], "rope_dim") != kRope) refuse("rope_dim must be %lld", (long long)kRope);
    const int64_t tokens = whole(x[TOKENS], "tokens");
    if (tokens < 1) refuse("tokens must be at least 1, got %lld", (long long)tokens);
    const at::Tensor &qt = tensor(x[Q], "q"), &tt = tensor(x[TABLE], "table");
    if (qt.dim() != 3) refuse("q must be 3-D");
    if (tt.dim() != 2) refuse("table must be a tensor [batch, max_pages]");
    const int64_t rows = qt.size(0), heads = qt.size(1), batch = tt.size(0), max_pages = tt.size(1);
    if (rows / tokens != batch || rows % tokens)
        refuse("q has %lld rows: table has %lld requests of %lld tokens", (long long)rows, (long long)batch, (long long)tokens);
    const at::Tensor &c = paged_cache(x[CACHE]);
    const Operand out = operand(x[OUT], "out", at::kBFloat16, dev, {rows, heads, kLatent}, WRITTEN);
    const Operand lse = operand(x[LSE], "lse", at::kFloat, dev, {rows, heads}, WRITTEN);
    const Operand work = workspace_operand(x[WORK], dev);
    const Operand q = operand(x[Q], "q", at::kBFloat16, dev, {rows, heads, kDim});
    const Operand cache = operand(x[CACHE], "cache", at::kBFloat16, dev, {c.size(0), c.size(1), kDim});
    const Operand table = operand(x[TABLE], "table", at::kInt, dev, {batch, max_pages});
    const Operand lens = operand(x[LENS], "lens", at::kInt, dev, {batch});
    want_rows(q);
    want_rows(cache);
    want_apart_rows(out);
    want_contiguous(lens);
    want_contiguous(lse);
    if ((max_pages > 1 && table.stride(1) != 1) || (batch > 1 && table.stride(0) < max_pages))
        refuse("table must be contiguous in its last dimension, its rows apart");
    if (rows && heads && (c.size(0) < 1 || max_pages < 1)) refuse("the cache and the table need a page at least");
    want_apart(out, {&q, &cache, &table, &lens});
    want_apart(lse, {&q, &cache, &table, &lens, &out});
    want_apart(work, {&q, &cache, &table, &lens, &out, &lse});
    skinny_latent_decode_args a{};
    a.q = q.ptr();
    a.cache = cache.ptr();
    a.table = static_cast<const int32_t *>(table.ptr());
    a.lens = static_cast<const int32_t *>(lens.ptr());
    a.out = out.ptr();
    a.lse = static_cast<float *>(lse.ptr());
    a.workspace = work.ptr();
    a.workspace_bytes = work.end - work.begin;
    a.q_row_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
    a.cache_page_stride = cache.stride(0);
    a.cache_row_stride = cache.stride(1);
    a.table_stride = table.stride(0);
    a.out_row_stride = out.stride(0);
    a.out_head_stride = out.stride(1);
    a.batch = batch;
    a.tokens = tokens;
    a.heads = heads;
    a.pages = c.size(0);
    a.page = c.size(1);
    a.max_pages = max_pages;
    a.latent = kLatent;
    a.rope = kRope;
    a.scale = positive_scale(x[SCALE]);
    return PyLong_FromLong(g_decode(&a, stream_of(x[STREAM])));
}

PyObject *prefill(PyObject *const *x) {
    enum { Q, K, V, K_ROT, CU_Q, CU_K, SCALE, CAUSAL, OUT, LSE, WORK, STREAM };
    const at::Device dev = device_of(x[Q], "q");
    const at::Tensor &qt = tensor(x[Q], "q"), &kt = tensor(x[K], "k"), &ct = tensor(x[CU_Q], "cu_q");
    if (qt.dim() != 3 || kt.dim() != 3) refuse("q and k must be 3-D tensors");
    if (ct.dim() != 1 || ct.size(0) < 1) refuse("cu_q must be a tensor [batch + 1]");
    const int64_t nq = qt.size(0), heads = qt.size(1), nk = kt.size(0), batch = ct.size(0) - 1;
    const Operand out = operand(x[OUT], "out", at::kBFloat16, dev, {nq, heads, kHead}, WRITTEN);
    const Operand lse = operand(x[LSE], "lse", at::kFloat, dev, {nq, heads}, WRITTEN);
    const Operand work = workspace_operand(x[WORK], dev);
    const Operand q = operand(x[Q], "q", at::kBFloat16, dev, {nq, heads, kQuery});
    const Operand k = operand(x[K], "k", at::kBFloat16, dev, {nk, heads, kHead});
    const Operand v = operand(x[V], "v", at::kBFloat16, dev, {nk, heads, kHead});
    const Operand kr = operand(x[K_ROT], "k_rot", at::kBFloat16, dev, {nk, kRope});
    const Operand cq = operand(x[CU_Q], "cu_q", at::kInt, dev, {batch + 1});
    const Operand ck = operand(x[CU_K], "cu_k", at::kInt, dev, {batch + 1});
    for (const Operand *o : {&q, &k, &v, &kr}) want_rows(*o);
    want_apart_rows(out);
    for (const Operand *o : {&cq, &ck, &lse}) want_contiguous(*o);
    want_apart(out, {&q, &k, &v, &kr, &cq, &ck});
    want_apart(lse, {&q, &k, &v, &kr, &cq, &ck, &out});
    want_apart(work, {&q, &k, &v, &kr, &cq, &ck, &out, &lse});
    skinny_latent_prefill_args a{};
    a.q = q.ptr();
    a.k = k.ptr();
    a.v = v.ptr();
    a.k_rot = kr.ptr();
    a.cu_q = static_cast<const int32_t *>(cq.ptr());
    a.cu_k = static_cast<const int32_t *>(ck.ptr());
    a.out = out.ptr();
    a.lse = static_cast<float *>(lse.ptr());
    a.workspace = work.ptr();
    a.workspace_bytes = work.end - work.begin;
    a.q_row_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
    a.k_row_stride = k.stride(0);
    a.k_head_stride = k.stride(1);
    a.v_row_stride = v.stride(0);
    a.v_head_stride = v.stride(1);
    a.k_rot_stride = kr.stride(0);
    a.out_row_stride = out.stride(0);
    a.out_head_stride = out.stride(1);
    a.nq = nq;
    a.nk = nk;
    a.batch = batch;
    a.heads = heads;
    a.head_dim = kHead;
    a.rope = kRope;
    a.scale = positive_scale(x[SCALE]);
    a.causal = truth(x[CAUSAL]);
    return PyLong_FromLong(g_prefill(&a, stream_of(x[STREAM])));
}

// Runs one of the above on exactly `want` arguments; no C++ exception leaves.
template <PyObject *(*F)(PyObject *const *), int want>
PyObject *call(PyObject *, PyObject *const *x, Py_ssize_t n) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", want, n);
        return nullptr;
    }
    if (!g_append || !g_decode || !g_prefill) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return F(x);
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *bind(PyObject *, PyObject *const *x, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three entry points wanted");
        return nullptr;
    }
    void *p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(x[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is NULL");
            return nullptr;
        }
    }
    g_append = reinterpret_cast<append_fn>(p[0]);
    g_decode = reinterpret_cast<decode_fn>(p[1]);
    g_prefill = reinterpret_cast<prefill_fn>(p[2]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, "bind(append, decode, prefill): addresses of the library's entry points"},
    {"append", FAST((call<append, 11>)), METH_FASTCALL, "status of skinny_latent_append_bf16"},
    {"decode", FAST((call<decode, 11>)), METH_FASTCALL, "status of skinny_latent_decode_bf16"},
    {"prefill", FAST((call<prefill, 12>)), METH_FASTCALL, "status of skinny_latent_prefill_bf16"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_latent", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__latent(void) { return PyModule_Create(&module); }
