// binding.cpp -- the attention calls' Python entry points, below attention.py:
// the checks of the tensors and the calls of the C ABI.
//
// A call takes six to eleven lists of P tensors.  Looking at each in Python
// (shape, strides, type, device, address) costs over half a microsecond a
// tensor, 22 us for the 24 tensors of one decode step's norm and rotation,
// whose kernel takes 7; here it is some 20 ns.  Nothing computes here.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tp_attention.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Raised {};        // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
    va_list v;
    va_start(v, format);
    PyErr_FormatV(type, format, v);
    va_end(v);
    throw Raised();
}

const char* name_of(ScalarType t) { return c10::toString(t); }

// One argument list's view: positional arguments as Python passes them.
struct Args {
    PyObject* const* a;
    Py_ssize_t n;
    const char* what;
    int device;
    const Tensor& tensor(PyObject* o, const char* name) const {
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: %s must be a torch tensor", what, name);
        return THPVariable_Unpack(o);
    }
    void on_device(const Tensor& t, const char* name) const {
        if (!t.is_cuda() || t.get_device() != device)
            raise(PyExc_ValueError, "%s: %s must be on the current device (%d)", what, name, device);
    }
    void type(const Tensor& t, const char* name, ScalarType dt) const {
        if (t.scalar_type() != dt)
            raise(PyExc_TypeError, "%s: %s must be %s, got %s", what, name, name_of(dt), name_of(t.scalar_type()));
    }
    long long integer(Py_ssize_t i) const {
        const long long x = PyLong_AsLongLong(a[i]);
        if (x == -1 && PyErr_Occurred()) throw Raised();
        return x;
    }
    int int32(Py_ssize_t i, const char* name) const {
        const long long x = integer(i);
        if (x < -0x7fffffffLL || x > 0x7fffffffLL) raise(PyExc_ValueError, "%s: %s does not fit 32 bits", what, name);
        return (int)x;
    }
    float real(Py_ssize_t i) const {
        const double x = PyFloat_AsDouble(a[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Raised();
        return (float)x;
    }
    bool none(Py_ssize_t i) const { return a[i] == Py_None; }
    // a contiguous tensor that all ranks read
    void* one(Py_ssize_t i, const char* name, ScalarType dt, int64_t numel = -1, int64_t* size = nullptr) const {
        const Tensor& t = tensor(a[i], name);
        on_device(t, name);
        type(t, name, dt);
        if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: %s must be contiguous", what, name);
        if (numel >= 0 && t.numel() != numel)
            raise(PyExc_ValueError, "%s: %s needs %lld elements, got %lld", what, name, (long long)numel, (long long)t.numel());
        if (size) *size = t.numel();
        return t.data_ptr();
    }
    // the workspace: any contiguous tensor on the device
    void* ws(Py_ssize_t i, size_t& bytes) const {
        const Tensor& t = tensor(a[i], "the workspace");
        if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
            raise(PyExc_ValueError, "%s: the workspace must be a contiguous device tensor", what);
        bytes = (size_t)t.nbytes();
        return t.data_ptr();
    }
    void* stream(Py_ssize_t i) const {
        void* s = PyLong_AsVoidPtr(a[i]);
        if (!s && PyErr_Occurred()) throw Raised();
        return s;
    }
};

// P per-rank tensors of one shape: the last dimensions dense, the first one
// (tokens) at a stride of its own, or everything dense where `packed`.
struct Ranks {
    void* p[RING_MAX_RANKS];
    int64_t row = 0;            // row stride
    bool given = false;
    void* const* or_null() { return given ? p : nullptr; }
};

struct List {
    PyObject* seq;
    explicit List(PyObject* o, const char* what, const char* name) : seq(PySequence_Fast(o, "")) {
        if (!seq) {
            PyErr_Clear();
            raise(PyExc_TypeError, "%s: %s is a list of one tensor per rank", what, name);
        }
    }
    ~List() { Py_DECREF(seq); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// The shape of the first tensor of a list of rank buffers, which sets P.
std::vector<int64_t> leading(const Args& c, Py_ssize_t i, const char* name, int dims, int& P, ScalarType* dt = nullptr) {
    const List l(c.a[i], c.what, name);
    if (l.size() < 1 || l.size() > RING_MAX_RANKS)
        raise(PyExc_ValueError, "%s: 1..%d rank buffers, got %lld", c.what, RING_MAX_RANKS, (long long)l.size());
    P = (int)l.size();
    const Tensor& t = c.tensor(l.at(0), name);
    if (t.dim() != dims)
        raise(PyExc_ValueError, "%s: %s has %d dimensions, got %s", c.what, name, dims, text(t.sizes()).c_str());
    for (int64_t n : t.sizes())
        if (n > 0x7fffffffLL) raise(PyExc_ValueError, "%s: %s is too large", c.what, name);
    if (dt) *dt = t.scalar_type();
    return t.sizes().vec();
}

Ranks ranks(const Args& c, Py_ssize_t i, const char* name, int P, at::IntArrayRef shape, ScalarType dt, bool packed) {
    Ranks r;
    const List l(c.a[i], c.what, name);
    if (l.size() != P)
        raise(PyExc_ValueError, "%s: %s needs %d rank buffers, got %lld", c.what, name, P, (long long)l.size());
    for (int q = 0; q < P; ++q) {
        const Tensor& t = c.tensor(l.at(q), name);
        c.on_device(t, name);
        c.type(t, name, dt);
        if (t.sizes() != shape)
            raise(PyExc_ValueError, "%s: every rank's %s must be %s, got %s", c.what, name, text(shape).c_str(),
                  text(t.sizes()).c_str());
        if (packed) {
            if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: %s must be contiguous", c.what, name);
        } else {
            int64_t row = 1;
            for (size_t d = shape.size() - 1; d > 0; --d) {
                if (shape[d] > 1 && t.numel() && t.stride(d) != row)
                    raise(PyExc_ValueError, "%s: the heads of a row of %s must be dense", c.what, name);
                row *= shape[d];
            }
            if (shape[0] > 1 && t.numel()) row = t.stride(0);
            if (q && row != r.row) raise(PyExc_ValueError, "%s: every rank's %s must have the same strides", c.what, name);
            r.row = row;
        }
        r.p[q] = t.data_ptr();
    }
    r.given = true;
    return r;
}

PyObject* code(int rc) { return PyLong_FromLong(rc); }

template <class T> T* const* as(Ranks& r) { return (T* const*)r.or_null(); }
const void* const* in(Ranks& r) { return (const void* const*)r.or_null(); }

// lengths, new_tokens, free_pages, used, block_table, lengths_after, cu_new,
// positions, slots, used_after, page_size, prefix_len
PyObject* plan(const Args& c) {
    int64_t B, nfree, cap;
    void* len = c.one(0, "lengths", at::kInt, -1, &B);
    void* add = c.one(1, "new_tokens", at::kInt, B);
    void* fp = c.one(2, "free_pages", at::kInt, -1, &nfree);
    void* used = c.one(3, "used", at::kInt, 1);
    const Tensor& tab = c.tensor(c.a[4], "block_table");
    if (tab.dim() != 2 || tab.size(0) != B)
        raise(PyExc_ValueError, "%s: block_table is (requests, pages), got %s", c.what, text(tab.sizes()).c_str());
    void* tp = c.one(4, "block_table", at::kInt);
    void* after = c.one(5, "lengths_after", at::kInt, B);
    void* cu = c.one(6, "cu_new", at::kInt, B + 1);
    void* pos = c.one(7, "positions", at::kInt, -1, &cap);
    void* slots = c.one(8, "slots", at::kLong, cap);
    void* ua = c.one(9, "used_after", at::kInt, 1);
    if (B > 0x7fffffff || nfree > 0x7fffffff || cap > 0x7fffffff || tab.size(1) > 0x7fffffff)
        raise(PyExc_ValueError, "%s: sizes must fit 32 bits", c.what);
    return code(kv_plan((const int*)len, (const int*)add, (const int*)fp, (const int*)used, (int*)tp, (int*)after, (int*)cu,
                        (int*)pos, (long long*)slots, (int*)ua, (int)B, (int)nfree, (int)tab.size(1),
                        c.int32(10, "page_size"), (int)cap, c.int32(11, "prefix_len"), c.stream(12)));
}

// What the norm-and-rotation calls share: qkv, gain_q, gain_k, cos_sin, pos
// at arguments i .. i + 4.
struct Rope {
    Ranks x, gq, gk;
    void *cs, *pos;
    int Hkv, dtype, rot;
    long long rows;
    ScalarType dt;
};
Rope rope_args(const Args& c, Py_ssize_t i, int P, int64_t T, int64_t Hq, int64_t D) {
    Rope r;
    int P2;
    const auto s = leading(c, i, "qkv", 2, P2, &r.dt);
    if (r.dt != at::kFloat && r.dt != at::kBFloat16)
        raise(PyExc_TypeError, "%s: qkv is float32 or bfloat16, got %s", c.what, name_of(r.dt));
    if (P2 != P || s[0] != T) raise(PyExc_ValueError, "%s: qkv and the heads differ in ranks or tokens", c.what);
    const int64_t hkv = D ? (s[1] / D - Hq) / 2 : 0;
    if (hkv < 1 || (Hq + 2 * hkv) * D != s[1])
        raise(PyExc_ValueError, "%s: rows of %lld values are not %lld query heads and two equal groups of heads of width %lld",
              c.what, (long long)s[1], (long long)Hq, (long long)D);
    r.Hkv = (int)hkv;
    r.x = ranks(c, i, "qkv", P, s, r.dt, false);
    if (c.none(i + 1) != c.none(i + 2)) raise(PyExc_ValueError, "%s: both gains or neither", c.what);
    if (!c.none(i + 1)) {
        r.gq = ranks(c, i + 1, "gain_q", P, {D}, at::kFloat, true);
        r.gk = ranks(c, i + 2, "gain_k", P, {D}, at::kFloat, true);
    }
    const Tensor& t = c.tensor(c.a[i + 3], "cos_sin");
    if (t.dim() != 2 || t.size(1) > 0x7fffffff)
        raise(PyExc_ValueError, "%s: cos_sin is (positions, rotated width), got %s", c.what, text(t.sizes()).c_str());
    r.cs = c.one(i + 3, "cos_sin", at::kFloat);
    r.rot = (int)t.size(1);
    r.rows = t.size(0);
    r.pos = c.one(i + 4, "pos", at::kInt, T);
    r.dtype = r.dt == at::kFloat ? RING_F32 : RING_BF16;
    return r;
}

// qkv, gain_q, gain_k, cos_sin, pos, q, k, v, k_cache, v_cache, slots, eps
PyObject* rope(const Args& c) {
    int P;
    const auto s = leading(c, 5, "q", 3, P);
    const int64_t T = s[0], D = s[2];
    Rope r = rope_args(c, 0, P, T, s[1], D);
    Ranks q = ranks(c, 5, "q", P, s, at::kBFloat16, true), k, v, kc, vc;
    if (c.none(6) != c.none(7) || c.none(8) != c.none(9) || c.none(8) != c.none(10))
        raise(PyExc_ValueError, "%s: k and v, and k_cache, v_cache and slots, go together", c.what);
    if (!c.none(6)) {
        k = ranks(c, 6, "k", P, {T, r.Hkv, D}, at::kBFloat16, true);
        v = ranks(c, 7, "v", P, {T, r.Hkv, D}, at::kBFloat16, true);
    }
    void* slots = nullptr;
    long long cached = 0;
    if (!c.none(8)) {
        int P2;
        const auto n = leading(c, 8, "k_cache", 3, P2);
        cached = n[0];
        kc = ranks(c, 8, "k_cache", P, {cached, r.Hkv, D}, at::kBFloat16, true);
        vc = ranks(c, 9, "v_cache", P, {cached, r.Hkv, D}, at::kBFloat16, true);
        slots = c.one(10, "slots", at::kLong, T);
    }
    return code(tp_qk_norm_rope(in(r.x), as<const float>(r.gq), as<const float>(r.gk), (const float*)r.cs, (const int*)r.pos,
                                as<void>(q), as<void>(k), as<void>(v), as<void>(kc), as<void>(vc), (const long long*)slots, P,
                                (int)T, (int)s[1], r.Hkv, (int)D, r.rot, r.rows, cached, r.x.row, c.real(11), r.dtype,
                                c.stream(12)));
}

// dq, dk, dv, qkv, gain_q, gain_k, cos_sin, pos, dqkv, dgain_q, dgain_k, eps, ws
PyObject* rope_grad(const Args& c) {
    int P;
    const auto s = leading(c, 0, "dq", 3, P);
    const int64_t T = s[0], D = s[2];
    Rope r = rope_args(c, 3, P, T, s[1], D);
    Ranks dq = ranks(c, 0, "dq", P, s, at::kBFloat16, true);
    Ranks dk = ranks(c, 1, "dk", P, {T, r.Hkv, D}, at::kBFloat16, true);
    Ranks dv = ranks(c, 2, "dv", P, {T, r.Hkv, D}, at::kBFloat16, true);
    Ranks dx = ranks(c, 8, "dqkv", P, {T, (s[1] + 2 * r.Hkv) * D}, r.dt, true), gq, gk;
    if (!c.none(4)) {
        if (c.none(9) || c.none(10)) raise(PyExc_ValueError, "%s: the gains' gradients need buffers", c.what);
        gq = ranks(c, 9, "dgain_q", P, {D}, at::kFloat, true);
        gk = ranks(c, 10, "dgain_k", P, {D}, at::kFloat, true);
    }
    size_t bytes;
    void* ws = c.ws(12, bytes);
    return code(tp_qk_norm_rope_grad(in(dq), in(dk), in(dv), in(r.x), as<const float>(r.gq), as<const float>(r.gk),
                                     (const float*)r.cs, (const int*)r.pos, as<void>(dx), as<float>(gq), as<float>(gk), P,
                                     (int)T, (int)s[1], r.Hkv, (int)D, r.rot, r.rows, r.x.row, c.real(11), r.dtype, ws, bytes,
                                     c.stream(13)));
}

struct Prompt {
    Ranks q, k, v, o;
    void *cq, *ck;
    int P, B, Tq, Tk, Hq, Hkv, D;
    at::DimVector sq, sk;
};
// q, k, v, o, cu_q, cu_k at arguments i .. i + 5
Prompt prompt_args(const Args& c, Py_ssize_t i) {
    Prompt p;
    const auto sq = leading(c, i, "q", 3, p.P);
    int P2;
    const auto sk = leading(c, i + 1, "k", 3, P2);
    p.Tq = (int)sq[0];
    p.Hq = (int)sq[1];
    p.D = (int)sq[2];
    p.Tk = (int)sk[0];
    p.Hkv = (int)sk[1];
    p.sq = {sq[0], sq[1], sq[2]};
    p.sk = {sk[0], sk[1], sq[2]};
    p.q = ranks(c, i, "q", p.P, p.sq, at::kBFloat16, false);
    p.k = ranks(c, i + 1, "k", p.P, p.sk, at::kBFloat16, false);
    p.v = ranks(c, i + 2, "v", p.P, p.sk, at::kBFloat16, false);
    p.o = ranks(c, i + 3, "o", p.P, p.sq, at::kBFloat16, false);
    int64_t n;
    p.cq = c.one(i + 4, "cu_q", at::kInt, -1, &n);
    if (n < 1 || n > 0x7fffffff)
        raise(PyExc_ValueError, "%s: cu_q holds the prompts' offsets, one more than prompts", c.what);
    p.ck = c.one(i + 5, "cu_k", at::kInt, n);
    p.B = (int)n - 1;
    return p;
}

// q, k, v, o, cu_q, cu_k, lse, causal, scale
PyObject* prompt(const Args& c) {
    Prompt p = prompt_args(c, 0);
    Ranks lse;
    if (!c.none(6)) lse = ranks(c, 6, "lse", p.P, {p.Hq, p.Tq}, at::kFloat, true);
    return code(tp_attention(in(p.q), in(p.k), in(p.v), as<void>(p.o), as<float>(lse), (const int*)p.cq, (const int*)p.ck, p.P,
                             p.B, p.Tq, p.Tk, p.Hq, p.Hkv, p.D, p.q.row, p.k.row, p.v.row, p.o.row, c.int32(7, "causal"),
                             c.real(8), c.stream(9)));
}

// q, k, v, o, cu_q, cu_k, lse, do, dq, dk, dv, causal, scale, ws
PyObject* prompt_grad(const Args& c) {
    Prompt p = prompt_args(c, 0);
    Ranks lse = ranks(c, 6, "lse", p.P, {p.Hq, p.Tq}, at::kFloat, true);
    Ranks go = ranks(c, 7, "do", p.P, p.sq, at::kBFloat16, false), dq = ranks(c, 8, "dq", p.P, p.sq, at::kBFloat16, false);
    Ranks dk = ranks(c, 9, "dk", p.P, p.sk, at::kBFloat16, false), dv = ranks(c, 10, "dv", p.P, p.sk, at::kBFloat16, false);
    size_t bytes;
    void* ws = c.ws(13, bytes);
    return code(tp_attention_grad(in(go), in(p.q), in(p.k), in(p.v), in(p.o), as<const float>(lse), as<void>(dq), as<void>(dk),
                                  as<void>(dv), (const int*)p.cq, (const int*)p.ck, p.P, p.B, p.Tq, p.Tk, p.Hq, p.Hkv, p.D,
                                  p.q.row, p.k.row, p.v.row, p.o.row, go.row, dq.row, dk.row, dv.row, c.int32(11, "causal"),
                                  c.real(12), ws, bytes, c.stream(14)));
}

// q, k_cache, v_cache, o, block_table, lengths, page_size, prefix_pages,
// prefix_len, scale, ws
PyObject* decode(const Args& c) {
    int P, P2;
    const auto sq = leading(c, 0, "q", 3, P), sk = leading(c, 1, "k_cache", 3, P2);
    const int64_t B = sq[0], D = sq[2];
    Ranks q = ranks(c, 0, "q", P, sq, at::kBFloat16, false), o = ranks(c, 3, "o", P, sq, at::kBFloat16, false);
    Ranks kc = ranks(c, 1, "k_cache", P, {sk[0], sk[1], D}, at::kBFloat16, true);
    Ranks vc = ranks(c, 2, "v_cache", P, {sk[0], sk[1], D}, at::kBFloat16, true);
    const Tensor& tab = c.tensor(c.a[4], "block_table");
    if (tab.dim() != 2 || tab.size(0) != B || tab.size(1) > 0x7fffffff)
        raise(PyExc_ValueError, "%s: block_table is (requests, pages), got %s", c.what, text(tab.sizes()).c_str());
    void* tp = c.one(4, "block_table", at::kInt);
    void* len = c.one(5, "lengths", at::kInt, B);
    const int page = c.int32(6, "page_size"), prefix = c.int32(8, "prefix_len"), W = (int)tab.size(1);
    if (page < 1 || sk[0] % page)
        raise(PyExc_ValueError, "%s: the cache's %lld rows are not whole pages of %d", c.what, (long long)sk[0], page);
    void* pp = nullptr;
    if (prefix > 0) {
        int64_t n = 0;
        if (!c.none(7)) pp = c.one(7, "prefix_pages", at::kInt, -1, &n);
        if (n * page < prefix) raise(PyExc_ValueError, "%s: prefix_pages does not hold %d tokens", c.what, prefix);
    }
    size_t bytes;
    void* ws = c.ws(10, bytes);
    return code(tp_attention_decode(in(q), in(kc), in(vc), as<void>(o), (const int*)tp, (const int*)len, (const int*)pp, P,
                                    (int)B, (int)sq[1], (int)sk[1], (int)D, W, page, (int)(sk[0] / page), prefix, q.row, o.row,
                                    c.real(9), ws, bytes, c.stream(11)));
}

struct Entry {
    const char* name;
    int args;               // before the stream and the current device, which every call ends with
    PyObject* (*call)(const Args&);
};
constexpr Entry kEntries[] = {{"kv_plan", 12, plan}, {"tp_qk_norm_rope", 12, rope}, {"tp_qk_norm_rope_grad", 13, rope_grad},
                              {"tp_attention", 9, prompt}, {"tp_attention_grad", 14, prompt_grad},
                              {"tp_attention_decode", 11, decode}};

template <int I> PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr const Entry& e = kEntries[I];
    if (n != e.args + 2) return PyErr_Format(PyExc_TypeError, "%s: %d arguments, got %zd", e.name, e.args + 2, n);
    try {
        Args c{a, n, e.name, 0};
        c.device = (int)c.integer(n - 1);
        return e.call(c);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& x) {
        return PyErr_Format(PyExc_RuntimeError, "%s: %s", e.name, x.what());
    }
}

#define ENTRY(I) {kEntries[I].name, (PyCFunction)(void (*)(void))entry<I>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(0), ENTRY(1), ENTRY(2), ENTRY(3), ENTRY(4), ENTRY(5), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
