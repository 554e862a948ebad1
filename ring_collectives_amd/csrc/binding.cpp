// binding.cpp -- the Python entry points of the attention calls and of the beam
// search, below attention.py and search.py: the checks of the tensors and the
// calls of the C ABI.
//
// A call takes six to eleven lists of P tensors.  Looking at each in Python
// (shape, strides, type, device, address) costs over half a microsecond a
// tensor, 22 us for the 24 tensors of one decode step's norm and rotation,
// whose kernel takes 7; here it is some 20 ns.  Nothing computes here.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tp_search.h"

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

// ---------------------------------------------------------------- beam search
// two or three tensors that a call takes or writes as one shape, any of them
void* shaped(const Args& c, Py_ssize_t i, const char* name, ScalarType dt, at::IntArrayRef shape) {
    const Tensor& t = c.tensor(c.a[i], name);
    if (t.sizes() != shape)
        raise(PyExc_ValueError, "%s: %s must be %s, got %s", c.what, name, text(shape).c_str(), text(t.sizes()).c_str());
    return c.one(i, name, dt);
}
// flags: bytes or bools
void* flags(const Args& c, Py_ssize_t i, const char* name, at::IntArrayRef shape) {
    if (c.none(i)) return nullptr;
    const ScalarType dt = c.tensor(c.a[i], name).scalar_type();
    return shaped(c, i, name, dt == at::kBool ? at::kBool : at::kByte, shape);
}
at::DimVector sizes_of(const Args& c, Py_ssize_t i, const char* name, int64_t dims, const char* what) {
    const Tensor& t = c.tensor(c.a[i], name);
    if (t.dim() != dims) raise(PyExc_ValueError, "%s: %s is %s, got %s", c.what, name, what, text(t.sizes()).c_str());
    for (int64_t n : t.sizes())
        if (n > 0x7fffffffLL) raise(PyExc_ValueError, "%s: %s is too large", c.what, name);
    return at::DimVector(t.sizes());
}

// logits, scores, parents, tokens, scores_after, vocab, done, done_after, end_token, ws
PyObject* select(const Args& c) {
    int P;
    ScalarType dt;
    const auto s = leading(c, 0, "logits", 2, P, &dt);
    if (dt != at::kFloat && dt != at::kBFloat16)
        raise(PyExc_TypeError, "%s: logits are float32 or bfloat16, got %s", c.what, name_of(dt));
    Ranks x = ranks(c, 0, "logits", P, s, dt, false);
    const auto sc = sizes_of(c, 1, "scores", 2, "(groups, beams)"), out = sizes_of(c, 2, "parents", 2, "(groups, places)");
    if (sc[0] * sc[1] != s[0])
        raise(PyExc_ValueError, "%s: %lld rows of logits are not %s beams", c.what, (long long)s[0], text(sc).c_str());
    if (out[0] != sc[0]) raise(PyExc_ValueError, "%s: parents are (%lld, places), got %s", c.what, (long long)sc[0], text(out).c_str());
    const void* score = shaped(c, 1, "scores", at::kFloat, sc);
    int *parents = (int*)shaped(c, 2, "parents", at::kInt, out), *tokens = (int*)shaped(c, 3, "tokens", at::kInt, out);
    float* after = (float*)shaped(c, 4, "scores_after", at::kFloat, out);
    const void* done = flags(c, 6, "done", sc);
    void* done_after = flags(c, 7, "done_after", out);
    if (!sc[1] || !out[1]) raise(PyExc_ValueError, "%s: groups have at least one beam and one place", c.what);
    if (c.none(6) != c.none(7)) raise(PyExc_ValueError, "%s: done and done_after go together", c.what);
    // rows that are one: their stride is any that the call takes
    const long long row = s[0] > 1 ? x.row : (s[1] + 7) / 8 * 8;
    size_t bytes;
    void* ws = c.ws(9, bytes);
    return code(beam_select(in(x), (const float*)score, (const unsigned char*)done, parents, tokens, after, (unsigned char*)done_after,
                            P, (int)sc[0], (int)sc[1], (int)out[1], (int)s[1], c.int32(5, "vocab"), row, c.int32(8, "end_token"),
                            dt == at::kFloat ? RING_F32 : RING_BF16, ws, bytes, c.stream(10)));
}

// block_table, lengths, parents, keep, free_pages, used, table_after,
// lengths_after, copies, n_copies, shared, used_after, group, page_size, pages, ws
PyObject* fork(const Args& c) {
    const auto tab = sizes_of(c, 0, "block_table", 2, "(rows, pages)"), after = sizes_of(c, 6, "table_after", 2, "(rows, pages)");
    if (after[1] != tab[1])
        raise(PyExc_ValueError, "%s: table_after has rows of %lld pages, got %s", c.what, (long long)tab[1], text(after).c_str());
    const int64_t B = tab[0], B2 = after[0];
    int64_t nfree;
    const int* table = (const int*)c.one(0, "block_table", at::kInt);
    const int* len = (const int*)c.one(1, "lengths", at::kInt, B);
    const int* par = (const int*)c.one(2, "parents", at::kInt, B2);
    const int* keep = c.none(3) ? nullptr : (const int*)c.one(3, "keep", at::kInt, B2);
    int* fp = (int*)c.one(4, "free_pages", at::kInt, -1, &nfree);
    const int* used = (const int*)c.one(5, "used", at::kInt, 1);
    int* ta = (int*)c.one(6, "table_after", at::kInt);
    int* la = (int*)c.one(7, "lengths_after", at::kInt, B2);
    int* copies = (int*)shaped(c, 8, "copies", at::kInt, {B2, 2});
    int* nc = (int*)c.one(9, "n_copies", at::kInt, 1);
    const int group = c.int32(12, "group");
    if (group < 1 || B2 % group) raise(PyExc_ValueError, "%s: %lld rows are not groups of %d", c.what, (long long)B2, group);
    int* shared = c.none(10) ? nullptr : (int*)c.one(10, "shared", at::kInt, B2 / group);
    int* ua = (int*)c.one(11, "used_after", at::kInt, 1);
    if (nfree > 0x7fffffff) raise(PyExc_ValueError, "%s: sizes must fit 32 bits", c.what);
    size_t bytes;
    void* ws = c.ws(15, bytes);
    return code(kv_fork(table, len, par, keep, fp, used, ta, la, copies, nc, shared, ua, (int)B, (int)B2, group, (int)nfree,
                        (int)tab[1], c.int32(13, "page_size"), c.int32(14, "pages"), ws, bytes, c.stream(16)));
}

// block_table, lengths, table_after, free_pages, copies, n_copies, used_after,
// page_size, first_page, ws
PyObject* compact(const Args& c) {
    const auto tab = sizes_of(c, 0, "block_table", 2, "(rows, pages)");
    int64_t nfree;
    const int* table = (const int*)c.one(0, "block_table", at::kInt);
    const int* len = (const int*)c.one(1, "lengths", at::kInt, tab[0]);
    int* ta = (int*)shaped(c, 2, "table_after", at::kInt, tab);
    int* fp = (int*)c.one(3, "free_pages", at::kInt, -1, &nfree);
    if (nfree > 0x7fffffff) raise(PyExc_ValueError, "%s: sizes must fit 32 bits", c.what);
    int* copies = (int*)shaped(c, 4, "copies", at::kInt, {nfree / 2, 2});
    int* nc = (int*)c.one(5, "n_copies", at::kInt, 1);
    int* ua = (int*)c.one(6, "used_after", at::kInt, 1);
    size_t bytes;
    void* ws = c.ws(9, bytes);
    return code(kv_compact(table, len, ta, fp, copies, nc, ua, (int)tab[0], (int)nfree, (int)tab[1], c.int32(7, "page_size"),
                           c.int32(8, "first_page"), ws, bytes, c.stream(10)));
}

// caches, copies, n_copies, pages
PyObject* copy_pages(const Args& c) {
    const List l(c.a[0], c.what, "caches");
    if (l.size() < 1 || l.size() > 2 * RING_MAX_RANKS)
        raise(PyExc_ValueError, "%s: 1..%d caches, got %lld", c.what, 2 * RING_MAX_RANKS, (long long)l.size());
    void* p[2 * RING_MAX_RANKS];
    const int pages = c.int32(3, "pages");
    if (pages < 0) raise(PyExc_ValueError, "%s: pages must not be negative", c.what);
    long long bytes = -1;
    for (Py_ssize_t i = 0; i < l.size(); ++i) {
        const Tensor& t = c.tensor(l.at(i), "caches");
        c.on_device(t, "caches");
        if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: caches must be contiguous", c.what);
        const long long n = (long long)t.nbytes();
        if (pages ? n % pages : n) raise(PyExc_ValueError, "%s: a cache of %lld bytes is not %d pages", c.what, n, pages);
        if (bytes >= 0 && n != bytes) raise(PyExc_ValueError, "%s: every cache must be of the same size", c.what);
        bytes = n;
        p[i] = t.data_ptr();
    }
    const auto s = sizes_of(c, 1, "copies", 2, "(copies, 2)");
    const int* copies = (const int*)shaped(c, 1, "copies", at::kInt, {s[0], 2});
    const int* nc = (const int*)c.one(2, "n_copies", at::kInt, 1);
    return code(kv_copy_pages(p, copies, nc, (int)l.size(), (int)s[0], pages, pages ? bytes / pages : 0, c.stream(4)));
}

// A 4-bit cache: P tensors (pages, Hkv, kv4_page_bytes(1, D, page_size)).
struct Cache4 {
    Ranks p;
    int pages, Hkv, page;
};
Cache4 cache4(const Args& c, Py_ssize_t i, int P, int64_t D, int page) {
    int P2;
    const auto s = leading(c, i, "cache", 3, P2);
    Cache4 r;
    r.p = ranks(c, i, "cache", P, s, at::kByte, true);
    r.pages = (int)s[0];
    r.Hkv = (int)s[1];
    r.page = page;
    const size_t bytes = D == 64 || D == 128 ? kv4_page_bytes(1, (int)D, page) : 0;
    if (bytes && (int64_t)bytes != s[2])
        raise(PyExc_ValueError, "%s: a page of %d rows of %lld values takes %lld bytes a head, the cache has %lld", c.what, page,
              (long long)D, (long long)bytes, (long long)s[2]);
    return r;
}

// k, v, cache, slots, page_size
PyObject* kv4_rows(const Args& c, Py_ssize_t k_at, Py_ssize_t cache_at, Py_ssize_t slots_at, bool write) {
    int P;
    const auto s = leading(c, k_at, "k", 3, P);
    Ranks k = ranks(c, k_at, "k", P, s, at::kBFloat16, false), v = ranks(c, k_at + 1, "v", P, s, at::kBFloat16, false);
    Cache4 h = cache4(c, cache_at, P, s[2], c.int32(4, "page_size"));
    if (h.Hkv != s[1]) raise(PyExc_ValueError, "%s: the cache holds %d heads, k %lld", c.what, h.Hkv, (long long)s[1]);
    const long long* slots = (const long long*)c.one(slots_at, "slots", at::kLong, s[0]);
    if (write)
        return code(tp_kv4_write(in(k), in(v), as<void>(h.p), slots, P, (int)s[0], h.Hkv, (int)s[2], h.page, h.pages, k.row, v.row,
                                 c.stream(5)));
    return code(tp_kv4_read(in(h.p), slots, as<void>(k), as<void>(v), P, (int)s[0], h.Hkv, (int)s[2], h.page, h.pages, k.row, v.row,
                            c.stream(5)));
}
PyObject* kv4_write(const Args& c) { return kv4_rows(c, 0, 2, 3, true); }
// cache, slots, k, v, page_size
PyObject* kv4_read(const Args& c) { return kv4_rows(c, 2, 0, 1, false); }

// q, cache, o, block_table, lengths, page_size, shared, group, scale, ws
PyObject* decode_kv4(const Args& c) {
    int P;
    const auto s = leading(c, 0, "q", 3, P);
    const int64_t B = s[0], D = s[2];
    Ranks q = ranks(c, 0, "q", P, s, at::kBFloat16, false), o = ranks(c, 2, "o", P, s, at::kBFloat16, false);
    Cache4 h = cache4(c, 1, P, D, c.int32(5, "page_size"));
    const auto tab = sizes_of(c, 3, "block_table", 2, "(requests, pages)");
    if (tab[0] != B) raise(PyExc_ValueError, "%s: block_table is (%lld, pages), got %s", c.what, (long long)B, text(tab).c_str());
    const int* tp = (const int*)c.one(3, "block_table", at::kInt);
    const int* len = (const int*)c.one(4, "lengths", at::kInt, B);
    const int group = c.int32(7, "group");
    if (group < 1 || B % group) raise(PyExc_ValueError, "%s: %lld rows are not groups of %d", c.what, (long long)B, group);
    const int* shared = c.none(6) ? nullptr : (const int*)c.one(6, "shared", at::kInt, B / group);
    size_t bytes;
    void* ws = c.ws(9, bytes);
    return code(tp_attention_decode_kv4(in(q), in(h.p), as<void>(o), tp, len, shared, P, (int)B, group, (int)s[1], h.Hkv, (int)D,
                                        (int)tab[1], h.page, h.pages, q.row, o.row, c.real(8), ws, bytes, c.stream(10)));
}

struct Entry {
    const char* name;
    int args;               // before the stream and the current device, which every call ends with
    PyObject* (*call)(const Args&);
};
constexpr Entry kEntries[] = {{"kv_plan", 12, plan}, {"tp_qk_norm_rope", 12, rope}, {"tp_qk_norm_rope_grad", 13, rope_grad},
                              {"tp_attention", 9, prompt}, {"tp_attention_grad", 14, prompt_grad},
                              {"tp_attention_decode", 11, decode}, {"beam_select", 10, select}, {"kv_fork", 16, fork},
                              {"kv_compact", 10, compact}, {"kv_copy_pages", 4, copy_pages}, {"tp_kv4_write", 5, kv4_write},
                              {"tp_kv4_read", 5, kv4_read}, {"tp_attention_decode_kv4", 10, decode_kv4}};

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
PyMethodDef methods[] = {ENTRY(0), ENTRY(1), ENTRY(2), ENTRY(3), ENTRY(4), ENTRY(5), ENTRY(6), ENTRY(7), ENTRY(8), ENTRY(9),
                         ENTRY(10), ENTRY(11), ENTRY(12), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
