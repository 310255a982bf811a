// binding.cpp -- native argument marshalling of the tree-draft operators and of
// those around a verification step: the checks of the tensors and the call of the C ABI.
//
// These calls sit between the small launches of a decoding loop.  With up to
// 15 tensors each, looking at type, shape, strides, device and address from
// Python took 8 to 15 us a call, more than most of the kernels; here it takes
// well under one.  The module is told the addresses of the library's functions
// (bind), so it links to no particular build of the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <initializer_list>
#include <string>

#include "mtp_rs.h"

namespace {

struct Functions {
    decltype(&mtp_tree_attention) attention = nullptr;
    decltype(&mtp_tree_attention_workspace) attention_ws = nullptr;
    decltype(&mtp_beam_select) select = nullptr;
    decltype(&mtp_beam_select_workspace) select_ws = nullptr;
    decltype(&mtp_beam_reorder) reorder = nullptr;
    decltype(&mtp_tree_commit) commit = nullptr;
    decltype(&mtp_prefix_attention) prefix = nullptr;
    decltype(&mtp_prefix_attention_workspace) prefix_ws = nullptr;
    decltype(&mtp_rope) rope = nullptr;
    decltype(&mtp_cache_append) append = nullptr;
    decltype(&mtp_adjust_logits) adjust = nullptr;
} fn;

constexpr int NOT_BOUND = -1;  // what a call returns before bind()

// A refusal: the Python exception's type and text.
struct Refusal {
    PyObject *type;
    std::string text;
};
[[noreturn]] void type_error(const std::string &s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refusal{PyExc_ValueError, s}; }

std::string show(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + (v.size() == 1 ? ",)" : ")");
}

const char *dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        default: return c10::toString(t);
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (o == Py_None) value_error(std::string(name) + " is required");
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor &t) {
    if (t.scalar_type() == at::kFloat) return MTP_DTYPE_F32;
    if (t.scalar_type() == at::kBFloat16) return MTP_DTYPE_BF16;
    type_error(std::string("logits, queries and states must be float32 or bfloat16, got ") + dtype_name(t.scalar_type()));
}

int index_of(const at::Tensor &t) { return t.is_cuda() ? t.get_device() : -1; }

using Shape = std::initializer_list<int64_t>;

void check(const at::Tensor &t, const char *name, at::ScalarType dtype, Shape shape, int index) {
    if (t.scalar_type() != dtype)
        type_error(std::string(name) + " must be " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
    if (t.sizes() != at::IntArrayRef(shape))
        value_error(std::string(name) + " must have shape " + show(at::IntArrayRef(shape)) + ", got " + show(t.sizes()));
    if (index_of(t) != index) value_error(std::string(name) + " must be on the device of the other tensors");
}

// The address of a contiguous tensor of this type and shape.
void *whole(PyObject *o, const char *name, at::ScalarType dtype, Shape shape, int index) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, dtype, shape, index);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void *whole_or_null(PyObject *o, const char *name, at::ScalarType dtype, Shape shape, int index) {
    return o == Py_None ? nullptr : whole(o, name, dtype, shape, index);
}
// The same where only the last dimension has to be contiguous; the strides of
// the others go to `strides`.
void *strided(const at::Tensor &t, const char *name, at::ScalarType dtype, Shape shape, int index, int64_t *strides) {
    check(t, name, dtype, shape, index);
    const auto s = t.strides();
    if (s.back() != 1 && t.sizes().back() != 1) value_error(std::string(name) + " must be contiguous in its last dimension");
    for (size_t i = 0; i + 1 < s.size(); ++i) strides[i] = s[i];
    return t.data_ptr();
}

void dims(const at::Tensor &t, const char *name, int64_t n) {
    if (t.dim() != n)
        value_error(std::string(name) + " must have " + std::to_string(n) + " dimensions, got " + show(t.sizes()));
}
void on_gpu(int index, const char *name) {
    if (index < 0) value_error(std::string(name) + " must be a CUDA tensor");
}

// Scratch memory on t's device, of the current stream, which is the call's; the
// tensor keeps it until the launch is done.
at::Tensor workspace(int64_t bytes, const at::Tensor &t) { return at::empty({bytes}, t.options().dtype(at::kByte)); }

mtp_stream_t stream_of(PyObject *o) { return reinterpret_cast<mtp_stream_t>(PyLong_AsVoidPtr(o)); }

// The library call itself, with other Python threads free to run.
template <typename F>
long call(F f) {
    PyThreadState *state = PyEval_SaveThread();
    const long rc = f();
    PyEval_RestoreThread(state);
    return rc;
}

template <typename F>
PyObject *guarded(F f) {
    try {
        const long rc = f();
        if (PyErr_Occurred()) return nullptr;
        return PyLong_FromLong(rc);
    } catch (const Refusal &r) {
        if (r.type) PyErr_SetString(r.type, r.text.c_str());  // (else Python's own error is set)
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
    return false;
}

// The arguments that tree_attention and prefix_attention share: q, k_new, v_new,
// k_cache, v_cache at a; page_table, cache_len, parents, n_nodes, scale, out,
// lse, row_flags at r.
int attention_args(PyObject *const *a, PyObject *const *r, mtp_tree_attention_args &s) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new"),
                     &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache"), &table = tensor(r[0], "page_table");
    dims(q, "q", 4);
    dims(k, "k_new", 4);
    dims(kc, "k_cache", 4);
    dims(table, "page_table", 2);
    const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), D = q.size(3), Hkv = k.size(2), pages = kc.size(0),
                  page = kc.size(1), most = table.size(1);
    const at::ScalarType dt = q.scalar_type();
    s.dtype = dtype_code(q);
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 4096)
        value_error("q has " + std::to_string(Hq) + " heads: not a multiple (up to 4096) of the " + std::to_string(Hkv) + " of k_new");
    if (T < 1 || T > MTP_MAX_NODES)
        value_error("trees have 1 to " + std::to_string(MTP_MAX_NODES) + " nodes, got " + std::to_string(T));
    if (D < 1 || D > 256) value_error("heads have 1 to 256 elements, got " + std::to_string(D));
    const double scale = PyFloat_AsDouble(r[4]);
    if (PyErr_Occurred()) throw Refusal{nullptr, ""};
    if (!(scale > 0.0 && scale < 1e30)) value_error("scale must be positive, got " + std::to_string(scale));
    const int index = index_of(q);
    s.out = whole(r[5], "out.out", dt, {B, T, Hq, D}, index);
    s.lse = static_cast<float *>(whole_or_null(r[6], "out.lse", at::kFloat, {B, T, Hq}, index));
    s.row_flags = static_cast<int32_t *>(whole_or_null(r[7], "out.row_flags", at::kInt, {B}, index));
    s.q = strided(q, "q", dt, {B, T, Hq, D}, index, s.q_stride);
    s.k_new = strided(k, "k_new", dt, {B, T, Hkv, D}, index, s.k_new_stride);
    s.v_new = strided(v, "v_new", dt, {B, T, Hkv, D}, index, s.v_new_stride);
    s.k_cache = strided(kc, "k_cache", dt, {pages, page, Hkv, D}, index, s.k_cache_stride);
    s.v_cache = strided(vc, "v_cache", dt, {pages, page, Hkv, D}, index, s.v_cache_stride);
    s.page_table = static_cast<int32_t *>(whole(r[0], "page_table", at::kInt, {B, most}, index));
    s.cache_len = static_cast<int32_t *>(whole(r[1], "cache_len", at::kInt, {B}, index));
    s.parents = static_cast<int32_t *>(whole_or_null(r[2], "parents", at::kInt, {B, T}, index));
    s.n_nodes = static_cast<int32_t *>(whole_or_null(r[3], "n_nodes", at::kInt, {B}, index));
    on_gpu(index, "q");
    for (int64_t x : {B, Hq, Hkv, pages, page, most})
        if (x > 0x7fffffff) value_error("a dimension is too large");
    s.B = static_cast<int>(B);
    s.T = static_cast<int>(T);
    s.Hq = static_cast<int>(Hq);
    s.Hkv = static_cast<int>(Hkv);
    s.D = static_cast<int>(D);
    s.num_pages = static_cast<int>(pages);
    s.page_size = static_cast<int>(page);
    s.max_pages = static_cast<int>(most);
    s.scale = static_cast<float>(scale);
    return index;
}

// tree_attention(q, k_new, v_new, k_cache, v_cache, page_table, cache_len,
//   parents, n_nodes, scale, out, lse, row_flags, stream)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 14)) return nullptr;
    return guarded([&]() -> long {
        mtp_tree_attention_args s = {};
        attention_args(a, a + 5, s);
        if (!fn.attention) return NOT_BOUND;
        const int64_t bytes = fn.attention_ws(&s);
        if (bytes < 0) return MTP_ERR_INVALID_ARG;
        const at::Tensor hold = workspace(bytes, THPVariable_Unpack(a[0]));
        s.workspace = hold.data_ptr();
        s.workspace_bytes = bytes;
        const mtp_stream_t stream = stream_of(a[13]);
        const auto f = fn.attention;  // (another thread may bind meanwhile)
        return call([&] { return f(&s, stream); });
    });
}

// prefix_attention(q, k_new, v_new, k_cache, v_cache, prefix_table, prefix_len,
//   group_start, page_table, cache_len, parents, n_nodes, scale, out, lse, row_flags, stream)
PyObject *prefix_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 17)) return nullptr;
    return guarded([&]() -> long {
        mtp_prefix_attention_args s = {};
        const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[5], "prefix_table");
        dims(table, "prefix_table", 2);
        const int index = index_of(q);
        const int64_t P = table.size(0), most = table.size(1);
        if (P < 1 || most < 1) value_error("at least one prefix and one page of it are needed, got " + show(table.sizes()));
        s.prefix_table = static_cast<int32_t *>(whole(a[5], "prefix_table", at::kInt, {P, most}, index));
        s.prefix_len = static_cast<int32_t *>(whole(a[6], "prefix_len", at::kInt, {P}, index));
        s.group_start = static_cast<int32_t *>(whole(a[7], "group_start", at::kInt, {P + 1}, index));
        attention_args(a, a + 8, s.own);
        for (int64_t x : {P, most})
            if (x > 0x7fffffff) value_error("a dimension is too large");
        s.prefixes = static_cast<int>(P);
        s.max_prefix_pages = static_cast<int>(most);
        if (!fn.prefix) return NOT_BOUND;
        const int64_t bytes = fn.prefix_ws(&s);
        if (bytes < 0) return MTP_ERR_INVALID_ARG;
        const at::Tensor hold = workspace(bytes, q);
        s.own.workspace = hold.data_ptr();
        s.own.workspace_bytes = bytes;
        const mtp_stream_t stream = stream_of(a[16]);
        const auto f = fn.prefix;
        return call([&] { return f(&s, stream); });
    });
}

// beam_select(logits, scores, temperature, K, tokens, parents, out_scores,
//   row_flags, stream)
PyObject *beam_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 9)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &z = tensor(a[0], "logits");
        dims(z, "logits", 3);
        const int64_t B = z.size(0), W = z.size(1), V = z.size(2);
        const int code = dtype_code(z);
        const int64_t K = PyLong_AsLongLong(a[3]);
        if (PyErr_Occurred()) return 0;
        if (W < 1 || W > MTP_MAX_BEAMS)
            value_error("1 to " + std::to_string(MTP_MAX_BEAMS) + " beams, got " + std::to_string(W));
        if (K < 1 || K > MTP_MAX_SELECT || K > W * V)
            value_error("K must be 1 to " + std::to_string(MTP_MAX_SELECT) + " and at most W V, got " + std::to_string(K));
        const int index = index_of(z);
        int32_t *tokens = static_cast<int32_t *>(whole(a[4], "out.tokens", at::kInt, {B, K}, index));
        int32_t *parents = static_cast<int32_t *>(whole(a[5], "out.parents", at::kInt, {B, K}, index));
        float *best = static_cast<float *>(whole(a[6], "out.scores", at::kFloat, {B, K}, index));
        int32_t *flags = static_cast<int32_t *>(whole_or_null(a[7], "out.row_flags", at::kInt, {B}, index));
        const void *pz = whole(a[0], "logits", z.scalar_type(), {B, W, V}, index);
        const float *scores = static_cast<float *>(whole(a[1], "scores", at::kFloat, {B, W}, index));
        const float *temp = static_cast<float *>(whole(a[2], "temperature", at::kFloat, {B}, index));
        on_gpu(index, "logits");
        if (B > 0x7fffffff || V > 0x7fffffff) value_error("a dimension is too large");
        if (!fn.select) return NOT_BOUND;
        const int b = static_cast<int>(B), w = static_cast<int>(W), v = static_cast<int>(V), k = static_cast<int>(K);
        const mtp_dtype dt = static_cast<mtp_dtype>(code);
        const int64_t bytes = fn.select_ws(dt, b, w, v, k);
        if (bytes < 0) return MTP_ERR_INVALID_ARG;
        const at::Tensor hold = workspace(bytes, z);
        void *ws = hold.data_ptr();
        const mtp_stream_t stream = stream_of(a[8]);
        const auto f = fn.select;
        return call([&] { return f(pz, dt, scores, temp, b, w, v, k, tokens, parents, best, flags, ws, bytes, stream); });
    });
}

// beam_reorder(states, parents, out_states, row_flags, stream)
PyObject *beam_reorder(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 5)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &x = tensor(a[0], "states"), &up = tensor(a[1], "parents");
        if (x.dim() < 3) value_error("states must be [N0, B, W, ...], got " + show(x.sizes()));
        dims(up, "parents", 2);
        const int64_t N0 = x.size(0), B = x.size(1), W = x.size(2), K = up.size(1);
        if (W < 1 || K < 1)
            value_error("at least one beam and one place are needed, got W = " + std::to_string(W) + ", K = " + std::to_string(K));
        const int index = index_of(x);
        int64_t row = static_cast<int64_t>(x.element_size());
        for (int64_t d = 3; d < x.dim(); ++d) row *= x.size(d);
        const at::Tensor &out = tensor(a[2], "out.states");
        if (out.scalar_type() != x.scalar_type())
            type_error(std::string("out.states must be ") + dtype_name(x.scalar_type()) + ", got " + dtype_name(out.scalar_type()));
        bool fits = out.dim() == x.dim() && out.size(0) == N0 && out.size(1) == B && out.size(2) == K;
        for (int64_t d = 3; fits && d < x.dim(); ++d) fits = out.size(d) == x.size(d);
        if (!fits) value_error("out.states must be [N0, B, K, ...] like states, got " + show(out.sizes()));
        if (!out.is_contiguous()) value_error("out.states must be contiguous");
        if (index_of(out) != index) value_error("out.states must be on the device of the other tensors");
        int32_t *flags = static_cast<int32_t *>(whole_or_null(a[3], "out.row_flags", at::kInt, {B}, index));
        if (!x.is_contiguous()) value_error("states must be contiguous");
        const int32_t *parents = static_cast<int32_t *>(whole(a[1], "parents", at::kInt, {B, K}, index));
        on_gpu(index, "states");
        for (int64_t d : {N0, B, W, K})
            if (d > 0x7fffffff) value_error("a dimension is too large");
        if (!fn.reorder) return NOT_BOUND;
        const mtp_stream_t stream = stream_of(a[4]);
        const auto f = fn.reorder;
        return call([&] {
            return f(x.data_ptr(), parents, static_cast<int>(N0), static_cast<int>(B), static_cast<int>(W),
                     static_cast<int>(K), row, out.data_ptr(), flags, stream);
        });
    });
}

// tree_commit(tokens, target_tokens, parents, k_new, v_new, k_cache, v_cache,
//   page_table, cache_len, n_nodes, out_tokens, accept_len, path, new_len,
//   row_flags, stream)
PyObject *tree_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 16)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &tokens = tensor(a[0], "tokens");
        dims(tokens, "tokens", 2);
        const int64_t B = tokens.size(0), T = tokens.size(1);
        if (T < 1 || T > MTP_MAX_NODES)
            value_error("trees have 1 to " + std::to_string(MTP_MAX_NODES) + " nodes, got " + std::to_string(T));
        mtp_tree_commit_args s = {};
        const int index = index_of(tokens);
        s.out_tokens = static_cast<int32_t *>(whole(a[10], "out.tokens", at::kInt, {B, T}, index));
        s.accept_len = static_cast<int32_t *>(whole(a[11], "out.accept_len", at::kInt, {B}, index));
        s.path = static_cast<int32_t *>(whole(a[12], "out.path", at::kInt, {B, T}, index));
        s.new_len = static_cast<int32_t *>(whole(a[13], "out.cache_len", at::kInt, {B}, index));
        s.row_flags = static_cast<int32_t *>(whole_or_null(a[14], "out.row_flags", at::kInt, {B}, index));
        s.tokens = static_cast<int32_t *>(whole(a[0], "tokens", at::kInt, {B, T}, index));
        s.target_tokens = static_cast<int32_t *>(whole(a[1], "target_tokens", at::kInt, {B, T}, index));
        s.parents = static_cast<int32_t *>(whole_or_null(a[2], "parents", at::kInt, {B, T}, index));
        s.n_nodes = static_cast<int32_t *>(whole_or_null(a[9], "n_nodes", at::kInt, {B}, index));
        s.B = static_cast<int>(B);
        s.T = static_cast<int>(T);
        if (B > 0x7fffffff) value_error("a dimension is too large");
        const auto launch = [&]() -> long {
            if (s.new_len == s.cache_len && B > 0) value_error("out.cache_len must not be cache_len itself");
            if (!fn.commit) return NOT_BOUND;
            const mtp_stream_t stream = stream_of(a[15]);
            const auto f = fn.commit;
            return call([&] { return f(&s, stream); });
        };
        if (a[3] == Py_None && a[4] == Py_None && a[5] == Py_None && a[6] == Py_None) {  // the verification alone
            if (a[7] != Py_None) value_error("page_table is of no use without k_new, v_new, k_cache and v_cache");
            s.cache_len = static_cast<int32_t *>(whole_or_null(a[8], "cache_len", at::kInt, {B}, index));
            on_gpu(index, "tokens");
            return launch();
        }
        const at::Tensor &k = tensor(a[3], "k_new"), &v = tensor(a[4], "v_new"), &kc = tensor(a[5], "k_cache"),
                         &vc = tensor(a[6], "v_cache"), &table = tensor(a[7], "page_table");
        s.dtype = dtype_code(k);
        const int one = k.dim() == 4 ? 1 : 0;  // without the layers' dimension
        dims(k, "k_new", 5 - one);
        dims(kc, "k_cache", 5 - one);
        dims(table, "page_table", 2);
        const int64_t layers = one ? 1 : k.size(0), Hkv = k.size(3 - one), D = k.size(4 - one), pages = kc.size(1 - one),
                      page = kc.size(2 - one), most = table.size(1);
        const at::ScalarType dt = k.scalar_type();
        if (one) {
            s.k_new = strided(k, "k_new", dt, {B, T, Hkv, D}, index, s.k_new_stride + 1);
            s.v_new = strided(v, "v_new", dt, {B, T, Hkv, D}, index, s.v_new_stride + 1);
            s.k_cache = strided(kc, "k_cache", dt, {pages, page, Hkv, D}, index, s.k_cache_stride + 1);
            s.v_cache = strided(vc, "v_cache", dt, {pages, page, Hkv, D}, index, s.v_cache_stride + 1);
        } else {
            s.k_new = strided(k, "k_new", dt, {layers, B, T, Hkv, D}, index, s.k_new_stride);
            s.v_new = strided(v, "v_new", dt, {layers, B, T, Hkv, D}, index, s.v_new_stride);
            s.k_cache = strided(kc, "k_cache", dt, {layers, pages, page, Hkv, D}, index, s.k_cache_stride);
            s.v_cache = strided(vc, "v_cache", dt, {layers, pages, page, Hkv, D}, index, s.v_cache_stride);
        }
        s.page_table = static_cast<int32_t *>(whole(a[7], "page_table", at::kInt, {B, most}, index));
        s.cache_len = static_cast<int32_t *>(whole(a[8], "cache_len", at::kInt, {B}, index));
        on_gpu(index, "tokens");
        for (int64_t x : {layers, Hkv, D, pages, page, most})
            if (x > 0x7fffffff) value_error("a dimension is too large");
        s.layers = static_cast<int>(layers);
        s.Hkv = static_cast<int>(Hkv);
        s.D = static_cast<int>(D);
        s.num_pages = static_cast<int>(pages);
        s.page_size = static_cast<int>(page);
        s.max_pages = static_cast<int>(most);
        return launch();
    });
}

// What mtp_rope and mtp_cache_append have in common: the frequencies and what
// their number has to fit.
int pairs_of(PyObject *o, const float **inv_freq, int64_t D, int index) {
    const at::Tensor &f = tensor(o, "inv_freq");
    dims(f, "inv_freq", 1);
    const int64_t n = f.size(0);
    if (2 * n > D) value_error("inv_freq has " + std::to_string(n) + " angles: more than pairs in a head of " + std::to_string(D));
    *inv_freq = static_cast<float *>(whole(o, "inv_freq", at::kFloat, {n}, index));
    return static_cast<int>(n);
}
const int32_t *positions_of(PyObject *o, int64_t B, int64_t T, int index, int64_t *strides) {
    const at::Tensor &p = tensor(o, "positions");
    check(p, "positions", at::kInt, {B, T}, index);
    strides[0] = p.stride(0);
    strides[1] = p.stride(1);
    return static_cast<int32_t *>(p.data_ptr());
}
float finite(PyObject *o, const char *name) {
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Refusal{nullptr, ""};
    const float f = static_cast<float>(x);
    if (!(f - f == 0.f)) value_error(std::string(name) + " must be finite, got " + std::to_string(x));
    return f;
}
void small(std::initializer_list<int64_t> sizes) {
    for (int64_t x : sizes)
        if (x > 0x7fffffff) value_error("a dimension is too large");
}
void head_size(int64_t D) {
    if (D < 1 || D > 256) value_error("heads have 1 to 256 elements, got " + std::to_string(D));
}

// rope(q, k, positions, inv_freq, interleaved, factor, inverse, q_out, k_out, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 10)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &q = tensor(a[0], "q");
        dims(q, "q", 4);
        mtp_rope_args s = {};
        const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), D = q.size(3);
        const at::ScalarType dt = q.scalar_type();
        s.dtype = dtype_code(q);
        head_size(D);
        const int index = index_of(q);
        int64_t Hkv = 0;
        s.q_out = strided(tensor(a[7], "out.q"), "out.q", dt, {B, T, Hq, D}, index, s.q_out_stride);
        if (a[1] != Py_None) {
            const at::Tensor &k = tensor(a[1], "k");
            dims(k, "k", 4);
            Hkv = k.size(2);
            s.k = strided(k, "k", dt, {B, T, Hkv, D}, index, s.k_stride);
            s.k_out = strided(tensor(a[8], "out.k"), "out.k", dt, {B, T, Hkv, D}, index, s.k_out_stride);
        } else if (a[8] != Py_None) {
            value_error("out.k is of no use without k");
        }
        s.q = strided(q, "q", dt, {B, T, Hq, D}, index, s.q_stride);
        s.positions = positions_of(a[2], B, T, index, s.pos_stride);
        s.pairs = pairs_of(a[3], &s.inv_freq, D, index);
        s.factor = finite(a[5], "factor");
        on_gpu(index, "q");
        small({B, T, Hq, Hkv});
        s.B = static_cast<int>(B);
        s.T = static_cast<int>(T);
        s.Hq = static_cast<int>(Hq);
        s.Hkv = static_cast<int>(Hkv);
        s.D = static_cast<int>(D);
        s.interleaved = a[4] == Py_True;
        s.inverse = a[6] == Py_True;
        if (!fn.rope) return NOT_BOUND;
        const mtp_stream_t stream = stream_of(a[9]);
        const auto f = fn.rope;
        return call([&] { return f(&s, stream); });
    });
}

// cache_append(k, v, k_cache, v_cache, page_table, cache_len, n_new, q,
//   inv_freq, positions, interleaved, factor, new_len, q_out, k_out, row_flags, stream)
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 17)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache"),
                         &table = tensor(a[4], "page_table");
        dims(k, "k", 4);
        dims(kc, "k_cache", 4);
        dims(table, "page_table", 2);
        mtp_cache_append_args s = {};
        const int64_t B = k.size(0), T = k.size(1), Hkv = k.size(2), D = k.size(3), pages = kc.size(0), page = kc.size(1), most = table.size(1);
        const at::ScalarType dt = k.scalar_type();
        s.dtype = dtype_code(k);
        head_size(D);
        const int index = index_of(k);
        s.new_len = static_cast<int32_t *>(whole(a[12], "out.cache_len", at::kInt, {B}, index));
        s.row_flags = static_cast<int32_t *>(whole_or_null(a[15], "out.row_flags", at::kInt, {B}, index));
        s.k = strided(k, "k", dt, {B, T, Hkv, D}, index, s.k_stride);
        s.v = strided(v, "v", dt, {B, T, Hkv, D}, index, s.v_stride);
        s.k_cache = strided(kc, "k_cache", dt, {pages, page, Hkv, D}, index, s.k_cache_stride);
        s.v_cache = strided(vc, "v_cache", dt, {pages, page, Hkv, D}, index, s.v_cache_stride);
        s.page_table = static_cast<int32_t *>(whole(a[4], "page_table", at::kInt, {B, most}, index));
        s.cache_len = static_cast<int32_t *>(whole(a[5], "cache_len", at::kInt, {B}, index));
        s.n_new = static_cast<int32_t *>(whole_or_null(a[6], "n_new", at::kInt, {B}, index));
        int64_t Hq = 0;
        if (a[7] != Py_None) {
            const at::Tensor &q = tensor(a[7], "q");
            dims(q, "q", 4);
            Hq = q.size(2);
            if (a[8] == Py_None) value_error("q is of no use without inv_freq");
            s.q = strided(q, "q", dt, {B, T, Hq, D}, index, s.q_stride);
            s.q_out = strided(tensor(a[13], "out.q"), "out.q", dt, {B, T, Hq, D}, index, s.q_out_stride);
        } else if (a[13] != Py_None) {
            value_error("out.q is of no use without q");
        }
        if (a[14] != Py_None) s.k_out = strided(tensor(a[14], "out.k"), "out.k", dt, {B, T, Hkv, D}, index, s.k_out_stride);
        if (a[8] != Py_None) s.pairs = pairs_of(a[8], &s.inv_freq, D, index);
        if (a[9] != Py_None) {
            if (a[8] == Py_None) value_error("positions are of no use without inv_freq");
            s.positions = positions_of(a[9], B, T, index, s.pos_stride);
        }
        s.factor = finite(a[11], "factor");
        on_gpu(index, "k");
        small({B, T, Hq, Hkv, pages, page, most});
        s.B = static_cast<int>(B);
        s.T = static_cast<int>(T);
        s.Hq = static_cast<int>(Hq);
        s.Hkv = static_cast<int>(Hkv);
        s.D = static_cast<int>(D);
        s.interleaved = a[10] == Py_True;
        s.num_pages = static_cast<int>(pages);
        s.page_size = static_cast<int>(page);
        s.max_pages = static_cast<int>(most);
        if (!fn.append) return NOT_BOUND;
        const mtp_stream_t stream = stream_of(a[16]);
        const auto f = fn.append;
        return call([&] { return f(&s, stream); });
    });
}

// adjust_logits(logits, history, history_len, prompt_len, tokens, parents,
//   n_nodes, repetition, frequency, presence, bias_ids, bias, mask, out, row_flags, stream)
PyObject *adjust_logits(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 16)) return nullptr;
    return guarded([&]() -> long {
        const at::Tensor &z = tensor(a[0], "logits");
        dims(z, "logits", 3);
        mtp_adjust_args s = {};
        const int64_t B = z.size(0), S = z.size(1), V = z.size(2);
        s.dtype = dtype_code(z);
        if (S < 1 || S > MTP_MAX_NODES)
            value_error("1 to " + std::to_string(MTP_MAX_NODES) + " rows of a sequence, got " + std::to_string(S));
        const int index = index_of(z);
        s.out = whole(a[13], "out.logits", z.scalar_type(), {B, S, V}, index);
        s.row_flags = static_cast<int32_t *>(whole_or_null(a[14], "out.row_flags", at::kInt, {B}, index));
        s.logits = whole(a[0], "logits", z.scalar_type(), {B, S, V}, index);
        int64_t L = 0;
        if (a[1] != Py_None) {
            const at::Tensor &h = tensor(a[1], "history");
            dims(h, "history", 2);
            L = h.size(1);
            s.history = static_cast<int32_t *>(whole(a[1], "history", at::kInt, {B, L}, index));
            s.history_len = static_cast<int32_t *>(whole(a[2], "history_len", at::kInt, {B}, index));
            s.prompt_len = static_cast<int32_t *>(whole_or_null(a[3], "prompt_len", at::kInt, {B}, index));
        } else if (a[2] != Py_None || a[3] != Py_None) {
            value_error("history_len and prompt_len are of no use without history");
        }
        s.tokens = static_cast<int32_t *>(whole_or_null(a[4], "tokens", at::kInt, {B, S}, index));
        s.parents = static_cast<int32_t *>(whole_or_null(a[5], "parents", at::kInt, {B, S}, index));
        if (s.parents && !s.tokens) value_error("parents are of no use without tokens");
        s.n_nodes = static_cast<int32_t *>(whole_or_null(a[6], "n_nodes", at::kInt, {B}, index));
        s.repetition = static_cast<float *>(whole_or_null(a[7], "repetition", at::kFloat, {B}, index));
        s.frequency = static_cast<float *>(whole_or_null(a[8], "frequency", at::kFloat, {B}, index));
        s.presence = static_cast<float *>(whole_or_null(a[9], "presence", at::kFloat, {B}, index));
        if ((a[10] == Py_None) != (a[11] == Py_None)) value_error("bias_ids and bias are of no use without each other");
        int64_t biases = 0;
        if (a[10] != Py_None) {
            const at::Tensor &ids = tensor(a[10], "bias_ids");
            dims(ids, "bias_ids", 2);
            biases = ids.size(1);
            if (biases > MTP_MAX_BIAS) value_error("at most " + std::to_string(MTP_MAX_BIAS) + " biases, got " + std::to_string(biases));
            s.bias_ids = static_cast<int32_t *>(whole(a[10], "bias_ids", at::kInt, {B, biases}, index));
            s.bias = static_cast<float *>(whole(a[11], "bias", at::kFloat, {B, biases}, index));
        }
        if (a[12] != Py_None) {
            const at::Tensor &m = tensor(a[12], "mask");
            s.mask = static_cast<int32_t *>(strided(m, "mask", at::kInt, {B, S, (V + 31) / 32}, index, s.mask_stride));
        }
        on_gpu(index, "logits");
        if (B > (1 << 20)) value_error("at most 2^20 sequences, got " + std::to_string(B));
        if (V < 1 || V > (1 << 24)) value_error("a vocabulary has 1 to 2^24 entries, got " + std::to_string(V));
        if (L > (1 << 28)) value_error("a history has at most 2^28 tokens, got " + std::to_string(L));
        s.B = static_cast<int>(B);
        s.S = static_cast<int>(S);
        s.V = static_cast<int>(V);
        s.L = static_cast<int>(L);
        s.n_bias = static_cast<int>(biases);
        if (!fn.adjust) return NOT_BOUND;
        const mtp_stream_t stream = stream_of(a[15]);
        const auto f = fn.adjust;
        return call([&] { return f(&s, stream); });
    });
}

// bind(addresses of the functions, in the order of Functions)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int N = 11;
    if (!count(n, N)) return nullptr;
    void *p[N];
    for (int i = 0; i < N; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    fn.attention = reinterpret_cast<decltype(fn.attention)>(p[0]);
    fn.attention_ws = reinterpret_cast<decltype(fn.attention_ws)>(p[1]);
    fn.select = reinterpret_cast<decltype(fn.select)>(p[2]);
    fn.select_ws = reinterpret_cast<decltype(fn.select_ws)>(p[3]);
    fn.reorder = reinterpret_cast<decltype(fn.reorder)>(p[4]);
    fn.commit = reinterpret_cast<decltype(fn.commit)>(p[5]);
    fn.prefix = reinterpret_cast<decltype(fn.prefix)>(p[6]);
    fn.prefix_ws = reinterpret_cast<decltype(fn.prefix_ws)>(p[7]);
    fn.rope = reinterpret_cast<decltype(fn.rope)>(p[8]);
    fn.append = reinterpret_cast<decltype(fn.append)>(p[9]);
    fn.adjust = reinterpret_cast<decltype(fn.adjust)>(p[10]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_attention)), METH_FASTCALL, nullptr},
    {"beam_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(beam_select)), METH_FASTCALL, nullptr},
    {"beam_reorder", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(beam_reorder)), METH_FASTCALL, nullptr},
    {"tree_commit", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_commit)), METH_FASTCALL, nullptr},
    {"prefix_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attention)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_append)), METH_FASTCALL, nullptr},
    {"adjust_logits", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adjust_logits)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
