// The serving-step calls of binding.py, natively: argument checks on torch
// tensors, then the C ABI.  A decode step makes these calls once or more per
// layer and their kernels take a few microseconds: a call costs the host 3 us
// here (5 for prefix attention's three kernels), where the same checks through
// Python attributes made it 9 to 12.  Argument checks and marshalling only: what
// fails raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "pkv.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const char* name, const char* what) {
    PyErr_Format(PyExc_ValueError, "%s %s", name, what);
    throw Refused{};
}

// Arguments of one call, taken in order.
class Args {
  public:
    Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
            throw Refused{};
        }
    }
    long long integer() {
        const long long v = PyLong_AsLongLong(a_[i_++]);
        if (v == -1 && PyErr_Occurred()) throw Refused{};
        return v;
    }
    int32_t int32(const char* name) {
        const long long v = integer();
        if (v < INT32_MIN || v > INT32_MAX) refuse(name, "does not fit into 32 bits");
        return static_cast<int32_t>(v);
    }
    double real() {
        const double v = PyFloat_AsDouble(a_[i_++]);
        if (v == -1.0 && PyErr_Occurred()) throw Refused{};
        return v;
    }
    void* address() {
        void* p = PyLong_AsVoidPtr(a_[i_++]);
        if (!p && PyErr_Occurred()) throw Refused{};
        return p;
    }
    bool none() const { return a_[i_] == Py_None; }
    void skip() { ++i_; }
    const at::Tensor& tensor(const char* name) {
        PyObject* o = a_[i_++];
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
            throw Refused{};
        }
        return THPVariable_Unpack(o);
    }

  private:
    PyObject* const* a_;
    Py_ssize_t i_ = 0;
};

constexpr auto kAny = at::ScalarType::Undefined;

// The pool's device: index >= 0, or -1 for the CPU (a pool that no call can run on).
struct Place {
    int index;
    void check(const char* name, const at::Tensor& t) const {
        const at::Device d = t.device();
        if (index >= 0 ? !(d.is_cuda() && d.index() == index) : !d.is_cpu())
            refuse(name, "must be on the pool's device");
    }
    // Data of a contiguous tensor of this dtype and shape (an empty list: any shape).
    void* data(const char* name, const at::Tensor& t, at::ScalarType type,
               std::initializer_list<int64_t> shape = {}) const {
        check(name, t);
        if (type != kAny && t.scalar_type() != type) refuse(name, "has another dtype than the call takes");
        if (shape.size() > 0 && !t.sizes().equals(at::IntArrayRef(shape))) refuse(name, "has another shape than the call takes");
        if (!t.is_contiguous()) refuse(name, "must be contiguous");
        return t.data_ptr();
    }
    // (a CPU pool's tensors pass the checks above, so that these can be tested anywhere)
    void runnable() const {
        if (index < 0) refuse("the pool", "is not on a GPU");
    }
};

pkv_dtype code_of(const char* name, const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return PKV_F32;
        case at::kBFloat16: return PKV_BF16;
        case at::kFloat8_e4m3fn:
        case at::kByte: return PKV_FP8_E4M3;
        default: refuse(name, "has an unsupported dtype");
    }
}

int32_t table_width(const at::Tensor& t, int64_t num_seqs) {
    if (t.dim() != 2 || t.size(0) != num_seqs) refuse("block_tables", "must be [num_seqs, max_blocks]");
    if (t.size(1) > INT32_MAX) refuse("block_tables", "has too many columns");
    return static_cast<int32_t>(t.size(1));
}
int32_t count_of(const char* name, int64_t n) {
    if (n > INT32_MAX) refuse(name, "has too many elements");
    return static_cast<int32_t>(n);
}

// Token stride (elements) of x [T, heads, head_dim], whose heads lie one after the other.
int64_t head_rows(const Place& at_, const char* name, const at::Tensor& x, int64_t tokens, int64_t heads, int64_t dim,
                  at::ScalarType type) {
    at_.check(name, x);
    if (x.dim() != 3 || x.size(0) != tokens || x.size(1) != heads || x.size(2) != dim)
        refuse(name, "must be [T, heads, head_dim]");
    if (x.scalar_type() != type) refuse(name, "must have q's dtype");
    if (x.numel() > 0 && ((dim > 1 && x.stride(2) != 1) || (heads > 1 && x.stride(1) != dim)))
        refuse(name, "must hold a token's heads one after the other");
    return tokens > 1 ? x.stride(0) : 0;
}

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <typename F>
long released(F&& f) {  // the library call, without the interpreter lock
    struct Unlocked {
        PyThreadState* state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    return f();
}

// (pool, device, head_dim, layer, q, block_tables, seq_lens, max_seq_len, group_offsets, prefix_lens, scale, algo,
//  workspace | None, out, stream)
PyObject* prefix_attention(PyObject*, PyObject* const* argv, Py_ssize_t n) {
    return guarded([&]() -> long {
        Args a(argv, n, 15);
        const auto* pool = static_cast<const pkv_pool*>(a.address());
        const Place at_{a.int32("device")};
        const int64_t dim = a.integer();
        const int32_t layer = a.int32("layer");
        const at::Tensor& q = a.tensor("q");
        const at::Tensor& tables = a.tensor("block_tables");
        const at::Tensor& lens = a.tensor("seq_lens");
        const int32_t max_len = a.int32("max_seq_len");
        const at::Tensor& offsets = a.tensor("group_offsets");
        const at::Tensor& prefix = a.tensor("prefix_lens");
        const float scale = static_cast<float>(a.real());
        const auto algo = static_cast<pkv_algo>(a.int32("algo"));
        if (q.dim() != 3 || q.size(2) != dim) refuse("q", "must be [num_seqs, num_q_heads, head_dim]");
        if (prefix.dim() != 1) refuse("prefix_lens", "must be [num_groups]");
        const int64_t B = q.size(0), G = prefix.size(0);
        const int32_t width = table_width(tables, B), num_seqs = count_of("q", B), heads = count_of("q", q.size(1));
        const int32_t groups = count_of("prefix_lens", G);
        const void* pq = at_.data("q", q, kAny);
        const pkv_dtype type = code_of("q", q);
        const auto* pt = static_cast<const int32_t*>(at_.data("block_tables", tables, at::kInt));
        const auto* pl = static_cast<const int32_t*>(at_.data("seq_lens", lens, at::kInt, {B}));
        const auto* po = static_cast<const int32_t*>(at_.data("group_offsets", offsets, at::kInt, {G + 1}));
        const auto* pp = static_cast<const int32_t*>(at_.data("prefix_lens", prefix, at::kInt));
        void* ws = nullptr;
        size_t ws_bytes = 0;
        if (a.none()) {
            a.skip();
        } else {
            const at::Tensor& w = a.tensor("workspace");
            ws = at_.data("workspace", w, kAny);
            ws_bytes = w.nbytes();
        }
        const at::Tensor& out = a.tensor("out");
        void* pout = at_.data("out", out, q.scalar_type(), {B, q.size(1), dim});
        void* stream = a.address();
        at_.runnable();
        return released([&] {
            return paged_prefix_decode_attention(pq, type, pool, layer, pt, width, pl, num_seqs, heads, max_len, po,
                                                 pp, groups, scale, algo, ws, ws_bytes, pout, stream);
        });
    });
}

// (pool, device, kv_heads, head_dim, f32, layer, q, k, v, positions, slot_mapping, cos_sin, axes, sections,
//  interleaved, q_weight | None, k_weight | None, eps, out, stream); out's dtype is float32 for f32, else bfloat16
PyObject* norm_rope(PyObject*, PyObject* const* argv, Py_ssize_t n) {
    return guarded([&]() -> long {
        Args a(argv, n, 20);
        const auto* pool = static_cast<const pkv_pool*>(a.address());
        const Place at_{a.int32("device")};
        const int64_t kv_heads = a.integer(), dim = a.integer();
        const at::ScalarType out_type = a.integer() ? at::kFloat : at::kBFloat16;
        const int32_t layer = a.int32("layer");
        const at::Tensor& q = a.tensor("q");
        const at::Tensor& k = a.tensor("k");
        const at::Tensor& v = a.tensor("v");
        const at::Tensor& positions = a.tensor("positions");
        const at::Tensor& slots = a.tensor("slot_mapping");
        const at::Tensor& cos_sin = a.tensor("cos_sin");
        if (q.dim() != 3) refuse("q", "must be [T, num_q_heads, head_dim]");
        const int64_t T = q.size(0), Hq = q.size(1);
        const int64_t qs = head_rows(at_, "q", q, T, Hq, dim, q.scalar_type());
        const int64_t ks = head_rows(at_, "k", k, T, kv_heads, dim, q.scalar_type());
        const int64_t vs = head_rows(at_, "v", v, T, kv_heads, dim, q.scalar_type());
        pkv_norm_rope r{};
        r.cos_sin = static_cast<const float*>(at_.data("cos_sin", cos_sin, at::kFloat));
        if (cos_sin.dim() != 2) refuse("cos_sin", "must be [max_pos, rotary_dim]");
        r.max_pos = count_of("cos_sin", cos_sin.size(0));
        r.rotary_dim = count_of("cos_sin", cos_sin.size(1));
        r.num_axes = a.int32("axes");
        const long long packed = a.integer();  // the sections, 20 bits each
        for (int i = 0; i < 3; ++i) r.sections[i] = static_cast<int32_t>((packed >> (20 * i)) & 0xFFFFF);
        r.interleaved = a.int32("interleaved");
        if (a.none()) {
            a.skip();
            if (!a.none()) refuse("q_weight", "and k_weight go together");
            a.skip();
            a.skip();  // eps
        } else {
            const at::Tensor& qw = a.tensor("q_weight");
            if (a.none()) refuse("q_weight", "and k_weight go together");
            const at::Tensor& kw = a.tensor("k_weight");
            r.q_weight = at_.data("q_weight", qw, kAny, {dim});
            r.k_weight = at_.data("k_weight", kw, qw.scalar_type(), {dim});
            r.weight_dtype = code_of("q_weight", qw);
            r.eps = static_cast<float>(a.real());
        }
        const void* pp = r.num_axes == 1 && positions.dim() == 1 ? at_.data("positions", positions, at::kInt, {T})
                                                                 : at_.data("positions", positions, at::kInt, {r.num_axes, T});
        const void* ps = at_.data("slot_mapping", slots, at::kLong, {T});
        const at::Tensor& out = a.tensor("out");
        void* po = at_.data("out", out, out_type, {T, Hq, dim});
        void* stream = a.address();
        const pkv_dtype type = code_of("q", q);
        const int32_t tokens = count_of("q", T), heads = count_of("q", Hq);
        at_.runnable();
        const void *pq = q.data_ptr(), *pk = k.data_ptr(), *pv = v.data_ptr();
        return released([&] {
            return kv_append_norm_rope(pool, layer, pq, pk, pv, type, qs, ks, vs, static_cast<const int32_t*>(pp),
                                       static_cast<const int64_t*>(ps), tokens, heads, &r, po, stream);
        });
    });
}

// (pool, device, block_tables, seq_lens, new_tokens, free_ring, free_state, max_tokens, slot_mapping, positions,
//  token_seqs, token_offsets, granted, seq_lens_out, free_state_out, stream)
PyObject* tables_grow(PyObject*, PyObject* const* argv, Py_ssize_t n) {
    return guarded([&]() -> long {
        Args a(argv, n, 16);
        const auto* pool = static_cast<const pkv_pool*>(a.address());
        const Place at_{a.int32("device")};
        const at::Tensor& tables = a.tensor("block_tables");
        const at::Tensor& lens = a.tensor("seq_lens");
        if (lens.dim() != 1) refuse("seq_lens", "must be [num_seqs]");
        const int64_t B = lens.size(0);
        const int32_t width = table_width(tables, B), num_seqs = count_of("seq_lens", B);
        auto i32 = [&](const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape = {}) {
            return static_cast<int32_t*>(at_.data(name, t, at::kInt, shape));
        };
        int32_t* pt = i32("block_tables", tables);
        const int32_t* pl = i32("seq_lens", lens);
        const int32_t* pn = i32("new_tokens", a.tensor("new_tokens"), {B});
        const at::Tensor& ring = a.tensor("free_ring");
        const int32_t* pr = i32("free_ring", ring);
        const int32_t* pf = i32("free_state", a.tensor("free_state"), {2});
        const int32_t T = a.int32("max_tokens");
        auto* slots = static_cast<int64_t*>(at_.data("slot_mapping", a.tensor("slot_mapping"), at::kLong, {T}));
        int32_t* positions = i32("positions", a.tensor("positions"), {T});
        int32_t* seqs = i32("token_seqs", a.tensor("token_seqs"), {T});
        int32_t* offsets = i32("token_offsets", a.tensor("token_offsets"), {B + 1});
        int32_t* granted = i32("granted", a.tensor("granted"), {B});
        int32_t* lens_out = i32("out.seq_lens", a.tensor("out.seq_lens"), {B});
        int32_t* free_out = i32("out.free_state", a.tensor("out.free_state"), {2});
        void* stream = a.address();
        const int32_t ring_size = count_of("free_ring", ring.numel());
        at_.runnable();
        return released([&] {
            return kv_tables_grow(pool, pt, width, pl, pn, num_seqs, pr, ring_size, pf, T, slots, positions, seqs, offsets,
                                  granted, lens_out, free_out, stream);
        });
    });
}

// (pool, device, block_tables, seq_lens, finished, keep_blocks | None, free_ring, free_state, seq_lens_out,
//  free_state_out, stream)
PyObject* tables_release(PyObject*, PyObject* const* argv, Py_ssize_t n) {
    return guarded([&]() -> long {
        Args a(argv, n, 11);
        const auto* pool = static_cast<const pkv_pool*>(a.address());
        const Place at_{a.int32("device")};
        const at::Tensor& tables = a.tensor("block_tables");
        const at::Tensor& lens = a.tensor("seq_lens");
        if (lens.dim() != 1) refuse("seq_lens", "must be [num_seqs]");
        const int64_t B = lens.size(0);
        const int32_t width = table_width(tables, B), num_seqs = count_of("seq_lens", B);
        auto i32 = [&](const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape = {}) {
            return static_cast<int32_t*>(at_.data(name, t, at::kInt, shape));
        };
        const int32_t* pt = i32("block_tables", tables);
        const int32_t* pl = i32("seq_lens", lens);
        const int32_t* pd = i32("finished", a.tensor("finished"), {B});
        const int32_t* pk = nullptr;
        if (a.none()) a.skip();
        else pk = i32("keep_blocks", a.tensor("keep_blocks"), {B});
        const at::Tensor& ring = a.tensor("free_ring");
        int32_t* pr = i32("free_ring", ring);
        const int32_t* pf = i32("free_state", a.tensor("free_state"), {2});
        int32_t* lens_out = i32("seq_lens_out", a.tensor("seq_lens_out"), {B});
        int32_t* free_out = i32("free_state_out", a.tensor("free_state_out"), {2});
        void* stream = a.address();
        const int32_t ring_size = count_of("free_ring", ring.numel());
        at_.runnable();
        return released([&] {
            return kv_tables_release(pool, pt, width, pl, pd, pk, num_seqs, pr, ring_size, pf, lens_out, free_out, stream);
        });
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<prefix_attention>("prefix_attention"), method<norm_rope>("norm_rope"),
                         method<tables_grow>("tables_grow"), method<tables_release>("tables_release"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkvstep", "Native argument checks of the serving-step calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkvstep() { return PyModule_Create(&module); }
