// torch_calls.cpp -- the entry points of the block-sparse step and of shared pages called with torch
// tensors: checks of types, shapes, packing and device, then the C call on the
// current stream. A Python module of its own next to libpka.so, which stays free
// of torch: a launch of these calls takes some microseconds, and the checks and
// conversions of up to 28 arguments in Python took 8 to 21 us.
//
// Each function returns the call's status (the caller raises for it) and raises
// ValueError itself for a tensor that is not what the call is told it is.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <sstream>

#include "pka.h"

namespace {

using at::Tensor;
constexpr auto kI8 = at::kChar, kU8 = at::kByte, kI32 = at::kInt, kI64 = at::kLong, kF32 = at::kFloat;
constexpr auto kBf16 = at::kBFloat16;

struct Raised {};  // the Python error is set

[[noreturn]] void refuse(const std::string& text) {
    PyErr_SetString(PyExc_ValueError, text.c_str());
    throw Raised();
}

int64_t integer(PyObject* o, int64_t limit = INT32_MAX) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    if (x > limit || x < -limit) refuse("an integer argument is out of range");
    return x;
}

float number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)x;
}

class Call {
public:
    Call(const char* where, PyObject* stream) : where_(where), device_(c10::cuda::current_device()) {
        if (stream == Py_None) {
            stream_ = c10::cuda::getCurrentCUDAStream(device_).stream();
        } else {
            PyObject* n = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
            if (!n) throw Raised();
            stream_ = PyLong_AsVoidPtr(n);
            Py_DECREF(n);
            if (PyErr_Occurred()) throw Raised();
        }
    }
    void* stream() const { return stream_; }
    int64_t device() const { return device_; }

    const Tensor& tensor(PyObject* o, const char* name, int dims) const {
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s: %s must be a tensor, not %s", where_, name, Py_TYPE(o)->tp_name);
            throw Raised();
        }
        const Tensor& t = THPVariable_Unpack(o);
        if (t.dim() != dims) refuse(text(name) + "must have " + std::to_string(dims) + " dimensions");
        return t;
    }

    // The address of a packed tensor of that type and shape on the current device.
    void* packed(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
        const Tensor& t = tensor(o, name, (int)shape.size());
        if (t.scalar_type() != type || t.get_device() != device_ || !t.is_contiguous() ||
            !std::equal(shape.begin(), shape.end(), t.sizes().begin())) {
            std::ostringstream s;
            s << text(name) << "must be a packed " << c10::toString(type) << " tensor of shape "
              << at::IntArrayRef(shape) << " on the current CUDA device, not " << c10::toString(t.scalar_type()) << " "
              << t.sizes() << (t.is_contiguous() ? "" : " (not packed)") << " on " << t.device();
            refuse(s.str());
        }
        return t.data_ptr();
    }
    void* packed_or_none(PyObject* o, const char* name, at::ScalarType type,
                         std::initializer_list<int64_t> shape) const {
        return o == Py_None ? nullptr : packed(o, name, type, shape);
    }
    int32_t* word(PyObject* o) const { return static_cast<int32_t*>(packed_or_none(o, "error_word", kI32, {1})); }

    // Rows of packed heads, any distance apart.
    const void* rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t d, int64_t& stride) const {
        const Tensor& t = tensor(o, name, 3);
        const auto n = t.sizes(), by = t.strides();
        if (t.scalar_type() != kBf16 || t.get_device() != device_ || n[0] != tokens || n[1] != heads || n[2] != d)
            refuse(text(name) + "must be a BFloat16 tensor of shape [" + std::to_string(tokens) + ", " +
                   std::to_string(heads) + ", " + std::to_string(d) + "] on the current CUDA device");
        if (tokens > 0 && ((by[1] != d && heads > 1) || (by[2] != 1 && d > 1)))
            refuse(text(name) + "must have the heads of a row packed");
        stride = tokens > 1 ? by[0] : heads * d;  // (a single row's is free, and what an empty tensor has)
        return t.data_ptr();
    }

private:
    std::string text(const char* name) const { return std::string(where_) + ": " + name + " "; }
    const char* where_;
    c10::DeviceIndex device_;
    void* stream_;
};

// (without the interpreter's lock: a launch waits where the stream's queue is full)
template <typename F>
long unlocked(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const long status = f();
    PyEval_RestoreThread(state);
    return status;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t expected, F f) {
    if (given != expected) return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", expected, given);
    try {
        return PyLong_FromLong(f());
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <typename T = int32_t>
T* as(void* p) {
    return static_cast<T*>(p);
}
template <typename T = int32_t>
T* as(const void* p) {
    return static_cast<T*>(const_cast<void*>(p));
}

// The scales of an 8-bit cache; false for None.
bool scales_of(PyObject* o, float (&s)[2]) {
    if (o == Py_None) return false;
    PyObject* pair = PySequence_Fast(o, "kv_scales must be (k_scale, v_scale)");
    if (!pair) throw Raised();
    const bool two = PySequence_Fast_GET_SIZE(pair) == 2;
    double x[2] = {0, 0};
    for (int i = 0; two && i < 2; ++i) x[i] = PyFloat_AsDouble(PySequence_Fast_GET_ITEM(pair, i));
    Py_DECREF(pair);
    if (!two) refuse("kv_scales must be (k_scale, v_scale)");
    if (PyErr_Occurred()) throw Raised();
    s[0] = (float)x[0];
    s[1] = (float)x[1];
    return true;
}

// ctx_lens, query_lens, block_table, block_size, free_pages, free_head, free_head_out, query_start_loc, seq_lens,
// positions, slot_mapping, error_word, stream
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Call c("pka_step_tables", a[12]);
        const Tensor& table = c.tensor(a[2], "block_table", 2);
        const int64_t B = table.size(0), width = table.size(1), bs = integer(a[3]);
        const int64_t T = c.tensor(a[10], "slot_mapping", 1).size(0), pages = c.tensor(a[4], "free_pages", 1).size(0);
        if (B > INT32_MAX || width > INT32_MAX || pages > INT32_MAX) refuse("pka_step_tables: a size is out of range");
        auto* ctx = as(c.packed(a[0], "ctx_lens", kI32, {B}));
        auto* len = as(c.packed(a[1], "query_lens", kI32, {B}));
        auto* bt = as(c.packed(a[2], "block_table", kI32, {B, width}));
        auto* free = as(c.packed(a[4], "free_pages", kI32, {pages}));
        auto* head = as(c.packed(a[5], "free_head", kI32, {1}));
        auto* out = as(c.packed(a[6], "free_head_out", kI32, {1}));
        auto* qsl = as(c.packed(a[7], "query_start_loc", kI32, {B + 1}));
        auto* seq = as(c.packed(a[8], "seq_lens", kI32, {B}));
        auto* pos = as(c.packed_or_none(a[9], "positions", kI32, {T}));
        auto* slots = as<int64_t>(c.packed(a[10], "slot_mapping", kI64, {T}));
        int32_t* err = c.word(a[11]);
        return unlocked([&] {
            return pka_step_tables(ctx, len, (int)B, T, bt, (int)width, (int)bs, free, (int)pages, head, out, qsl, seq,
                                   pos, slots, err, c.stream());
        });
    });
}

// q, k, v, q_weight, k_weight, eps, cos_sin, interleaved, positions, slot_mapping, q_out, k_out, v_out, k_cache,
// v_cache, kv_scales, error_word, stream
PyObject* qk_rope_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 18, [&] {
        const Call c("pka_qk_rope_cache_write", a[17]);
        const Tensor &q = c.tensor(a[0], "q", 3), &k = c.tensor(a[1], "k", 3), &cache = c.tensor(a[13], "k_cache", 4);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k.size(1), nb = cache.size(0);
        const int64_t bs = cache.size(2);
        int64_t rotary = 0, longest = 0;
        if (a[6] != Py_None) {
            const Tensor& t = c.tensor(a[6], "cos_sin", 2);
            longest = t.size(0);
            rotary = t.size(1);
        }
        for (const int64_t x : {Hq, d, Hkv, bs, rotary, longest})
            if (x > INT32_MAX) refuse("pka_qk_rope_cache_write: a size is out of range");
        int64_t qs, ks, vs;
        const void* qp = c.rows(a[0], "q", T, Hq, d, qs);
        const void* kp = c.rows(a[1], "k", T, Hkv, d, ks);
        const void* vp = c.rows(a[2], "v", T, Hkv, d, vs);
        float scales[2];
        const bool fp8 = scales_of(a[15], scales);
        const auto kind = fp8 ? kU8 : kBf16;
        void* qw = c.packed_or_none(a[3], "q_weight", kBf16, {d});
        void* kw = c.packed_or_none(a[4], "k_weight", kBf16, {d});
        const float eps = number(a[5]);
        auto* cs = as<float>(c.packed_or_none(a[6], "cos_sin", kF32, {longest, rotary}));
        const int inter = PyObject_IsTrue(a[7]);
        if (inter < 0) throw Raised();
        auto* pos = as(c.packed(a[8], "positions", kI32, {T}));
        auto* slots = as<int64_t>(c.packed(a[9], "slot_mapping", kI64, {T}));
        void* qo = c.packed(a[10], "q_out", kBf16, {T, Hq, d});
        void* ko = c.packed_or_none(a[11], "k_out", kBf16, {T, Hkv, d});
        void* vo = c.packed_or_none(a[12], "v_out", kBf16, {T, Hkv, d});
        void* kc = c.packed(a[13], "k_cache", kind, {nb, Hkv, bs, d});
        void* vc = c.packed(a[14], "v_cache", kind, {nb, Hkv, bs, d});
        int32_t* err = c.word(a[16]);
        return unlocked([&] {
            if (fp8)
                return pka_qk_rope_cache_write_fp8(qp, kp, vp, qs, ks, vs, qw, kw, eps, cs, (int)rotary, (int)longest,
                                                   inter, pos, slots, T, (int)Hq, (int)Hkv, (int)d, qo, ko, vo, kc, vc,
                                                   nb, (int)bs, scales[0], scales[1], err, c.stream());
            return pka_qk_rope_cache_write(qp, kp, vp, qs, ks, vs, qw, kw, eps, cs, (int)rotary, (int)longest, inter,
                                           pos, slots, T, (int)Hq, (int)Hkv, (int)d, qo, ko, vo, kc, vc, nb, (int)bs,
                                           err, c.stream());
        });
    });
}

// k_cache, slot_mapping, bounds, bound_scales, error_word, stream
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const Call c("pka_page_bounds", a[5]);
        const Tensor& cache = c.tensor(a[0], "k_cache", 4);
        const int64_t nb = cache.size(0), Hkv = cache.size(1), bs = cache.size(2), d = cache.size(3);
        const int64_t T = c.tensor(a[1], "slot_mapping", 1).size(0);
        if (Hkv > INT32_MAX || bs > INT32_MAX || d > INT32_MAX) refuse("pka_page_bounds: a size is out of range");
        const bool fp8 = cache.scalar_type() == kU8;
        const void* kc = c.packed(a[0], "k_cache", fp8 ? kU8 : kBf16, {nb, Hkv, bs, d});
        auto* slots = as<int64_t>(c.packed(a[1], "slot_mapping", kI64, {T}));
        auto* bounds = as<int8_t>(c.packed(a[2], "bounds", kI8, {nb, Hkv, 2, d}));
        auto* scales = as<float>(c.packed(a[3], "bound_scales", kF32, {nb, Hkv}));
        int32_t* err = c.word(a[4]);
        return unlocked([&] {
            return pka_page_bounds(kc, fp8 ? 2 : 1, slots, T, (int)Hkv, (int)d, nb, (int)bs, bounds, scales, err,
                                   c.stream());
        });
    });
}

// q, bounds, bound_scales, block_table, query_start_loc, seq_lens, block_size, num_first, num_last, max_seq_len,
// selected, error_word, stream
PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Call c("pka_select_pages", a[12]);
        const Tensor &q = c.tensor(a[0], "q", 3), &units = c.tensor(a[2], "bound_scales", 2);
        const Tensor &table = c.tensor(a[3], "block_table", 2), &sel = c.tensor(a[10], "selected", 3);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), nb = units.size(0), Hkv = units.size(1);
        const int64_t B = table.size(0), width = table.size(1), K = sel.size(2);
        for (const int64_t x : {T, Hq, d, Hkv, B, width, K})
            if (x > INT32_MAX) refuse("pka_select_pages: a size is out of range");
        const int bs = (int)integer(a[6]), first = (int)integer(a[7]), last = (int)integer(a[8]);
        const int longest = (int)integer(a[9]);
        const void* qp = c.packed(a[0], "q", kBf16, {T, Hq, d});
        auto* bounds = as<int8_t>(c.packed(a[1], "bounds", kI8, {nb, Hkv, 2, d}));
        auto* scales = as<float>(c.packed(a[2], "bound_scales", kF32, {nb, Hkv}));
        auto* bt = as(c.packed(a[3], "block_table", kI32, {B, width}));
        auto* qsl = as(c.packed(a[4], "query_start_loc", kI32, {B + 1}));
        auto* seq = as(c.packed(a[5], "seq_lens", kI32, {B}));
        auto* list = as(c.packed(a[10], "selected", kI32, {T, Hkv, K}));
        int32_t* err = c.word(a[11]);
        return unlocked([&] {
            return pka_select_pages(qp, bounds, scales, bt, (int)width, qsl, seq, (int)B, (int)T, (int)Hq, (int)Hkv,
                                    (int)d, nb, bs, first, last, longest, (int)K, list, err, c.stream());
        });
    });
}

// q, k_cache, v_cache, block_table, query_start_loc, seq_lens, selected, scale, max_seq_len, out, lse, kv_scales,
// error_word, stream
PyObject* sparse_attn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const Call c("pka_sparse_attn_forward", a[13]);
        const Tensor &q = c.tensor(a[0], "q", 3), &cache = c.tensor(a[1], "k_cache", 4);
        const Tensor &table = c.tensor(a[3], "block_table", 2), &sel = c.tensor(a[6], "selected", 3);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), nb = cache.size(0), Hkv = cache.size(1);
        const int64_t bs = cache.size(2), B = table.size(0), width = table.size(1), K = sel.size(2);
        for (const int64_t x : {T, Hq, d, Hkv, bs, B, width, K})
            if (x > INT32_MAX) refuse("pka_sparse_attn_forward: a size is out of range");
        float scales[2];
        const bool fp8 = scales_of(a[11], scales);
        const auto kind = fp8 ? kU8 : kBf16;
        const float scale = number(a[7]);
        const int longest = (int)integer(a[8]);
        const void* qp = c.packed(a[0], "q", kBf16, {T, Hq, d});
        const void* kc = c.packed(a[1], "k_cache", kind, {nb, Hkv, bs, d});
        const void* vc = c.packed(a[2], "v_cache", kind, {nb, Hkv, bs, d});
        auto* bt = as(c.packed(a[3], "block_table", kI32, {B, width}));
        auto* qsl = as(c.packed(a[4], "query_start_loc", kI32, {B + 1}));
        auto* seq = as(c.packed(a[5], "seq_lens", kI32, {B}));
        auto* list = as(c.packed(a[6], "selected", kI32, {T, Hkv, K}));
        void* out = c.packed(a[9], "out", kBf16, {T, Hq, d});
        auto* lse = as<float>(c.packed_or_none(a[10], "lse", kF32, {T, Hq}));
        int32_t* err = c.word(a[12]);
        return unlocked([&] {
            if (fp8)
                return pka_sparse_attn_forward_fp8(qp, kc, vc, bt, (int)width, qsl, seq, (int)B, (int)T, (int)Hq,
                                                   (int)Hkv, (int)d, nb, (int)bs, scale, scales[0], scales[1], list,
                                                   (int)K, longest, out, lse, err, c.stream());
            return pka_sparse_attn_forward(qp, kc, vc, bt, (int)width, qsl, seq, (int)B, (int)T, (int)Hq, (int)Hkv,
                                           (int)d, nb, (int)bs, scale, list, (int)K, longest, out, lse, err,
                                           c.stream());
        });
    });
}

// logits, scores, out_scores, parents, tokens, end_token, finished, out_finished, error_word, stream
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const Call c("pka_beam_select", a[9]);
        const Tensor &x = c.tensor(a[0], "logits", 2), &s = c.tensor(a[1], "scores", 2);
        const int64_t G = s.size(0), W = s.size(1), V = x.size(1), K = c.tensor(a[2], "out_scores", 2).size(1);
        for (const int64_t i : {G, W, V, K})
            if (i > INT32_MAX) refuse("pka_beam_select: a size is out of range");
        const bool bf16 = x.scalar_type() == kBf16;
        if ((!bf16 && x.scalar_type() != kF32) || x.get_device() != c.device() || x.size(0) != G * W ||
            (x.numel() > 0 && V > 1 && x.stride(1) != 1))
            refuse("pka_beam_select: logits must be BFloat16 or Float rows of packed elements, one for each of scores, on "
                   "the current CUDA device");
        const int64_t stride = x.size(0) > 1 ? x.stride(0) : V;
        auto* scores = as<float>(c.packed(a[1], "scores", kF32, {G, W}));
        auto* best = as<float>(c.packed(a[2], "out_scores", kF32, {G, K}));
        auto* parents = as(c.packed(a[3], "parents", kI32, {G, K}));
        auto* tokens = as(c.packed(a[4], "tokens", kI32, {G, K}));
        const int end = (int)integer(a[5]);
        auto* finished = as<uint8_t>(c.packed_or_none(a[6], "finished", kU8, {G, W}));
        auto* ended = as<uint8_t>(c.packed_or_none(a[7], "out_finished", kU8, {G, K}));
        int32_t* err = c.word(a[8]);
        const void* logits = x.data_ptr();
        return unlocked([&] {
            return pka_beam_select(logits, bf16 ? 1 : 0, stride, scores, finished, (int)G, (int)W, (int)V, end, (int)K,
                                   best, parents, tokens, ended, err, c.stream());
        });
    });
}

// parents, ctx_lens, block_table, block_size, share_counts, free_pages, free_head, free_head_out, ctx_lens_out,
// block_table_out, copy_src, copy_dst, error_word, stream
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const Call c("pka_fork_pages", a[13]);
        const Tensor& table = c.tensor(a[2], "block_table", 2);
        const int64_t B = table.size(0), width = table.size(1), N = c.tensor(a[0], "parents", 1).size(0);
        const int64_t nb = c.tensor(a[4], "share_counts", 1).size(0), pages = c.tensor(a[5], "free_pages", 1).size(0);
        for (const int64_t i : {B, width, N, pages})
            if (i > INT32_MAX) refuse("pka_fork_pages: a size is out of range");
        const int bs = (int)integer(a[3]);
        auto* parents = as(c.packed(a[0], "parents", kI32, {N}));
        auto* ctx = as(c.packed(a[1], "ctx_lens", kI32, {B}));
        auto* bt = as(c.packed(a[2], "block_table", kI32, {B, width}));
        auto* counts = as(c.packed(a[4], "share_counts", kI32, {nb}));
        auto* free = as(c.packed(a[5], "free_pages", kI32, {pages}));
        auto* head = as(c.packed(a[6], "free_head", kI32, {1}));
        auto* out = as(c.packed(a[7], "free_head_out", kI32, {1}));
        auto* ctx_out = as(c.packed(a[8], "ctx_lens_out", kI32, {N}));
        auto* bt_out = as(c.packed(a[9], "block_table_out", kI32, {N, width}));
        auto* src = as(c.packed(a[10], "copy_src", kI32, {N}));
        auto* dst = as(c.packed(a[11], "copy_dst", kI32, {N}));
        int32_t* err = c.word(a[12]);
        return unlocked([&] {
            return pka_fork_pages(parents, (int)N, ctx, bt, (int)B, (int)width, bs, counts, nb, free, (int)pages, head,
                                  out, ctx_out, bt_out, src, dst, err, c.stream());
        });
    });
}

// caches, copy_src, copy_dst, error_word, stream
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const Call c("pka_copy_pages", a[4]);
        PyObject* caches = PySequence_Fast(a[0], "pka_copy_pages: caches must be a sequence of tensors");
        if (!caches) throw Raised();
        struct Hold {
            PyObject* o;
            ~Hold() { Py_DECREF(o); }
        } hold{caches};
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(caches);
        if (count > PKA_MAX_COPY_CACHES) refuse("pka_copy_pages: too many caches for one call");
        void* at[PKA_MAX_COPY_CACHES];
        int64_t nb = 1, page = 16;
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* o = PySequence_Fast_GET_ITEM(caches, i);
            if (!THPVariable_Check(o)) {
                PyErr_SetString(PyExc_TypeError, "pka_copy_pages: caches must be tensors");
                throw Raised();
            }
            const Tensor& t = THPVariable_Unpack(o);
            if (t.dim() < 2 || t.get_device() != c.device() || !t.is_contiguous() || t.numel() == 0)
                refuse("pka_copy_pages: caches must be packed [num_blocks, ...] tensors on the current CUDA device");
            const int64_t bytes = t.numel() / t.size(0) * (int64_t)t.element_size();
            if (i > 0 && (t.size(0) != nb || bytes != page))
                refuse("pka_copy_pages: caches must have the same number of pages, all of one size");
            nb = t.size(0);
            page = bytes;
            at[i] = t.data_ptr();
        }
        const int64_t pairs = c.tensor(a[1], "copy_src", 1).size(0);
        if (pairs > INT32_MAX) refuse("pka_copy_pages: a size is out of range");
        auto* src = as(c.packed(a[1], "copy_src", kI32, {pairs}));
        auto* dst = as(c.packed(a[2], "copy_dst", kI32, {pairs}));
        int32_t* err = c.word(a[3]);
        return unlocked(
            [&] { return pka_copy_pages(at, (int)count, nb, page, src, dst, (int)pairs, err, c.stream()); });
    });
}

// q, k_cache, v_cache, block_table, query_start_loc, seq_lens, group_starts, prefix_lens, scale, max_query_len,
// max_seq_len, out, lse, workspace, kv_scales, error_word, stream
PyObject* prefix_attn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] {
        const Call c("pka_prefix_attn_forward", a[16]);
        const Tensor &q = c.tensor(a[0], "q", 3), &cache = c.tensor(a[1], "k_cache", 4);
        const Tensor &table = c.tensor(a[3], "block_table", 2), &work = c.tensor(a[13], "workspace", 1);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), nb = cache.size(0), Hkv = cache.size(1);
        const int64_t bs = cache.size(2), B = table.size(0), width = table.size(1);
        const int64_t groups = c.tensor(a[7], "prefix_lens", 1).size(0);
        for (const int64_t x : {T, Hq, d, Hkv, bs, B, width, groups})
            if (x > INT32_MAX) refuse("pka_prefix_attn_forward: a size is out of range");
        float scales[2];
        const bool fp8 = scales_of(a[14], scales);
        const auto kind = fp8 ? kU8 : kBf16;
        const float scale = number(a[8]);
        const int most = (int)integer(a[9]), longest = (int)integer(a[10]);
        const void* qp = c.packed(a[0], "q", kBf16, {T, Hq, d});
        const void* kc = c.packed(a[1], "k_cache", kind, {nb, Hkv, bs, d});
        const void* vc = c.packed(a[2], "v_cache", kind, {nb, Hkv, bs, d});
        auto* bt = as(c.packed(a[3], "block_table", kI32, {B, width}));
        auto* qsl = as(c.packed(a[4], "query_start_loc", kI32, {B + 1}));
        auto* seq = as(c.packed(a[5], "seq_lens", kI32, {B}));
        auto* starts = as(c.packed(a[6], "group_starts", kI32, {groups + 1}));
        auto* prefix = as(c.packed(a[7], "prefix_lens", kI32, {groups}));
        void* out = c.packed(a[11], "out", kBf16, {T, Hq, d});
        auto* lse = as<float>(c.packed_or_none(a[12], "lse", kF32, {T, Hq}));
        void* scratch = c.packed(a[13], "workspace", kU8, {work.size(0)});
        const size_t size = (size_t)work.size(0);
        int32_t* err = c.word(a[15]);
        return unlocked([&] {
            if (fp8)
                return pka_prefix_attn_forward_fp8(qp, kc, vc, bt, (int)width, qsl, seq, (int)B, starts, prefix,
                                                   (int)groups, (int)T, (int)Hq, (int)Hkv, (int)d, nb, (int)bs, scale,
                                                   scales[0], scales[1], most, longest, out, lse, scratch, size, err,
                                                   c.stream());
            return pka_prefix_attn_forward(qp, kc, vc, bt, (int)width, qsl, seq, (int)B, starts, prefix, (int)groups,
                                           (int)T, (int)Hq, (int)Hkv, (int)d, nb, (int)bs, scale, most, longest, out,
                                           lse, scratch, size, err, c.stream());
        });
    });
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<step_tables>("step_tables"),
    method<qk_rope_cache_write>("qk_rope_cache_write"),
    method<page_bounds>("page_bounds"),
    method<select_pages>("select_pages"),
    method<sparse_attn_forward>("sparse_attn_forward"),
    method<beam_select>("beam_select"),
    method<fork_pages>("fork_pages"),
    method<copy_pages>("copy_pages"),
    method<prefix_attn_forward>("prefix_attn_forward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pka_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pka_torch() { return PyModule_Create(&module); }
