// calls.cpp -- the Python side of the calls around beams, trees and rotary positions: tensors checked and handed to the C ABI.
//
// These calls stand in serving steps of a few microseconds, and looking a tensor's type, shape, device and address up from Python takes
// a third of one.  Each function here takes the binding's arguments in their order, the stream and the cache's struct as addresses,
// and returns the call's status, or None where a tensor is not what the call wants: the binding then says which.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "kvq8attn.h"

namespace {

constexpr auto kI32 = at::kInt, kI64 = at::kLong, kF32 = at::kFloat;

// The arguments one after another; ok turns false at the first that does not fit.
struct Args {
    PyObject* const* at;
    int64_t device;
    bool ok = true;

    const at::Tensor* tensor() {
        PyObject* o = *at++;
        if (!THPVariable_Check(o)) return ok = false, nullptr;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.get_device() != device || device < 0) return ok = false, nullptr;
        return &t;
    }
    // the address of a contiguous tensor of this type and shape
    template <typename T>
    T* whole(at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor();
        if (!t || t->scalar_type() != type || !t->sizes().equals(at::IntArrayRef(shape)) || !t->is_contiguous()) return ok = false, nullptr;
        return static_cast<T*>(t->data_ptr());
    }
    // the same, or null for None
    template <typename T>
    T* whole_or_none(at::ScalarType type, std::initializer_list<int64_t> shape) {
        if (*at == Py_None) return ++at, nullptr;
        return whole<T>(type, shape);
    }
    int64_t number() {
        const long long v = PyLong_AsLongLong(*at++);
        if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
        return v;
    }
    template <typename T>
    T* address() { return reinterpret_cast<T*>(number()); }
    struct Space {
        void* at = nullptr;
        size_t bytes = 0;
    };
    Space space() {
        const at::Tensor* t = tensor();
        if (!t || !t->is_contiguous()) return ok = false, Space{};
        return {t->data_ptr(), (size_t)t->nbytes()};
    }
    // tokens of `heads` contiguous rows of `dim` values; their number and the stride between them
    void* tokens(int& dtype, int64_t& n, int64_t heads, int64_t dim, int64_t& stride, int64_t* found_heads = nullptr) {
        const at::Tensor* t = tensor();
        if (!t || t->dim() != 3) return ok = false, nullptr;
        const int d = dtype_of(*t);
        if (found_heads) *found_heads = heads = t->size(1);
        if (d < 0 || (dtype >= 0 && d != dtype) || (n >= 0 && t->size(0) != n) || t->size(1) != heads || t->size(2) != dim ||
            t->stride(2) != 1 || (t->stride(1) != dim && heads > 1))
            return ok = false, nullptr;
        dtype = d;
        n = t->size(0);
        stride = n > 1 ? t->stride(0) : heads * dim;
        return t->data_ptr();
    }
    static int dtype_of(const at::Tensor& t) {
        return t.scalar_type() == at::kFloat ? KVQ8_F32 : t.scalar_type() == at::kHalf ? KVQ8_F16 : t.scalar_type() == at::kBFloat16 ? KVQ8_BF16 : -1;
    }
};

int64_t length(PyObject* o, int dim = 0) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.dim() > dim ? t.size(dim) : -1;
}
int64_t device_of(PyObject* o) { return THPVariable_Check(o) ? THPVariable_Unpack(o).get_device() : -1; }

// A status, or None where an argument did not fit or a size does not fit the C ABI's ints.
template <typename F>
PyObject* done(const Args& a, std::initializer_list<int64_t> sizes, F call) {
    if (!a.ok) Py_RETURN_NONE;
    for (int64_t n : sizes)
        if (n < -0x7fffffffLL || n > 0x7fffffffLL) Py_RETURN_NONE;
    int status;
    Py_BEGIN_ALLOW_THREADS  // a launch may wait for room in the stream's queue
    status = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

// torch raises C++ exceptions for tensors that have no strides or no memory: such a tensor is none that a call takes.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(args, n);
    } catch (const std::exception&) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define EXPECT(n_args)                                                                \
    if (n != (n_args)) return PyErr_Format(PyExc_TypeError, "%d arguments are wanted", (int)(n_args))

// logits, row_starts, n_out, scores, weights, ended, parents, tokens, totals, workspace, stream
PyObject* select(PyObject* const* args, Py_ssize_t n) {
    EXPECT(11);
    Args a{args, device_of(args[0])};
    const at::Tensor* x = a.tensor();
    if (!x || x->dim() != 2 || Args::dtype_of(*x) < 0 || (x->stride(1) != 1 && x->size(1) > 1)) Py_RETURN_NONE;
    const int64_t rows = x->size(0), vocab = x->size(1), seqs = length(args[1]) - 1;
    const int32_t* starts = a.whole<int32_t>(kI32, {seqs + 1});
    const int64_t out = a.number();
    const float* scores = a.whole_or_none<float>(kF32, {rows});
    const float* weights = a.whole_or_none<float>(kF32, {rows});
    const int32_t* ended = a.whole_or_none<int32_t>(kI32, {rows});
    int32_t* parents = a.whole<int32_t>(kI32, {seqs, out});
    int32_t* tokens = a.whole<int32_t>(kI32, {seqs, out});
    float* totals = a.whole<float>(kF32, {seqs, out});
    const Args::Space space = a.space();
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {rows, vocab, seqs, out}, [&] {
        return beam_select(x->data_ptr(), Args::dtype_of(*x), rows > 1 ? x->stride(0) : vocab, (int)rows, (int)vocab, starts, (int)seqs,
                           scores, weights, ended, (int)out, parents, tokens, totals, space.at, space.bytes, stream);
    });
}

// parents, state_of, counts, state_of_out, status, n_seqs, workspace, stream
PyObject* counts_fork(PyObject* const* args, Py_ssize_t n) {
    EXPECT(8);
    Args a{args, device_of(args[2])};
    const int64_t kids = length(args[0]), states = length(args[2]), vocab = length(args[2], 1);
    const int64_t seqs = args[1] == Py_None ? PyLong_AsLongLong(args[5]) : length(args[1]);
    const int32_t* parents = a.whole<int32_t>(kI32, {kids});
    const int32_t* state_of = a.whole_or_none<int32_t>(kI32, {seqs});
    uint32_t* counts = a.whole<uint32_t>(kI32, {states, vocab});
    int32_t* out = a.whole<int32_t>(kI32, {kids});
    int32_t* status = a.whole<int32_t>(kI32, {1});
    a.number();
    const Args::Space space = a.space();
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {kids, seqs, states, vocab}, [&] {
        return token_counts_fork(parents, (int)kids, state_of, (int)seqs, counts, (int)states, (int)vocab, out, status, space.at, space.bytes, stream);
    });
}

// parents, lens, held, page_size, page_table, shares, free_ring, ring_state, page_table_out, lens_out, held_out, shares_out, ring_out,
// copy_src, copy_dst, copy_rows, status, workspace, stream
PyObject* paged_fork(PyObject* const* args, Py_ssize_t n) {
    EXPECT(19);
    Args a{args, device_of(args[4])};
    const int64_t kids = length(args[0]), seqs = length(args[4]), wide = length(args[4], 1), pages = length(args[6]);
    const int32_t* parents = a.whole<int32_t>(kI32, {kids});
    const int32_t* lens = a.whole<int32_t>(kI32, {seqs});
    const int32_t* held = a.whole<int32_t>(kI32, {seqs});
    const int64_t page = a.number();
    const int32_t* table = a.whole<int32_t>(kI32, {seqs, wide});
    const int32_t* shares = a.whole<int32_t>(kI32, {pages});
    int32_t* ring = a.whole<int32_t>(kI32, {pages});
    const int32_t* state = a.whole<int32_t>(kI32, {2});
    int32_t* table_out = a.whole<int32_t>(kI32, {kids, wide});
    int32_t* lens_out = a.whole<int32_t>(kI32, {kids});
    int32_t* held_out = a.whole<int32_t>(kI32, {kids});
    int32_t* shares_out = a.whole<int32_t>(kI32, {pages});
    int32_t* state_out = a.whole<int32_t>(kI32, {2});
    int32_t* src = a.whole<int32_t>(kI32, {kids});
    int32_t* dst = a.whole<int32_t>(kI32, {kids});
    int32_t* rows = a.whole<int32_t>(kI32, {kids});
    int32_t* status = a.whole<int32_t>(kI32, {1});
    const Args::Space space = a.space();
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {kids, seqs, wide, pages, page}, [&] {
        return kvq8_paged_fork(parents, (int)kids, lens, held, (int)seqs, (int)page, table, (int)wide, shares, ring, (int)pages, state, table_out,
                               lens_out, held_out, shares_out, state_out, src, dst, rows, status, space.at, space.bytes, stream);
    });
}

// cache, device, src_pages, dst_pages, rows, stream
PyObject* paged_copy(PyObject* const* args, Py_ssize_t n) {
    EXPECT(6);
    Args a{args, -1};
    const kvq8_paged_cache* cache = a.address<const kvq8_paged_cache>();
    a.device = a.number();
    const int64_t entries = length(args[2]);
    const int32_t* src = a.whole<int32_t>(kI32, {entries});
    const int32_t* dst = a.whole<int32_t>(kI32, {entries});
    const int32_t* rows = a.whole_or_none<int32_t>(kI32, {entries});
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {entries}, [&] { return kvq8_paged_copy(cache, src, dst, rows, (int)entries, stream); });
}

// cache, device, page_table, lens, row_starts, kept, lens_out, stream
PyObject* paged_compact(PyObject* const* args, Py_ssize_t n) {
    EXPECT(8);
    Args a{args, -1};
    const kvq8_paged_cache* cache = a.address<const kvq8_paged_cache>();
    a.device = a.number();
    const int64_t seqs = length(args[2]), wide = length(args[2], 1);
    const int32_t* table = a.whole<int32_t>(kI32, {seqs, wide});
    const int32_t* lens = a.whole<int32_t>(kI32, {seqs});
    const int32_t* starts = a.whole<int32_t>(kI32, {seqs + 1});
    const uint64_t* kept = a.whole<uint64_t>(kI64, {seqs});
    int32_t* lens_out = a.whole_or_none<int32_t>(kI32, {seqs});
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {seqs, wide}, [&] { return kvq8_paged_compact(cache, table, (int)wide, lens, starts, (int)seqs, kept, lens_out, stream); });
}

// cache, device, q, k, v, slots, positions, turns, axis_of, pairs, q_out, stream
PyObject* paged_append_rope(PyObject* const* args, Py_ssize_t n) {
    EXPECT(12);
    Args a{args, -1};
    const kvq8_paged_cache* cache = a.address<const kvq8_paged_cache>();
    a.device = a.number();
    if (!a.ok) Py_RETURN_NONE;
    int dtype = -1;
    int64_t tok = -1, heads = 0, q_stride = 0, k_stride = 0, v_stride = 0, out_stride = 0;
    const int64_t dim = cache->head_dim, kv_heads = cache->n_kv_heads;
    const void* q = a.tokens(dtype, tok, 0, dim, q_stride, &heads);
    const void* k = a.tokens(dtype, tok, kv_heads, dim, k_stride);
    const void* v = a.tokens(dtype, tok, kv_heads, dim, v_stride);
    const int64_t* slots = a.whole<int64_t>(kI64, {tok});
    const int64_t axes = length(args[6], 1) < 0 ? 1 : length(args[6]), half = length(args[7]);
    const int32_t* positions = length(args[6], 1) < 0 ? a.whole<int32_t>(kI32, {tok}) : a.whole<int32_t>(kI32, {axes, tok});
    const uint64_t* turns = a.whole<uint64_t>(kI64, {half});
    const int32_t* axis_of = a.whole_or_none<int32_t>(kI32, {half});
    const int64_t pairs = a.number();
    void* out = a.tokens(dtype, tok, heads, dim, out_stride);
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {tok, heads, axes, 2 * half}, [&] {
        return kvq8_paged_append_rope(q, k, v, dtype, (int)tok, (int)heads, q_stride, k_stride, v_stride, positions, (int)axes, turns, axis_of,
                                      (int)(2 * half), pairs != 0, cache, slots, out, out_stride, stream);
    });
}

// cache, device, slots, k, v, stream
PyObject* paged_read(PyObject* const* args, Py_ssize_t n) {
    EXPECT(6);
    Args a{args, -1};
    const kvq8_paged_cache* cache = a.address<const kvq8_paged_cache>();
    a.device = a.number();
    if (!a.ok) Py_RETURN_NONE;
    const int64_t tok = length(args[2]), heads = cache->n_kv_heads, dim = cache->head_dim;
    const int64_t* slots = a.whole<int64_t>(kI64, {tok});
    void* at[2] = {};
    int64_t strides[2][2] = {};
    int dtype = -1;
    for (int z = 0; z < 2 && a.ok; ++z) {
        const at::Tensor* t = a.tensor();
        if (!t || !t->sizes().equals({tok, heads, dim}) || t->stride(2) != 1 || Args::dtype_of(*t) < 0 || (z && Args::dtype_of(*t) != dtype)) Py_RETURN_NONE;
        dtype = Args::dtype_of(*t);
        strides[z][0] = tok > 1 ? t->stride(0) : dim;
        strides[z][1] = heads > 1 ? t->stride(1) : dim;
        at[z] = t->data_ptr();
    }
    kvq8_stream_t stream = a.address<CUstream_st>();
    return done(a, {tok}, [&] { return kvq8_paged_read(cache, slots, (int)tok, dtype, at[0], at[1], strides[0], strides[1], stream); });
}

#define FUNCTION(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<name>)), METH_FASTCALL, nullptr }
PyMethodDef kFunctions[] = {FUNCTION(select),     FUNCTION(counts_fork),   FUNCTION(paged_fork),
                            FUNCTION(paged_copy), FUNCTION(paged_compact), FUNCTION(paged_append_rope),
                            FUNCTION(paged_read),
                            {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kFunctions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
