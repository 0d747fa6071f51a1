// calls.cpp -- the Python binding of paged_rotary, paged_append_rotary,
// paged_decode_shared and paged_merge_states: argument checks, result tensors
// and the call of the C entry point of the same name (include/pagedkv.h), in
// one step of C++.
//
// These calls are made once per layer and step, on GPU work of a few
// microseconds, so what a call costs on the host is what a small batch costs:
// the same checks in Python and the conversion of 20 to 35 arguments by ctypes
// took 17 to 30 us a call on a GB300's host, of which 5 to 16 remain.  binding.py holds
// the signatures and documentation and passes every argument by position.  The
// C entry points are called through the addresses that it hands over when it
// loads the library, so that a switch to another build of it is followed.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <stdexcept>
#include <string>
#include <vector>

#include "pagedkv.h"

namespace {

PyObject *g_error = nullptr, *g_check = nullptr;  // PagedKVError; raises for a non-zero status
decltype(&paged_rotary) g_rotary = nullptr;
decltype(&paged_append_rotary) g_append_rotary = nullptr;
decltype(&paged_decode_shared) g_decode_shared = nullptr;
decltype(&paged_merge_states) g_merge_states = nullptr;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python error is set

using Tensor = at::Tensor;

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
void *address(const Tensor &t) { return t.data_ptr(); }
void *address(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int32_t int32(PyObject *o) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused("an argument does not fit 32 bits");
    return static_cast<int32_t>(v);
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}
// None or an address.
const float *pointer(PyObject *o) {
    return o == Py_None ? nullptr : reinterpret_cast<const float *>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o)));
}

int dtype_code(const Tensor &t) {
    if (t.scalar_type() == at::kHalf) return PKV_F16;
    if (t.scalar_type() == at::kBFloat16) return PKV_BF16;
    return -1;
}

// The current device, where every tensor of a call has to be (the library
// launches there).
struct Device {
    int index;
    explicit Device(const Tensor &first) : index(first.is_cuda() ? c10::cuda::current_device() : -2) {}
    void holds(const Tensor &t) const {
        if ((t.is_cuda() ? t.get_device() : -1) != index)
            throw Refused("tensor arguments must live on the current CUDA device");
    }
    void holds(const Tensor *t) const {
        if (t) holds(*t);
    }
    void *stream(PyObject *given) const {
        if (given != Py_None) {
            void *st = reinterpret_cast<void *>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(given)));
            if (PyErr_Occurred()) throw Raised();
            return st;
        }
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    }
};

int layout_code(PyObject *o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "NHD") == 0) return PKV_NHD;
        if (PyUnicode_CompareWithASCIIString(o, "HND") == 0) return PKV_HND;
    } else if (PyLong_Check(o)) {
        const long v = PyLong_AsLong(o);
        if (v == PKV_NHD || v == PKV_HND) return static_cast<int>(v);
        PyErr_Clear();
    }
    throw Refused("kv_layout must be NHD or HND");
}

// Dimensions `from` and on are contiguous.
bool rows_contiguous(const Tensor &t, int64_t from) {
    int64_t n = 1;
    for (int64_t i = t.dim() - 1; i >= from; --i) {
        if (t.size(i) != 1 && t.stride(i) != n) return t.numel() == 0;
        n *= t.size(i);
    }
    return true;
}

// A [pages, 2, ..] tensor or a (K, V) tuple of [pages, ..] tensors.
struct Cache {
    const Tensor *base;
    char *k, *v;
    int64_t stride, pages, heads, page_size, head_dim;
    Cache(PyObject *o, int layout) {
        int64_t at;
        if (PyTuple_Check(o) || PyList_Check(o)) {
            if (PySequence_Fast_GET_SIZE(o) != 2) throw Refused("a cache is one tensor or a (K, V) tuple");
            base = &tensor(PySequence_Fast_GET_ITEM(o, 0), "the K cache");
            const Tensor &other = tensor(PySequence_Fast_GET_ITEM(o, 1), "the V cache");
            if (base->dim() != 4) throw Refused("K and V caches are 4-D");
            if (other.sizes() != base->sizes() || other.stride(0) != base->stride(0))
                throw Refused("K and V caches must have the same shape and page stride");
            if (other.scalar_type() != base->scalar_type() || other.device() != base->device())
                throw Refused("K and V caches hold the same type on the same device");
            if (!rows_contiguous(*base, 1) || !rows_contiguous(other, 1)) throw Refused("each page must be contiguous");
            v = static_cast<char *>(other.data_ptr());
            at = 1;
        } else {
            base = &tensor(o, "the cache");
            if (base->dim() != 5 || base->size(1) != 2) throw Refused("a single kv_cache tensor must be [pages, 2, ...]");
            if (!rows_contiguous(*base, 1)) throw Refused("each page must be contiguous");
            v = static_cast<char *>(base->data_ptr()) + base->stride(1) * base->element_size();
            at = 2;
        }
        if (!base->is_cuda()) throw Refused("tensor arguments must live on a CUDA device");
        k = static_cast<char *>(base->data_ptr());
        stride = base->stride(0);
        pages = base->size(0);
        heads = base->size(at + (layout == PKV_HND ? 0 : 1));
        page_size = base->size(at + (layout == PKV_HND ? 1 : 0));
        head_dim = base->size(at + 2);
    }
};

// [tokens, heads, head_dim] whose heads are contiguous.
struct Rows {
    int64_t n, heads, dim, stride;
    Rows(const Tensor &t, const char *name) {
        if (t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
            throw Refused(std::string(name) + " must be [tokens, heads, head_dim] with contiguous heads");
        n = t.size(0);
        heads = t.size(1);
        dim = t.size(2);
        stride = n > 1 ? t.stride(0) : heads * dim;  // (of one token any stride will do)
    }
};

const int32_t *int32_of(const Tensor &t, int64_t n, const char *name) {
    if (t.scalar_type() != at::kInt || t.numel() < n || !t.is_contiguous())
        throw Refused(std::string(name) + " must be contiguous int32 with >= " + std::to_string(n) + " entries");
    return static_cast<const int32_t *>(t.data_ptr());
}

// `given`, checked, or a new tensor.
Tensor result(PyObject *given, const char *name, at::IntArrayRef shape, const Tensor &like, at::ScalarType type) {
    if (given == Py_None) return at::empty(shape, like.options().dtype(type));
    const Tensor &t = tensor(given, name);
    if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous())
        throw Refused(std::string(name) + " must be a contiguous tensor of its result's shape and dtype");
    return t;
}

void check(int status) {
    if (status == PKV_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "i", status);
    if (r) {
        Py_DECREF(r);
        PyErr_Format(g_error, "libpagedkv status %d", status);
    }
    throw Raised();
}

template <typename F>
int unlocked(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS status = f();
    Py_END_ALLOW_THREADS return status;
}

template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Raised &) {
    } catch (const Refused &e) {
        PyErr_SetString(g_error, e.what());
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// A reference of this call's own.
struct Owned {
    PyObject *o;
    explicit Owned(PyObject *p) : o(p) {}
    Owned(const Owned &) = delete;
    Owned &operator=(const Owned &) = delete;
    ~Owned() { Py_XDECREF(o); }
};

void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) throw Refused("wrong number of arguments");
}

// What the two rotary calls share.
struct Rotary {
    const Tensor &query, &key, &frequencies;
    const Tensor *qw, *kw;
    Rows q, k;
    int dtype;
    Tensor query_out;
    Rotary(PyObject *query_, PyObject *key_, PyObject *frequencies_, PyObject *qw_, PyObject *kw_, PyObject *out)
        : query(tensor(query_, "query")),
          key(tensor(key_, "key")),
          frequencies(tensor(frequencies_, "frequencies")),
          qw(optional(qw_, "query_weight")),
          kw(optional(kw_, "key_weight")),
          q(query, "query"),
          k(key, "key"),
          dtype(dtype_code(query)) {
        if (k.n != q.n || k.dim != q.dim) throw Refused("query and key have the same tokens and head_dim");
        if (dtype < 0 || key.scalar_type() != query.scalar_type())
            throw Refused("query and key are both fp16 or both bf16");
        if (frequencies.scalar_type() != at::kDouble || frequencies.dim() != 1 || !frequencies.is_contiguous())
            throw Refused("frequencies must be contiguous float64 [rotary_dim // 2]");
        for (const Tensor *w : {qw, kw})
            if (w && (w->scalar_type() != query.scalar_type() || w->numel() != q.dim || !w->is_contiguous()))
                throw Refused("norm weights must be contiguous [head_dim] of the query's type");
        query_out = result(out, "query_out", query.sizes(), query, query.scalar_type());
    }
};

// query, key, positions, frequencies, rotary_start, interleaved, magnitude,
// query_weight, key_weight, eps, query_out, key_out, stream
PyObject *call_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        arguments(n, 13);
        const Rotary r(a[0], a[1], a[3], a[7], a[8], a[10]);
        const Tensor &positions = tensor(a[2], "positions");
        const int32_t *at = int32_of(positions, r.q.n, "positions");
        const Tensor key_out = result(a[11], "key_out", r.key.sizes(), r.key, r.key.scalar_type());
        const Device dev(r.query);
        for (const Tensor *t : {&r.query, &r.key, &positions, &r.frequencies, r.qw, r.kw, &r.query_out, &key_out}) dev.holds(t);
        const int32_t start = int32(a[4]);
        const bool paired = truth(a[5]);
        const float magnitude = static_cast<float>(number(a[6])), eps = static_cast<float>(number(a[9]));
        void *st = dev.stream(a[12]);
        check(unlocked([&] {
            return g_rotary(address(r.query), address(r.key), r.q.stride, r.k.stride, r.q.n, at,
                            static_cast<const double *>(address(r.frequencies)), static_cast<int32_t>(2 * r.frequencies.size(0)),
                            start, paired, magnitude, address(r.qw), address(r.kw), eps, static_cast<int32_t>(r.q.heads),
                            static_cast<int32_t>(r.k.heads), static_cast<int32_t>(r.q.dim), r.dtype, address(r.query_out),
                            address(key_out), st);
        }));
        PyObject *q = THPVariable_Wrap(r.query_out), *k = THPVariable_Wrap(key_out);
        PyObject *both = q && k ? PyTuple_Pack(2, q, k) : nullptr;
        Py_XDECREF(q);
        Py_XDECREF(k);
        return both;
    });
}

// query, key, value, batch_indices, positions, paged_kv_cache, kv_indices,
// kv_indptr, kv_last_page_len, frequencies, kv_layout, rotary_start,
// interleaved, magnitude, query_weight, key_weight, eps, rotary_positions,
// query_out, err_word, stream
PyObject *call_append_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        arguments(n, 21);
        const int layout = layout_code(a[10]);
        const Cache c(a[5], layout);
        const Rotary r(a[0], a[1], a[9], a[14], a[15], a[18]);
        const Tensor &value = tensor(a[2], "value");
        const Rows v(value, "value");
        if (r.k.heads != c.heads || r.q.dim != c.head_dim || v.heads != c.heads || v.dim != c.head_dim || v.n != r.q.n)
            throw Refused("key/value must both be [tokens, heads, head_dim] of the cache, query heads as wide");
        if (c.base->scalar_type() != r.query.scalar_type() || value.scalar_type() != r.query.scalar_type())
            throw Refused("query, key, value and the cache hold the same 16-bit type");
        const Tensor &requests = tensor(a[3], "batch_indices"), &positions = tensor(a[4], "positions");
        const Tensor &indices = tensor(a[6], "kv_indices"), &indptr = tensor(a[7], "kv_indptr");
        const Tensor &last = tensor(a[8], "kv_last_page_len");
        const Tensor *turn = optional(a[17], "rotary_positions"), *err = optional(a[19], "err_word");
        const int32_t *request = int32_of(requests, r.q.n, "batch_indices"), *at = int32_of(positions, r.q.n, "positions");
        const int32_t *rot = turn ? int32_of(*turn, r.q.n, "rotary_positions") : nullptr;
        const int32_t *page = int32_of(indices, 0, "kv_indices"), *first = int32_of(indptr, 0, "kv_indptr");
        const int32_t *end = int32_of(last, 0, "kv_last_page_len");
        if (last.dim() != 1 || indptr.numel() != last.size(0) + 1)
            throw Refused("kv_indptr must have one entry more than kv_last_page_len");
        const Device dev(r.query);
        for (const Tensor *t : {&r.query, &r.key, &value, c.base, &requests, &positions, turn, &indices, &indptr, &last,
                                &r.frequencies, r.qw, r.kw, &r.query_out, err})
            dev.holds(t);
        const int32_t start = int32(a[11]);
        const bool paired = truth(a[12]);
        const float magnitude = static_cast<float>(number(a[13])), eps = static_cast<float>(number(a[16]));
        void *st = dev.stream(a[20]);
        check(unlocked([&] {
            return g_append_rotary(address(r.query), address(r.key), address(value), r.q.stride, r.k.stride, v.stride, r.q.n,
                                   request, at, rot, c.k, c.v, c.stride, c.pages, page, first, end,
                                   static_cast<int32_t>(last.size(0)), static_cast<const double *>(address(r.frequencies)),
                                   static_cast<int32_t>(2 * r.frequencies.size(0)), start, paired, magnitude, address(r.qw),
                                   address(r.kw), eps, static_cast<int32_t>(r.q.heads), static_cast<int32_t>(c.heads),
                                   static_cast<int32_t>(c.head_dim), static_cast<int32_t>(c.page_size), layout, r.dtype,
                                   address(r.query_out), static_cast<int32_t *>(address(err)), st);
        }));
        return THPVariable_Wrap(r.query_out);
    });
}

// The row stride of a table of n rows of pages, for sequences of up to
// `longest` tokens.
int32_t page_table(const Tensor &t, int64_t n, int64_t longest, int64_t page_size) {
    if (t.dim() != 2 || t.scalar_type() != at::kInt || t.size(0) < n || (t.size(1) > 1 && t.stride(1) != 1))
        throw Refused("page tables must be int32 [rows, pages] with unit column stride");
    if (n && t.size(1) * page_size < longest)
        throw Refused("a page table has fewer columns than its longest sequence needs");
    const int64_t s = t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
    if (s < 0 || s > INT32_MAX) throw Refused("a page table's rows are too far apart");
    return static_cast<int32_t>(s);
}

// query, kv_cache, workspace, prefix_tables, prefix_lens, group_indptr,
// max_prefix_len, block_tables, seq_lens, max_seq_len, scale 1, scale 2, their
// device addresses or None, sinks, kv_layout, q_len_per_req, out, lse,
// err_word, stream
PyObject *call_decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        arguments(n, 21);
        const int layout = layout_code(a[15]);
        const Cache c(a[1], layout);
        const Tensor &query = tensor(a[0], "query");
        const int dtype = dtype_code(query);
        if (query.dim() != 3 || query.size(2) != c.head_dim || !query.is_contiguous())
            throw Refused("query must be contiguous [rows, num_qo_heads, head_dim]");
        if (dtype < 0 || c.base->scalar_type() != query.scalar_type())
            throw Refused("query and cache are both fp16 or both bf16");
        const Tensor &lens = tensor(a[8], "seq_lens"), &prefix = tensor(a[4], "prefix_lens");
        const Tensor &indptr = tensor(a[5], "group_indptr"), &workspace = tensor(a[2], "workspace");
        const Tensor &prefix_tables = tensor(a[3], "prefix_tables"), &tables = tensor(a[7], "block_tables");
        const Tensor *sinks = optional(a[14], "sinks"), *lse = optional(a[18], "lse"), *err = optional(a[19], "err_word");
        if (lens.dim() != 1 || lens.element_size() != 4 || !lens.is_contiguous())
            throw Refused("seq_lens must be a contiguous 1-D tensor of 32-bit lengths");
        const int64_t B = lens.size(0);
        const int32_t Q = int32(a[16]), max_prefix = int32(a[6]), max_len = int32(a[9]);
        if (query.size(0) < B * Q) throw Refused("query has fewer rows than the requests need");
        if (prefix.scalar_type() != at::kInt || prefix.dim() != 1 || !prefix.is_contiguous() ||
            indptr.scalar_type() != at::kInt || indptr.dim() != 1 || indptr.size(0) != prefix.size(0) + 1 ||
            !indptr.is_contiguous())
            throw Refused("prefix_lens [groups] and group_indptr [groups + 1] must be contiguous int32");
        const int64_t G = prefix.size(0);
        const int32_t prefix_stride = page_table(prefix_tables, G, max_prefix, c.page_size);
        const int32_t table_stride = page_table(tables, B, max_len, c.page_size);
        if (!workspace.is_contiguous()) throw Refused("workspace must be contiguous");
        if (lse && (lse->scalar_type() != at::kFloat || lse->sizes() != query.sizes().slice(0, 2) || !lse->is_contiguous()))
            throw Refused("lse must be a contiguous float32 [rows, num_qo_heads] tensor");
        if (sinks && (sinks->scalar_type() != at::kFloat || sinks->numel() != query.size(1) || !sinks->is_contiguous()))
            throw Refused("sinks must be contiguous float32 [num_qo_heads]");
        const Tensor out = result(a[17], "out", query.sizes(), query, query.scalar_type());
        const Device dev(query);
        for (const Tensor *t : {&query, c.base, &workspace, &prefix_tables, &prefix, &indptr, &tables, &lens, sinks, &out, lse, err})
            dev.holds(t);
        const float s1 = static_cast<float>(number(a[10])), s2 = static_cast<float>(number(a[11]));
        const float *s1_dev = pointer(a[12]), *s2_dev = pointer(a[13]);
        void *st = dev.stream(a[20]);
        check(unlocked([&] {
            return g_decode_shared(address(query), c.k, c.v, c.stride, c.pages, address(workspace), workspace.nbytes(),
                                   static_cast<const int32_t *>(address(prefix_tables)), prefix_stride,
                                   static_cast<const int32_t *>(address(prefix)), static_cast<const int32_t *>(address(indptr)),
                                   static_cast<int32_t>(G), max_prefix, static_cast<const int32_t *>(address(tables)),
                                   table_stride, static_cast<const uint32_t *>(address(lens)), static_cast<int32_t>(B), max_len,
                                   s1, s2, s1_dev, s2_dev, static_cast<const float *>(address(sinks)), Q,
                                   static_cast<int32_t>(query.size(1)), static_cast<int32_t>(c.heads),
                                   static_cast<int32_t>(c.head_dim), static_cast<int32_t>(c.page_size), layout, dtype,
                                   address(out), static_cast<float *>(address(lse)), static_cast<int32_t *>(address(err)), st);
        }));
        return THPVariable_Wrap(out);
    });
}

// states, out, lse, stream
PyObject *call_merge_states(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        arguments(n, 4);
        const Owned seq(PySequence_Fast(a[0], "states must be a sequence"));
        if (!seq.o) throw Raised();
        // (references of this call's own: the lists are the caller's, and other
        // threads run while the kernels are launched)
        std::vector<Tensor> outs, lses;
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq.o); ++i) {
            const Owned pair(PySequence_Fast(PySequence_Fast_GET_ITEM(seq.o, i), "a state is an (out, lse) pair"));
            PyObject *p = pair.o;
            if (!p) throw Raised();
            if (PySequence_Fast_GET_SIZE(p) != 2) throw Refused("a state is an (out, lse) pair");
            outs.push_back(tensor(PySequence_Fast_GET_ITEM(p, 0), "a state's output"));
            lses.push_back(tensor(PySequence_Fast_GET_ITEM(p, 1), "a state's log-sum-exp"));
        }
        const size_t parts = outs.size();
        if (parts == 0) throw Refused("no states to merge");
        const Tensor &first = outs[0];
        const int dtype = dtype_code(first);
        if (first.dim() != 3 || dtype < 0) throw Refused("a state's output is [rows, heads, head_dim] in fp16 or bf16");
        const auto rows = first.sizes().slice(0, 2);
        const Tensor out = result(a[1], "out", first.sizes(), first, first.scalar_type());
        const Tensor lse = result(a[2], "lse", rows, first, at::kFloat);
        const Device dev(first);
        dev.holds(out);
        dev.holds(lse);
        std::vector<const void *> o;
        std::vector<const float *> l;
        for (size_t i = 0; i < parts; ++i) {
            if (outs[i].sizes() != first.sizes() || outs[i].scalar_type() != first.scalar_type() || !outs[i].is_contiguous())
                throw Refused("outputs must be contiguous tensors of the same shape and type");
            if (lses[i].sizes() != rows || lses[i].scalar_type() != at::kFloat || !lses[i].is_contiguous())
                throw Refused("log-sum-exps must be contiguous float32 [rows, heads]");
            dev.holds(outs[i]);
            dev.holds(lses[i]);
            o.push_back(outs[i].data_ptr());
            l.push_back(static_cast<const float *>(lses[i].data_ptr()));
        }
        void *st = dev.stream(a[3]);
        check(unlocked([&] {
            return g_merge_states(o.data(), l.data(), static_cast<int32_t>(std::min<size_t>(parts, INT32_MAX)),
                                  first.size(0) * first.size(1), static_cast<int32_t>(first.size(2)), dtype, address(out),
                                  static_cast<float *>(address(lse)), st);
        }));
        PyObject *x = THPVariable_Wrap(out), *y = THPVariable_Wrap(lse);
        PyObject *both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return both;
    });
}

// use(error, check, addresses of the four entry points): before any call, and
// again for another build of the library.
PyObject *call_use(PyObject *, PyObject *args) {
    PyObject *error, *check_status;
    unsigned long long p[4];
    if (!PyArg_ParseTuple(args, "OOKKKK", &error, &check_status, &p[0], &p[1], &p[2], &p[3])) return nullptr;
    Py_INCREF(error);
    Py_INCREF(check_status);
    Py_XDECREF(g_error);
    Py_XDECREF(g_check);
    g_error = error;
    g_check = check_status;
    g_rotary = reinterpret_cast<decltype(g_rotary)>(static_cast<uintptr_t>(p[0]));
    g_append_rotary = reinterpret_cast<decltype(g_append_rotary)>(static_cast<uintptr_t>(p[1]));
    g_decode_shared = reinterpret_cast<decltype(g_decode_shared)>(static_cast<uintptr_t>(p[2]));
    g_merge_states = reinterpret_cast<decltype(g_merge_states)>(static_cast<uintptr_t>(p[3]));
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"use", call_use, METH_VARARGS, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_rotary)), METH_FASTCALL, nullptr},
    {"append_rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_append_rotary)), METH_FASTCALL, nullptr},
    {"decode_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_decode_shared)), METH_FASTCALL, nullptr},
    {"merge_states", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_merge_states)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Tensors are taken apart by torch's own headers, whose layouts another version
// need not share: imported under the torch that it was compiled for, or not at all.
PyMODINIT_FUNC PyInit__calls(void) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    PyObject *text = version ? PyObject_Str(version) : nullptr;
    const char *now = text ? PyUnicode_AsUTF8(text) : nullptr;
    PyObject *made = nullptr;
    if (now && std::string(now) == PKV_TORCH_VERSION) made = PyModule_Create(&module);
    else if (now) PyErr_Format(PyExc_ImportError, "built for torch %s, this is %s", PKV_TORCH_VERSION, now);
    Py_XDECREF(text);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    return made;
}
