// The Python side of the attention and cache entry points: looks at the tensors of a
// call, refuses what does not fit, allocates what the caller left out and calls the C
// function of the same name (include/kda.h), whose address the package passes in.
// Their kernels take a few microseconds; the same checks written in Python took
// eight to fourteen per call.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <string>

#include "kda.h"

namespace {

struct Entry {
    decltype(&kda_attn_prefill_workspace_size) attn_prefill_workspace_size;
    decltype(&kda_attn_prefill) attn_prefill;
    decltype(&kda_attn_decode_workspace_size) attn_decode_workspace_size;
    decltype(&kda_attn_decode) attn_decode;
    decltype(&kda_cache_workspace_size) cache_workspace_size;
    decltype(&kda_cache_alloc) cache_alloc;
    decltype(&kda_cache_fork) cache_fork;
    decltype(&kda_cache_free) cache_free;
    decltype(&kda_cache_compact) cache_compact;
    decltype(&kda_cache_copy) cache_copy;
    decltype(&kda_cache_append) cache_append;
} kda_c;
PyObject *error_class = nullptr;  // KDAError(code, what)

PyObject *fail(int rc, const char *what) {
    PyObject *e = PyObject_CallFunction(error_class, "is", rc, what);
    if (e != nullptr) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return nullptr;
}
// The call itself, without the interpreter's lock (a full launch queue may block it).
template <typename F>
int call(F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = f();
    Py_END_ALLOW_THREADS return rc;
}

const at::Tensor &tensor(const char *name, PyObject *o) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}
int32_t i32(const char *name, int64_t x) {
    TORCH_CHECK_VALUE(x >= INT32_MIN && x <= INT32_MAX, name, " is too large");
    return static_cast<int32_t>(x);
}
int32_t i32(const char *name, PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return i32(name, static_cast<int64_t>(x));
}
float f32(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(x);
}
bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}
// The device of a call's tensors and its stream (None: the device's current one), while
// the call lasts: what it allocates belongs to that stream, as the kernels do.
struct Place {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard other;
    void *stream;
    Place(PyObject *o, int dev) : device(static_cast<c10::DeviceIndex>(dev)) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream().stream();
            return;
        }
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        if (h == nullptr) throw python_error();
        stream = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (stream == nullptr && PyErr_Occurred()) throw python_error();
        other.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), static_cast<c10::DeviceIndex>(dev)));
    }
};

int cuda_index(const at::Tensor &t) {
    TORCH_CHECK_VALUE(t.is_cuda(), "KDA tensors must be CUDA tensors");
    return t.get_device();
}
void check_kind(const char *name, const at::Tensor &t, at::ScalarType dtype, int dev) {
    TORCH_CHECK_VALUE(t.is_cuda(), "KDA tensors must be CUDA tensors");
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, " must have dtype ", at::toString(dtype));
    TORCH_CHECK_VALUE(t.get_device() == dev, "KDA tensors must be on one device");
}
void *take(const char *name, const at::Tensor &t, at::ScalarType dtype, int dev) {
    check_kind(name, t, dtype, dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.data_ptr();
}
void *take(const char *name, PyObject *o, at::ScalarType dtype, int dev) {  // None: NULL
    return o == Py_None ? nullptr : take(name, tensor(name, o), dtype, dev);
}
template <typename T>
T *take_as(const char *name, PyObject *o, at::ScalarType dtype, int dev) {
    return static_cast<T *>(take(name, o, dtype, dev));
}
void check_shape(const char *name, PyObject *o, at::IntArrayRef shape) {
    if (o != Py_None) TORCH_CHECK_VALUE(tensor(name, o).sizes() == shape, name, " must have the shape ", shape);
}

// Token rows [.., H, D]: the heads and channels of a row must be contiguous, the
// tokens evenly spaced.
struct Rows {
    void *p = nullptr;
    int64_t ld = 0;  // elements from one token to the next
};
Rows take_rows(const char *name, const at::Tensor &t, at::ScalarType dtype, int dev) {
    check_kind(name, t, dtype, dev);
    const auto size = t.sizes(), st = t.strides();
    const int64_t n = t.dim(), H = size[n - 2], D = size[n - 1];
    TORCH_CHECK_VALUE((st[n - 1] == 1 || D <= 1) && (st[n - 2] == D || H <= 1), name,
                      ": the [heads, D] rows must be contiguous");
    Rows r;
    r.p = t.data_ptr();
    if (t.numel() == 0) {  // no token: the strides say nothing
        r.ld = H * D;
    } else if (n == 3) {
        r.ld = size[0] > 1 ? st[0] : H * D;
    } else if (size[1] == 1) {
        r.ld = size[0] > 1 ? st[0] : H * D;
    } else {
        TORCH_CHECK_VALUE(size[0] <= 1 || st[0] == size[1] * st[1], name, ": the tokens must be evenly spaced");
        r.ld = st[1];
    }
    return r;
}
struct BlockTable {
    int32_t *p;
    int64_t ld;
    int32_t rows, cols;
    int dev;
};
BlockTable take_table(PyObject *o) {
    const at::Tensor &t = tensor("block_table", o);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_cuda() && t.dim() == 2,
                      "block_table must be a CUDA int32 [rows, cols] tensor");
    TORCH_CHECK_VALUE(t.size(1) <= 1 || t.stride(1) == 1, "the rows of block_table must be contiguous");
    BlockTable b;
    b.p = static_cast<int32_t *>(t.data_ptr());
    b.rows = i32("block_table", t.size(0));
    b.cols = i32("block_table", t.size(1));
    b.ld = b.rows > 1 ? t.stride(0) : b.cols;
    b.dev = static_cast<int>(t.get_device());
    return b;
}
int32_t io_of(at::ScalarType t) {  // -1: neither
    return t == at::kBFloat16 ? KDA_BF16 : (t == at::kFloat ? KDA_F32 : -1);
}
PyObject *bad_dtype(at::ScalarType t) {
    return fail(KDA_ERR_UNSUPPORTED, (std::string("dtype ") + at::toString(t)).c_str());
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}
struct Space {
    at::Tensor made;
    void *p;
    size_t bytes;
};
// The caller's workspace, or a new one of `need` bytes.
template <typename F>
Space workspace(PyObject *o, const at::Tensor &like, int dev, F need) {
    Space s;
    if (o == Py_None) {
        s.made = empty({static_cast<int64_t>(std::max<size_t>(need(), 256))}, at::kByte, like);
        s.made.narrow(0, 0, 256).zero_();
        s.p = s.made.data_ptr();
        s.bytes = s.made.numel();
    } else {
        const at::Tensor &t = tensor("workspace", o);
        s.p = take("workspace", t, at::kByte, dev);
        s.bytes = t.numel();
    }
    return s;
}
// An output: the caller's (of this shape), or a new one; `obj` is a new reference.
struct Out {
    PyObject *obj = nullptr;
    void *p = nullptr;
    Out() = default;
    Out(const Out &) = delete;
    ~Out() { Py_XDECREF(obj); }
    void take_or_make(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like,
                      int dev) {
        if (o != Py_None) {
            check_shape(name, o, shape);
            p = take(name, o, dtype, dev);
            obj = Py_NewRef(o);
        } else {
            at::Tensor t = empty(shape, dtype, like);
            p = t.data_ptr();
            obj = THPVariable_Wrap(std::move(t));
        }
    }
    void none() { obj = Py_NewRef(Py_None); }
    PyObject *give() {
        PyObject *o = obj;
        obj = nullptr;
        return o;
    }
};
PyObject *pair(Out &a, Out &b) {
    PyObject *t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, a.give());
    PyTuple_SET_ITEM(t, 1, b.give());
    return t;
}

#define ARGS(n) \
    if (nargs != (n)) { \
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments"); \
        return nullptr; \
    }

// (q, k, v, scale, cu_seqlens, cu_seqlens_k, N, out, lse, output_lse, workspace, stream)
PyObject *attn_prefill(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(12)
    const at::Tensor &q = tensor("q", x[0]), &k = tensor("k", x[1]), &v = tensor("v", x[2]);
    const int dev = cuda_index(q);
    const Place place(x[11], dev);
    const auto dt = q.scalar_type();
    const int32_t io = io_of(dt);
    if (io < 0) return bad_dtype(dt);
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "q and k must have the shape [tokens, heads, D]");
    const int32_t Tq = i32("q", q.size(0)), Hq = i32("q", q.size(1)), D = i32("q", q.size(2));
    const int32_t Tk = i32("k", k.size(0)), Hkv = i32("k", k.size(1));
    TORCH_CHECK_VALUE(v.sizes() == k.sizes() && k.size(2) == D, "k and v must have the shape [Tk_total, Hkv, D]");
    const Rows rq = take_rows("q", q, dt, dev), rk = take_rows("k", k, dt, dev), rv = take_rows("v", v, dt, dev);
    int32_t N, nq = Tq, nk = Tk;
    const int32_t *cu = take_as<int32_t>("cu_seqlens", x[4], at::kInt, dev);
    const int32_t *cuk = take_as<int32_t>("cu_seqlens_k", x[5], at::kInt, dev);
    if (x[4] != Py_None) {
        N = i32("cu_seqlens", THPVariable_Unpack(x[4]).numel() - 1);
        TORCH_CHECK_VALUE(x[5] == Py_None || THPVariable_Unpack(x[5]).numel() == N + 1,
                          "cu_seqlens_k must have as many offsets as cu_seqlens");
    } else {
        N = i32("N", x[6]);
        TORCH_CHECK_VALUE(x[5] == Py_None, "cu_seqlens_k needs cu_seqlens");
        TORCH_CHECK_VALUE(N >= 1 && Tq % N == 0 && Tk % N == 0, "q and k must hold N sequences of equal length");
        nq = Tq / N;
        nk = Tk / N;
    }
    Out out, lse;
    out.take_or_make("out", x[7], q.sizes(), dt, q, dev);
    if (x[8] != Py_None || truth(x[9])) lse.take_or_make("lse", x[8], {Tq, Hq}, at::kFloat, q, dev);
    else lse.none();
    const Space ws = workspace(x[10], q, dev, [&] { return kda_c.attn_prefill_workspace_size(N, Tq, Tk, Hq, Hkv, D, io); });
    const float scale = f32(x[3]);
    const int rc = call([&] {
        return kda_c.attn_prefill(rq.p, rk.p, rv.p, rq.ld, rk.ld, rv.ld, scale, cu, cuk, N, nq, nk, Hq, Hkv, D, io, out.p,
                                  static_cast<float *>(lse.p), ws.p, ws.bytes, place.stream);
    });
    return rc == KDA_OK ? pair(out, lse) : fail(rc, "kda_attn_prefill");
    END_HANDLE_TH_ERRORS
}

// (q, k_pages, v_pages, block_table, seq_lens, scale, k_new, v_new, tree_mask, out, lse, output_lse, workspace,
// stream)
PyObject *attn_decode(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(14)
    const at::Tensor &q = tensor("q", x[0]), &kp = tensor("k_pages", x[1]), &vp = tensor("v_pages", x[2]);
    const int dev = cuda_index(q);
    const Place place(x[13], dev);
    const auto dt = q.scalar_type();
    const int32_t io = io_of(dt);
    if (io < 0) return bad_dtype(dt);
    TORCH_CHECK_VALUE(q.dim() == 4 && kp.dim() == 4, "q must have the shape [B, T, Hq, D], the pools [P, Hkv, page, D]");
    const int32_t B = i32("q", q.size(0)), T = i32("q", q.size(1)), Hq = i32("q", q.size(2)), D = i32("q", q.size(3));
    const int32_t P = i32("k_pages", kp.size(0)), Hkv = i32("k_pages", kp.size(1)), page = i32("k_pages", kp.size(2));
    TORCH_CHECK_VALUE(vp.sizes() == kp.sizes() && kp.size(3) == D,
                      "k_pages and v_pages must have the shape [P, Hkv, page, D]");
    const Rows rq = take_rows("q", q, dt, dev);
    Rows rk, rv;
    check_shape("k_new", x[6], {B, T, Hkv, D});
    check_shape("v_new", x[7], {B, T, Hkv, D});
    if (x[6] != Py_None) rk = take_rows("k_new", THPVariable_Unpack(x[6]), dt, dev);
    if (x[7] != Py_None) rv = take_rows("v_new", THPVariable_Unpack(x[7]), dt, dev);
    const BlockTable table = take_table(x[3]);
    TORCH_CHECK_VALUE(table.dev == dev, "KDA tensors must be on one device");
    TORCH_CHECK_VALUE(table.rows == B && tensor("seq_lens", x[4]).sizes() == at::IntArrayRef({B}),
                      "block_table and seq_lens must have a row for each sequence");
    check_shape("tree_mask", x[8], {B, T});
    const int32_t *lens = take_as<int32_t>("seq_lens", x[4], at::kInt, dev);
    const uint64_t *mask = take_as<uint64_t>("tree_mask", x[8], at::kLong, dev);
    const void *k_pages = take("k_pages", kp, dt, dev), *v_pages = take("v_pages", vp, dt, dev);
    Out out, lse;
    out.take_or_make("out", x[9], q.sizes(), dt, q, dev);
    if (x[10] != Py_None || truth(x[11])) lse.take_or_make("lse", x[10], {B, T, Hq}, at::kFloat, q, dev);
    else lse.none();
    const Space ws = workspace(x[12], q, dev, [&] {
        return kda_c.attn_decode_workspace_size(B, T, Hq, Hkv, D, page, table.cols, io);
    });
    const float scale = f32(x[5]);
    const int rc = call([&] {
        return kda_c.attn_decode(rq.p, rq.ld, rk.p, rv.p, rk.ld, rv.ld, k_pages, v_pages, P, page, table.p, table.ld,
                                 table.cols, lens, mask, scale, B, T, Hq, Hkv, D, io, out.p, static_cast<float *>(lse.p),
                                 ws.p, ws.bytes, place.stream);
    });
    return rc == KDA_OK ? pair(out, lse) : fail(rc, "kda_attn_decode");
    END_HANDLE_TH_ERRORS
}

struct Refs {
    int32_t *p;
    int32_t pages;
};
Refs take_refs(PyObject *o, int dev) {
    const at::Tensor &t = tensor("refs", o);
    return {static_cast<int32_t *>(take("refs", t, at::kInt, dev)), i32("refs", t.numel())};
}
Space cache_space(PyObject *ws, PyObject *table, const BlockTable &b, const Refs &r) {
    return workspace(ws, THPVariable_Unpack(table), b.dev, [&] { return kda_c.cache_workspace_size(r.pages, b.rows); });
}
int32_t *take_lens(PyObject *o, const BlockTable &b) {
    TORCH_CHECK_VALUE(tensor("seq_lens", o).sizes() == at::IntArrayRef({b.rows}),
                      "seq_lens must have an entry for each row");
    return take_as<int32_t>("seq_lens", o, at::kInt, b.dev);
}

// (block_table, want, refs, page_size, workspace, stream)
PyObject *cache_alloc(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(6)
    const BlockTable b = take_table(x[0]);
    const Place place(x[5], b.dev);
    TORCH_CHECK_VALUE(tensor("want", x[1]).sizes() == at::IntArrayRef({b.rows}), "want must have an entry for each row");
    const int32_t *want = take_as<int32_t>("want", x[1], at::kInt, b.dev);
    const Refs refs = take_refs(x[2], b.dev);
    const int32_t page = i32("page_size", x[3]);
    const Space ws = cache_space(x[4], x[0], b, refs);
    const int rc = call([&] {
        return kda_c.cache_alloc(b.p, b.ld, b.rows, b.cols, want, refs.p, refs.pages, page, ws.p, ws.bytes, place.stream);
    });
    if (rc != KDA_OK) return fail(rc, "kda_cache_alloc");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (block_table, seq_lens, refs, src, dst, page_size, copies, workspace, stream)
PyObject *cache_fork(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(9)
    const BlockTable b = take_table(x[0]);
    const Place place(x[8], b.dev);
    int32_t *const lens = take_lens(x[1], b);
    const Refs refs = take_refs(x[2], b.dev);
    const int32_t n = i32("src", tensor("src", x[3]).numel()), page = i32("page_size", x[5]);
    TORCH_CHECK_VALUE(tensor("dst", x[4]).numel() == n, "src and dst must pair up");
    const int32_t *src = take_as<int32_t>("src", x[3], at::kInt, b.dev), *dst = take_as<int32_t>("dst", x[4], at::kInt, b.dev);
    Out copies;
    copies.take_or_make("copies", x[6], {n, 2}, at::kInt, THPVariable_Unpack(x[0]), b.dev);
    const Space ws = cache_space(x[7], x[0], b, refs);
    const int rc = call([&] {
        return kda_c.cache_fork(b.p, b.ld, b.rows, b.cols, lens, refs.p, refs.pages, page, src, dst, n,
                                static_cast<int32_t *>(copies.p), ws.p, ws.bytes, place.stream);
    });
    return rc == KDA_OK ? copies.give() : fail(rc, "kda_cache_fork");
    END_HANDLE_TH_ERRORS
}

// (block_table, seq_lens, refs, rows, workspace, stream)
PyObject *cache_free(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(6)
    const BlockTable b = take_table(x[0]);
    const Place place(x[5], b.dev);
    int32_t *const lens = take_lens(x[1], b);
    const Refs refs = take_refs(x[2], b.dev);
    const int32_t n = i32("rows", tensor("rows", x[3]).numel());
    const int32_t *rows = take_as<int32_t>("rows", x[3], at::kInt, b.dev);
    const Space ws = cache_space(x[4], x[0], b, refs);
    const int rc = call([&] {
        return kda_c.cache_free(b.p, b.ld, b.rows, b.cols, lens, refs.p, refs.pages, rows, n, ws.p, ws.bytes, place.stream);
    });
    if (rc != KDA_OK) return fail(rc, "kda_cache_free");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (block_table, refs, copies, count, workspace, stream)
PyObject *cache_compact(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(6)
    const BlockTable b = take_table(x[0]);
    const Place place(x[5], b.dev);
    const Refs refs = take_refs(x[1], b.dev);
    Out copies, count;
    copies.take_or_make("copies", x[2], {refs.pages, 2}, at::kInt, THPVariable_Unpack(x[0]), b.dev);
    if (x[3] != Py_None) TORCH_CHECK_VALUE(tensor("count", x[3]).numel() >= 1, "count must have an entry");
    if (x[3] != Py_None) {
        count.p = take("count", x[3], at::kInt, b.dev);
        count.obj = Py_NewRef(x[3]);
    } else {
        count.take_or_make("count", x[3], {1}, at::kInt, THPVariable_Unpack(x[0]), b.dev);
    }
    const Space ws = cache_space(x[4], x[0], b, refs);
    const int rc = call([&] {
        return kda_c.cache_compact(b.p, b.ld, b.rows, b.cols, refs.p, refs.pages, static_cast<int32_t *>(copies.p),
                                   static_cast<int32_t *>(count.p), ws.p, ws.bytes, place.stream);
    });
    return rc == KDA_OK ? pair(copies, count) : fail(rc, "kda_cache_compact");
    END_HANDLE_TH_ERRORS
}

// (pools, copies, count, stream)
PyObject *cache_copy(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(4)
    struct Items {
        PyObject *o;
        ~Items() { Py_XDECREF(o); }
    } items{PySequence_Fast(x[0], "pools must be a sequence of tensors")};
    if (items.o == nullptr) return nullptr;
    const int32_t n_pools = i32("pools", PySequence_Fast_GET_SIZE(items.o));
    if (n_pools == 0) Py_RETURN_NONE;
    const at::Tensor &first = tensor("pools", PySequence_Fast_GET_ITEM(items.o, 0)), &copies = tensor("copies", x[1]);
    const int dev = cuda_index(first);
    const Place place(x[3], dev);
    TORCH_CHECK_VALUE(copies.dim() == 2 && copies.size(1) == 2, "copies must have the shape [n, 2]");
    TORCH_CHECK_VALUE(first.dim() > 0, "the pools must have entries of one size");
    const int32_t entries = i32("pools", first.size(0)), n = i32("copies", copies.size(0));
    const int64_t bytes = static_cast<int64_t>(first.nbytes());
    c10::SmallVector<void *, 64> ptrs;
    for (int32_t i = 0; i < n_pools; ++i) {
        const at::Tensor &p = tensor("pools", PySequence_Fast_GET_ITEM(items.o, i));
        TORCH_CHECK_VALUE(p.dim() > 0 && p.size(0) == entries && static_cast<int64_t>(p.nbytes()) == bytes,
                          "the pools must have entries of one size");
        ptrs.push_back(take("pools", p, p.scalar_type(), dev));
    }
    const int32_t *pairs = static_cast<int32_t *>(take("copies", copies, at::kInt, dev));
    const int32_t *count = take_as<int32_t>("count", x[2], at::kInt, dev);
    const int rc = call([&] {
        return kda_c.cache_copy(ptrs.data(), n_pools, bytes / std::max(entries, 1), entries, pairs, n, count, place.stream);
    });
    if (rc != KDA_OK) return fail(rc, "kda_cache_copy");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (k, v, k_pages, v_pages, block_table, start, cu_seqlens, index, count, workspace, stream)
PyObject *cache_append(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    ARGS(11)
    const at::Tensor &k = tensor("k", x[0]), &v = tensor("v", x[1]), &kp = tensor("k_pages", x[2]),
                     &vp = tensor("v_pages", x[3]);
    const int dev = cuda_index(k);
    const Place place(x[10], dev);
    const auto dt = k.scalar_type();
    const int32_t io = io_of(dt);
    if (io < 0) return bad_dtype(dt);
    TORCH_CHECK_VALUE(kp.dim() == 4 && vp.sizes() == kp.sizes() && v.sizes() == k.sizes() && k.dim() >= 2 &&
                          k.size(-2) == kp.size(1) && k.size(-1) == kp.size(3),
                      "k, v must be rows of [Hkv, D], the pools [P, Hkv, page, D]");
    const int32_t P = i32("k_pages", kp.size(0)), Hkv = i32("k_pages", kp.size(1)), page = i32("k_pages", kp.size(2)),
                  D = i32("k_pages", kp.size(3));
    int32_t N, T;
    if (x[6] != Py_None) {
        TORCH_CHECK_VALUE(k.dim() == 3, "packed rows must be [T_total, Hkv, D]");
        N = i32("cu_seqlens", tensor("cu_seqlens", x[6]).numel() - 1);
        T = i32("k", k.size(0));
    } else {
        TORCH_CHECK_VALUE(k.dim() == 4, "rows without cu_seqlens must be [N, T, Hkv, D]");
        N = i32("k", k.size(0));
        T = i32("k", k.size(1));
    }
    const Rows rk = take_rows("k", k, dt, dev), rv = take_rows("v", v, dt, dev);
    const BlockTable b = take_table(x[4]);
    TORCH_CHECK_VALUE(b.dev == dev, "KDA tensors must be on one device");
    TORCH_CHECK_VALUE(b.rows >= N && tensor("start", x[5]).sizes() == at::IntArrayRef({N}),
                      "block_table and start must have a row for each sequence");
    check_shape("index", x[7], {N, T});
    check_shape("count", x[8], {N});
    const int32_t *cu = take_as<int32_t>("cu_seqlens", x[6], at::kInt, dev), *index = take_as<int32_t>("index", x[7], at::kInt, dev),
                  *count = take_as<int32_t>("count", x[8], at::kInt, dev), *start = take_as<int32_t>("start", x[5], at::kInt, dev);
    void *const k_pages = take("k_pages", kp, dt, dev), *const v_pages = take("v_pages", vp, dt, dev);
    void *const ws = take("workspace", x[9], at::kByte, dev);
    const int rc = call([&] {
        return kda_c.cache_append(rk.p, rv.p, rk.ld, rv.ld, cu, N, T, index, count, start, b.p, b.ld, b.cols, P, page, Hkv,
                                  D, io, k_pages, v_pages, ws, place.stream);
    });
    if (rc != KDA_OK) return fail(rc, "kda_cache_append");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (addresses of the C functions in the order of Entry, KDAError)
PyObject *init(PyObject *, PyObject *const *x, Py_ssize_t nargs) {
    constexpr Py_ssize_t n = sizeof(Entry) / sizeof(void *);
    ARGS(2)
    void *p[n];
    if (!PyTuple_Check(x[0]) || PyTuple_GET_SIZE(x[0]) != n) {
        PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(x[0], i));
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
            return nullptr;
        }
    }
    std::memcpy(static_cast<void *>(&kda_c), p, sizeof(kda_c));
    Py_XSETREF(error_class, Py_NewRef(x[1]));
    Py_RETURN_NONE;
}

#define METHOD(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(init),       METHOD(attn_prefill),  METHOD(attn_decode), METHOD(cache_alloc), METHOD(cache_fork),
                         METHOD(cache_free), METHOD(cache_compact), METHOD(cache_copy),  METHOD(cache_append),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_bind() { return PyModule_Create(&module); }
