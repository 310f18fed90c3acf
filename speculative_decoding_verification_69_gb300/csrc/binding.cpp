// binding.cpp -- the Python side of include/spec_cache.h: reads shapes, strides
// and pointers out of torch tensors, checks them, allocates results and calls
// the C ABI.  Compiled, because the same steps in Python (ctypes) cost 23.5 us of
// host time for an attention call whose kernels take 12.8 us at one token and one
// request, and 19 for two resizes and an append; here 9.1 (its workspace included) and 6.8.
//
// Every function takes its arguments by position and returns None (or its
// results); a status other than SPEC_OK becomes SpecVerifyError.
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <string>
#include <vector>

#include "spec_cache.h"

namespace {

const at::Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch tensor");
    return THPVariable_Unpack(o);
}

void together(const at::Tensor &t, const at::Tensor &with, const char *name) {
    TORCH_CHECK_VALUE(t.device() == with.device(), name, " is on ", t.device(), ", not on ", with.device());
}

uint32_t *status(PyObject *o, const at::Tensor &with) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "dev_status");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_cuda() && t.numel() > 0,
                      "dev_status must be an int32 CUDA tensor");
    together(t, with, "dev_status");
    return reinterpret_cast<uint32_t *>(t.data_ptr<int>());
}

long long integer(PyObject *o, const char *name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be an integer");
    }
    return x;
}

int small(PyObject *o, const char *name) {
    const long long x = integer(o, name);
    TORCH_CHECK_VALUE(x >= INT_MIN && x <= INT_MAX, name, " is out of range");
    return (int)x;
}

// An int32 CUDA tensor, contiguous, of this shape (-1: any extent), on the device of `with`
// if that is given.
const at::Tensor &ints(PyObject *o, const char *name, const at::Tensor *with, int64_t n0, int64_t n1 = -2) {
    const at::Tensor &t = tensor(o, name);
    const int dims = n1 == -2 ? 1 : 2;
    bool ok = t.scalar_type() == at::kInt && t.is_cuda() && t.is_contiguous() && t.dim() == dims;
    ok = ok && (n0 < 0 || t.size(0) == n0) && (dims == 1 || n1 < 0 || t.size(1) == n1);
    if (!ok) {
        auto extent = [](int64_t n) { return n < 0 ? std::string("*") : std::to_string(n); };
        TORCH_CHECK_VALUE(false, name, " must be a contiguous int32 CUDA tensor [", extent(n0),
                          dims == 2 ? ", " + extent(n1) : std::string(), "]");
    }
    if (with) together(t, *with, name);
    return t;
}

// The stride of a dimension; one of one element is never stepped over, so any
// valid stride stands for it.
long long stride(const at::Tensor &t, int dim) {
    return t.size(dim) > 1 ? t.stride(dim) : t.size(-1);
}

// The operators have no backward pass: a call whose gradient would be lost is refused.
void no_gradient(const at::Tensor &t, const char *name) {
    TORCH_CHECK_VALUE(!(t.requires_grad() && c10::GradMode::is_enabled()), name,
                      " requires a gradient, and this call has none: make it under torch.no_grad(), or detach ", name);
}

// A pool of pages, [num_pages, page_size, heads, head_dim], with the layers in
// front of them when `layered`.
spec_pages_t pool(PyObject *ko, PyObject *vo, bool layered) {
    const at::Tensor &k = tensor(ko, "k"), &v = tensor(vo, "v");
    const int d = layered ? 1 : 0;
    TORCH_CHECK_VALUE(k.dim() == 4 + d && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
                      "k and v must be alike, [", layered ? "layers, " : "",
                      "num_pages, page_size, kv_heads, head_dim]");
    spec_pages_t p = {};
    switch (k.scalar_type()) {
    case at::kFloat: p.dtype = SPEC_DTYPE_F32; break;
    case at::kBFloat16: p.dtype = SPEC_DTYPE_BF16; break;
    case at::kHalf: p.dtype = SPEC_DTYPE_F16; break;
    default: TORCH_CHECK_TYPE(false, "a cache is bfloat16, float16 or float32");
    }
    TORCH_CHECK_VALUE(k.is_cuda() && v.is_cuda(), "k and v must be CUDA tensors");
    together(v, k, "v");
    no_gradient(k, "k");
    no_gradient(v, "v");
    bool same = k.stride(-1) == 1 && v.stride(-1) == 1;
    for (int i = 0; i < 3 + d; ++i) same = same && stride(k, i) == stride(v, i);
    TORCH_CHECK_VALUE(same, "k and v need the same strides and a contiguous head_dim");
    for (int i = 0; i < 4 + d; ++i) TORCH_CHECK_VALUE(k.size(i) <= INT_MAX, "a cache dimension is too large");
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.layers = layered ? (int)k.size(0) : 1;
    p.num_pages = (int)k.size(d);
    p.page_size = (int)k.size(d + 1);
    p.heads = (int)k.size(d + 2);
    p.head_dim = (int)k.size(d + 3);
    p.layer_stride = layered ? stride(k, 0) : 0;
    p.page_stride = stride(k, d);
    p.token_stride = stride(k, d + 1);
    p.head_stride = stride(k, d + 2);
    return p;
}

// A [B, N, heads, head_dim] tensor of the cache's dtype.
const at::Tensor &rows(PyObject *o, const char *name, const at::Tensor &k, int64_t heads) {
    const at::Tensor &t = tensor(o, name);
    TORCH_CHECK_VALUE(t.dim() == 4 && t.scalar_type() == k.scalar_type() && t.is_cuda() &&
                          t.size(3) == k.size(-1) && t.stride(3) == 1 && (heads < 0 || t.size(2) == heads) &&
                          t.size(0) <= INT_MAX && t.size(1) <= INT_MAX && t.size(2) <= INT_MAX,
                      name, " must be a CUDA tensor [B, N, ", heads < 0 ? std::string("heads") : std::to_string(heads),
                      ", ", k.size(-1), "] of the cache's dtype, its last dimension contiguous");
    together(t, k, name);
    no_gradient(t, name);
    return t;
}

spec_dtype_t dtype16(const at::Tensor &t, const char *name) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf, name,
                     " must be bfloat16 or float16");
    return t.scalar_type() == at::kBFloat16 ? SPEC_DTYPE_BF16 : SPEC_DTYPE_F16;
}

// A 4-bit pool, [num_pages, kv_heads, bytes], with the layers in front when `layered` is 1
// (-1: with or without them).
spec_pages4_t pool4(PyObject *o, int layered, long long page_size, long long head_dim) {
    const at::Tensor &t = tensor(o, "pool");
    if (layered < 0) layered = t.dim() == 4;
    const int d = layered;
    TORCH_CHECK_VALUE(t.dim() == 3 + d && t.scalar_type() == at::kByte && t.is_cuda(),
                      "a 4-bit pool is a uint8 CUDA tensor [", layered ? "layers, " : "",
                      "num_pages, kv_heads, page_bytes]");
    for (int i = 0; i < 3 + d; ++i) TORCH_CHECK_VALUE(t.size(i) <= INT_MAX, "a cache dimension is too large");
    const size_t bytes = page_size > INT_MAX || head_dim > INT_MAX || page_size < 0 || head_dim < 0
                             ? 0
                             : spec_cache4_page_bytes((int)page_size, (int)head_dim);
    TORCH_CHECK_VALUE(bytes != 0, "page_size must be a power of two of at least 8, head_dim a multiple of 8 up to ",
                      SPEC_MAX_HEAD_DIM);
    TORCH_CHECK_VALUE(t.size(2 + d) == (int64_t)bytes && t.stride(2 + d) == 1, "pages of ", page_size, " tokens with a head_dim of ",
                      head_dim, " have ", bytes, " contiguous bytes per head");
    spec_pages4_t p = {};
    p.data = t.data_ptr();
    p.layers = layered ? (int)t.size(0) : 1;
    p.num_pages = (int)t.size(d);
    p.heads = (int)t.size(d + 1);
    p.page_size = (int)page_size;
    p.head_dim = (int)head_dim;
    p.layer_stride = layered ? stride(t, 0) : 0;
    p.page_stride = stride(t, d);
    p.head_stride = stride(t, d + 1);
    return p;
}

// A [B, N, heads, head_dim] tensor, bfloat16 or float16, on the device of `with`.
const at::Tensor &rows16(PyObject *o, const char *name, const at::Tensor &with, int64_t heads) {
    const at::Tensor &t = tensor(o, name);
    dtype16(t, name);
    TORCH_CHECK_VALUE(t.dim() == 4 && t.is_cuda() && t.stride(3) == 1 && (heads < 0 || t.size(2) == heads) &&
                          t.size(0) <= INT_MAX && t.size(1) <= INT_MAX && t.size(2) <= INT_MAX && t.size(3) <= INT_MAX,
                      name, " must be a CUDA tensor [B, N, ", heads < 0 ? std::string("heads") : std::to_string(heads),
                      ", head_dim], its last dimension contiguous");
    together(t, with, name);
    no_gradient(t, name);
    return t;
}

// A page table [B, max_pages], or [B, heads, max_pages] with a list for every key head.
const at::Tensor &lists(PyObject *o, const at::Tensor &with, int64_t B, int64_t heads) {
    const at::Tensor &t = tensor(o, "page_table");
    if (t.dim() != 3) return ints(o, "page_table", &with, B, -1);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_cuda() && t.is_contiguous() && t.size(0) == B &&
                          t.size(1) == heads,
                      "page_table must be a contiguous int32 CUDA tensor [", B, ", *] or [", B, ", ", heads, ", *]");
    together(t, with, "page_table");
    return t;
}

// The stream given, or torch's current one.
void *handle(PyObject *o, const at::Tensor &with) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(with.device().index()).stream();
    return reinterpret_cast<void *>((intptr_t)integer(o, "stream"));
}

// The workspace given, or one of this call's own from torch's allocator, on the current
// stream: reused in that stream's order, and in a captured graph part of the graph's memory.
at::Tensor workspace(PyObject *o, const at::Tensor &with, size_t bytes) {
    if (o == Py_None) return at::empty({(int64_t)std::max<size_t>(bytes, 256)}, with.options().dtype(at::kByte));
    const at::Tensor &t = tensor(o, "workspace");
    TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous(), "workspace must be a contiguous CUDA tensor");
    together(t, with, "workspace");
    return t;
}

PyObject *done(spec_status_t st) {
    if (st == SPEC_OK) Py_RETURN_NONE;
    PyObject *m = PyImport_ImportModule("speculative_decoding_verification_69_gb300");
    PyObject *e = m ? PyObject_GetAttrString(m, "SpecVerifyError") : nullptr;
    if (e) PyErr_Format(e, "%s (%d)", spec_status_str(st), (int)st);
    Py_XDECREF(e);
    Py_XDECREF(m);
    return nullptr;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *x = THPVariable_Wrap(a), *y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject *both = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return both;
}

void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// (page_table, page_count, page_ref, want_len, page_size, extra, dev_status, stream)
PyObject *resize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const at::Tensor &table = ints(a[0], "page_table", nullptr, -1, -1);
    const int64_t B = table.size(0);
    const at::Tensor &held = ints(a[1], "page_count", &table, B), &ref = ints(a[2], "page_ref", &table, -1),
                     &want = ints(a[3], "want_len", &table, B);
    const c10::DeviceGuard guard(table.device());
    return done(spec_cache_resize(table.data_ptr<int>(), held.data_ptr<int>(), ref.data_ptr<int>(),
                                  want.data_ptr<int>(), small(a[5], "extra"), small(a[4], "page_size"), (int)B,
                                  (int)table.size(1), (int)ref.size(0), status(a[6], table),
                                  handle(a[7], table)));
    END_HANDLE_TH_ERRORS
}

// (k, v, page_table, page_count, page_ref, cache_len, src, dst, workspace, dev_status, stream)
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 11);
    const spec_pages_t p = pool(a[0], a[1], true);
    const at::Tensor &k = tensor(a[0], "k");
    const at::Tensor &table = ints(a[2], "page_table", &k, -1, -1);
    const int64_t S = table.size(0);
    const at::Tensor &held = ints(a[3], "page_count", &k, S), &ref = ints(a[4], "page_ref", &k, p.num_pages),
                     &len = ints(a[5], "cache_len", &k, S), &src = ints(a[6], "src", &k, -1),
                     &dst = ints(a[7], "dst", &k, src.size(0));
    const c10::DeviceGuard guard(table.device());
    const at::Tensor ws = workspace(a[8], k, spec_cache_fork_workspace_bytes((int)std::min<int64_t>(src.size(0), INT_MAX)));
    return done(spec_cache_fork(&p, table.data_ptr<int>(), held.data_ptr<int>(), ref.data_ptr<int>(),
                                len.data_ptr<int>(), src.data_ptr<int>(), dst.data_ptr<int>(), (int)src.size(0),
                                (int)S, (int)table.size(1), ws.data_ptr(), (size_t)ws.nbytes(),
                                status(a[9], k), handle(a[10], k)));
    END_HANDLE_TH_ERRORS
}

// (k, v, src_pages, dst_pages, dev_status, stream)
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);
    const spec_pages_t p = pool(a[0], a[1], true);
    const at::Tensor &k = tensor(a[0], "k");
    const at::Tensor &src = ints(a[2], "src_pages", &k, -1), &dst = ints(a[3], "dst_pages", &k, src.size(0));
    const c10::DeviceGuard guard(src.device());
    return done(spec_cache_copy(&p, src.data_ptr<int>(), dst.data_ptr<int>(), (int)src.size(0),
                                status(a[4], k), handle(a[5], k)));
    END_HANDLE_TH_ERRORS
}

// (k, v, page_table, cache_len, k_new, v_new, count, dev_status, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ::count(n, 9);
    const spec_pages_t p = pool(a[0], a[1], false);
    const at::Tensor &k = tensor(a[0], "k");
    const at::Tensor &kn = rows(a[4], "k_new", k, p.heads), &vn = rows(a[5], "v_new", k, p.heads);
    bool same = kn.sizes() == vn.sizes();
    for (int i = 0; i < 3; ++i) same = same && stride(kn, i) == stride(vn, i);
    TORCH_CHECK_VALUE(same, "k_new and v_new need the same shape and strides");
    const int64_t B = kn.size(0);
    const at::Tensor &table = ints(a[2], "page_table", &k, B, -1), &len = ints(a[3], "cache_len", &k, B);
    const int *cnt = a[6] == Py_None ? nullptr : ints(a[6], "count", &k, B).data_ptr<int>();
    const c10::DeviceGuard guard(table.device());
    return done(spec_cache_append(&p, table.data_ptr<int>(), len.data_ptr<int>(), kn.data_ptr(), vn.data_ptr(),
                                  stride(kn, 0), stride(kn, 1), stride(kn, 2), cnt, (int)B, (int)kn.size(1),
                                  (int)table.size(1), status(a[7], k), handle(a[8], k)));
    END_HANDLE_TH_ERRORS
}

// (k, v, page_table, cache_len, out_nodes, accept_len, new_len, nodes, dev_status, stream)
PyObject *commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ::count(n, 10);
    const spec_pages_t p = pool(a[0], a[1], true);
    const at::Tensor &k = tensor(a[0], "k");
    const at::Tensor &table = ints(a[2], "page_table", &k, -1, -1);
    const int64_t B = table.size(0);
    const at::Tensor &len = ints(a[3], "cache_len", &k, B);
    const int *out = nullptr;
    int N;
    if (a[4] != Py_None) {
        const at::Tensor &t = ints(a[4], "out_nodes", &k, B, -1);
        out = t.data_ptr<int>();
        N = (int)t.size(1);
    } else {
        TORCH_CHECK_VALUE(a[7] != Py_None, "linear drafts need their number of nodes");
        N = small(a[7], "nodes");
    }
    const at::Tensor &acc = ints(a[5], "accept_len", &k, B), &fresh = ints(a[6], "new_len", &k, B);
    const c10::DeviceGuard guard(table.device());
    return done(spec_cache_commit(&p, table.data_ptr<int>(), len.data_ptr<int>(), out, acc.data_ptr<int>(),
                                  fresh.data_ptr<int>(), (int)B, N, (int)table.size(1),
                                  status(a[8], k), handle(a[9], k)));
    END_HANDLE_TH_ERRORS
}

// What the two attentions share: arguments behind the pool, results, and how they are returned.
struct Attention {
    const at::Tensor &q;
    int64_t B, N, Hq, D;
    const at::Tensor &table, &len;
    const int *parent, *nodes;
    double scale;
    int window, sinks;
    at::Tensor out, lse;

    // a: page_table, cache_len; then `rest`: parent, node_count, scale, window, sinks, out, return_lse
    Attention(const at::Tensor &query, const at::Tensor &with, int64_t heads, PyObject *const *a, PyObject *const *rest)
        : q(query), B(q.size(0)), N(q.size(1)), Hq(q.size(2)), D(q.size(3)), table(lists(a[0], with, B, heads)),
          len(ints(a[1], "cache_len", &with, B)) {
        parent = rest[0] == Py_None ? nullptr : ints(rest[0], "parent", &with, B, N).data_ptr<int>();
        nodes = rest[1] == Py_None ? nullptr : ints(rest[1], "node_count", &with, B).data_ptr<int>();
        scale = 1.0 / std::sqrt((double)D);
        if (rest[2] != Py_None) {
            scale = PyFloat_AsDouble(rest[2]);
            if (PyErr_Occurred()) throw python_error();
        }
        window = small(rest[3], "window"), sinks = small(rest[4], "sinks");
        if (rest[5] != Py_None) {
            out = tensor(rest[5], "out");
            TORCH_CHECK_VALUE(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() && out.is_cuda() &&
                                  out.is_contiguous() && out.device() == q.device(),
                              "out must be a contiguous CUDA tensor of q's shape and dtype");
            no_gradient(out, "out");
        } else {
            out = at::empty(q.sizes(), q.options());
        }
        const int with_lse = PyObject_IsTrue(rest[6]);
        if (with_lse < 0) throw python_error();
        if (with_lse) lse = at::empty({B, N, Hq}, q.options().dtype(at::kFloat));
    }
    float *lse_ptr() { return lse.defined() ? lse.data_ptr<float>() : nullptr; }
    PyObject *results(spec_status_t st) {
        if (st != SPEC_OK) return done(st);
        return lse.defined() ? pair(out, lse) : THPVariable_Wrap(out);
    }
};

// (q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out, return_lse, workspace,
//  dev_status, stream) -> out, or (out, lse)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 15);
    const spec_pages_t p = pool(a[1], a[2], false);
    const at::Tensor &k = tensor(a[1], "k");
    Attention x(rows(a[0], "q", k, -1), k, p.heads, a + 3, a + 5);
    const c10::DeviceGuard guard(k.device());
    const at::Tensor ws =
        workspace(a[12], k, spec_tree_attention_workspace_bytes((int)x.B, (int)x.N, (int)x.Hq, p.heads, (int)x.D));
    const auto call = x.table.dim() == 3 ? spec_sparse_attention : spec_tree_attention;
    return x.results(call(x.q.data_ptr(), stride(x.q, 0), stride(x.q, 1), stride(x.q, 2), &p, x.table.data_ptr<int>(),
                          x.len.data_ptr<int>(), x.parent, x.nodes, (int)x.B, (int)x.N, (int)x.Hq,
                          (int)x.table.size(-1), (float)x.scale, x.window, x.sinks, x.out.data_ptr(), x.lse_ptr(),
                          ws.data_ptr(), (size_t)ws.nbytes(), status(a[13], k), handle(a[14], k)));
    END_HANDLE_TH_ERRORS
}

// (q, pool, page_table, cache_len, page_size, parent, node_count, scale, window, sinks, out, return_lse, workspace,
//  dev_status, stream) -> out, or (out, lse)
PyObject *tree_attention4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 15);
    const at::Tensor &data = tensor(a[1], "pool"), &q = rows16(a[0], "q", data, -1);
    const spec_pages4_t p = pool4(a[1], 0, integer(a[4], "page_size"), q.size(3));
    Attention x(q, data, p.heads, a + 2, a + 5);
    const c10::DeviceGuard guard(data.device());
    const at::Tensor ws =
        workspace(a[12], data, spec_tree_attention4_workspace_bytes((int)x.B, (int)x.N, (int)x.Hq, p.heads, (int)x.D));
    return x.results(spec_tree_attention4(
        q.data_ptr(), dtype16(q, "q"), stride(q, 0), stride(q, 1), stride(q, 2), &p, x.table.data_ptr<int>(),
        x.table.dim() == 3 ? 1 : 0, x.len.data_ptr<int>(), x.parent, x.nodes, (int)x.B, (int)x.N, (int)x.Hq,
        (int)x.table.size(-1), (float)x.scale, x.window, x.sinks, x.out.data_ptr(), x.lse_ptr(), ws.data_ptr(),
        (size_t)ws.nbytes(), status(a[13], data), handle(a[14], data)));
    END_HANDLE_TH_ERRORS
}

// (pool, page_table, cache_len, k_new, v_new, page_size, count, dev_status, stream)
PyObject *append4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ::count(n, 9);
    const at::Tensor &data = tensor(a[0], "pool"), &kn = rows16(a[3], "k_new", data, -1);
    const spec_pages4_t p = pool4(a[0], 0, integer(a[5], "page_size"), kn.size(3));
    rows16(a[3], "k_new", data, p.heads);
    const at::Tensor &vn = rows16(a[4], "v_new", data, p.heads);
    bool same = kn.sizes() == vn.sizes() && kn.scalar_type() == vn.scalar_type();
    for (int i = 0; i < 3; ++i) same = same && stride(kn, i) == stride(vn, i);
    TORCH_CHECK_VALUE(same, "k_new and v_new need the same shape, strides and dtype");
    const int64_t B = kn.size(0);
    const at::Tensor &table = ints(a[1], "page_table", &data, B, -1), &len = ints(a[2], "cache_len", &data, B);
    const int *cnt = a[6] == Py_None ? nullptr : ints(a[6], "count", &data, B).data_ptr<int>();
    const c10::DeviceGuard guard(data.device());
    return done(spec_cache4_append(&p, table.data_ptr<int>(), len.data_ptr<int>(), kn.data_ptr(), vn.data_ptr(),
                                   dtype16(kn, "k_new"), stride(kn, 0), stride(kn, 1), stride(kn, 2), cnt, (int)B,
                                   (int)kn.size(1), (int)table.size(1), status(a[7], data), handle(a[8], data)));
    END_HANDLE_TH_ERRORS
}

// (pool, page_table, start, n, page_size, head_dim, count, half, dev_status, stream) -> (k, v)
PyObject *read4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ::count(n, 10);
    const at::Tensor &data = tensor(a[0], "pool");
    const spec_pages4_t p = pool4(a[0], -1, integer(a[4], "page_size"), integer(a[5], "head_dim"));
    const at::Tensor &table = ints(a[1], "page_table", &data, -1, -1);
    const int64_t B = table.size(0), N = small(a[3], "n");
    TORCH_CHECK_VALUE(N >= 1, "n must be at least 1");
    const at::Tensor &start = ints(a[2], "start", &data, B);
    const int *cnt = a[6] == Py_None ? nullptr : ints(a[6], "count", &data, B).data_ptr<int>();
    const int half = PyObject_IsTrue(a[7]);
    if (half < 0) return nullptr;
    const c10::DeviceGuard guard(data.device());
    const auto options = data.options().dtype(half ? at::kHalf : at::kBFloat16);
    std::vector<int64_t> shape = {B, N, p.heads, p.head_dim};
    if (data.dim() == 4) shape.insert(shape.begin(), p.layers);
    const at::Tensor k = at::empty(shape, options), v = at::empty(shape, options);
    const spec_status_t st = spec_cache4_read(
        &p, table.data_ptr<int>(), start.data_ptr<int>(), cnt, k.data_ptr(), v.data_ptr(),
        half ? SPEC_DTYPE_F16 : SPEC_DTYPE_BF16, (int)B, (int)N, (int)table.size(1), status(a[8], data),
        handle(a[9], data));
    if (st != SPEC_OK) return done(st);
    return pair(k, v);
    END_HANDLE_TH_ERRORS
}

// (pool, page_table, cache_len, out_nodes, accept_len, page_size, head_dim, new_len, nodes, dev_status, stream)
PyObject *commit4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ::count(n, 11);
    const at::Tensor &data = tensor(a[0], "pool");
    const spec_pages4_t p = pool4(a[0], 1, integer(a[5], "page_size"), integer(a[6], "head_dim"));
    const at::Tensor &table = ints(a[1], "page_table", &data, -1, -1);
    const int64_t B = table.size(0);
    const at::Tensor &len = ints(a[2], "cache_len", &data, B);
    const int *out = nullptr;
    int N;
    if (a[3] != Py_None) {
        const at::Tensor &t = ints(a[3], "out_nodes", &data, B, -1);
        out = t.data_ptr<int>();
        N = (int)t.size(1);
    } else {
        TORCH_CHECK_VALUE(a[8] != Py_None, "linear drafts need their number of nodes");
        N = small(a[8], "nodes");
    }
    const at::Tensor &acc = ints(a[4], "accept_len", &data, B), &fresh = ints(a[7], "new_len", &data, B);
    const c10::DeviceGuard guard(data.device());
    return done(spec_cache4_commit(&p, table.data_ptr<int>(), len.data_ptr<int>(), out, acc.data_ptr<int>(),
                                   fresh.data_ptr<int>(), (int)B, N, (int)table.size(1), status(a[9], data),
                                   handle(a[10], data)));
    END_HANDLE_TH_ERRORS
}

// (pool, src_pages, dst_pages, page_size, head_dim, dev_status, stream)
PyObject *copy4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const at::Tensor &data = tensor(a[0], "pool");
    const spec_pages4_t p = pool4(a[0], 1, integer(a[3], "page_size"), integer(a[4], "head_dim"));
    const at::Tensor &src = ints(a[1], "src_pages", &data, -1), &dst = ints(a[2], "dst_pages", &data, src.size(0));
    TORCH_CHECK_VALUE(src.size(0) <= INT_MAX, "too many pages");
    const c10::DeviceGuard guard(data.device());
    return done(spec_cache4_copy(&p, src.data_ptr<int>(), dst.data_ptr<int>(), (int)src.size(0), status(a[5], data),
                                 handle(a[6], data)));
    END_HANDLE_TH_ERRORS
}

// (pool, page_table, page_count, page_ref, cache_len, src, dst, page_size, head_dim, workspace, dev_status, stream)
PyObject *fork4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12);
    const at::Tensor &data = tensor(a[0], "pool");
    const spec_pages4_t p = pool4(a[0], 1, integer(a[7], "page_size"), integer(a[8], "head_dim"));
    const at::Tensor &table = ints(a[1], "page_table", &data, -1, -1);
    const int64_t S = table.size(0);
    const at::Tensor &held = ints(a[2], "page_count", &data, S), &ref = ints(a[3], "page_ref", &data, p.num_pages),
                     &len = ints(a[4], "cache_len", &data, S), &src = ints(a[5], "src", &data, -1),
                     &dst = ints(a[6], "dst", &data, src.size(0));
    const c10::DeviceGuard guard(data.device());
    const at::Tensor ws =
        workspace(a[9], data, spec_cache_fork_workspace_bytes((int)std::min<int64_t>(src.size(0), INT_MAX)));
    return done(spec_cache4_fork(&p, table.data_ptr<int>(), held.data_ptr<int>(), ref.data_ptr<int>(),
                                 len.data_ptr<int>(), src.data_ptr<int>(), dst.data_ptr<int>(), (int)src.size(0),
                                 (int)S, (int)table.size(1), ws.data_ptr(), (size_t)ws.nbytes(), status(a[10], data),
                                 handle(a[11], data)));
    END_HANDLE_TH_ERRORS
}

// Bounds of pages, [num_pages, heads, 2, head_dim] contiguous.
const at::Tensor &bounds_of(PyObject *o, const at::Tensor &with, int64_t pages, int64_t heads, int64_t D) {
    const at::Tensor &t = tensor(o, "bounds");
    dtype16(t, "bounds");
    TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous() && t.dim() == 4 && (pages < 0 || t.size(0) == pages) &&
                          (heads < 0 || t.size(1) == heads) && t.size(2) == 2 && (D < 0 || t.size(3) == D),
                      "bounds must be a contiguous CUDA tensor [num_pages, kv_heads, 2, head_dim]");
    together(t, with, "bounds");
    no_gradient(t, "bounds");
    return t;
}

// (k, bounds, page_table, cache_len, start, dev_status, stream)
PyObject *bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const spec_pages_t p = pool(a[0], a[0], false);
    const at::Tensor &k = tensor(a[0], "k"), &to = bounds_of(a[1], k, p.num_pages, p.heads, p.head_dim);
    TORCH_CHECK_VALUE(to.scalar_type() == k.scalar_type(), "bounds must be of the cache's dtype");
    const at::Tensor &table = ints(a[2], "page_table", &k, -1, -1);
    const int64_t B = table.size(0);
    const at::Tensor &len = ints(a[3], "cache_len", &k, B);
    const int *start = a[4] == Py_None ? nullptr : ints(a[4], "start", &k, B).data_ptr<int>();
    const c10::DeviceGuard guard(k.device());
    return done(spec_cache_bounds(&p, table.data_ptr<int>(), start, len.data_ptr<int>(), to.data_ptr(), (int)B,
                                  (int)table.size(1), status(a[5], k), handle(a[6], k)));
    END_HANDLE_TH_ERRORS
}

// (pool, bounds, page_table, cache_len, page_size, start, dev_status, stream)
PyObject *bounds4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const at::Tensor &data = tensor(a[0], "pool"), &to = bounds_of(a[1], data, -1, -1, -1);
    const spec_pages4_t p = pool4(a[0], 0, integer(a[4], "page_size"), to.size(3));
    bounds_of(a[1], data, p.num_pages, p.heads, p.head_dim);
    const at::Tensor &table = ints(a[2], "page_table", &data, -1, -1);
    const int64_t B = table.size(0);
    const at::Tensor &len = ints(a[3], "cache_len", &data, B);
    const int *start = a[5] == Py_None ? nullptr : ints(a[5], "start", &data, B).data_ptr<int>();
    const c10::DeviceGuard guard(data.device());
    return done(spec_cache4_bounds(&p, table.data_ptr<int>(), start, len.data_ptr<int>(), to.data_ptr(),
                                   dtype16(to, "bounds"), (int)B, (int)table.size(1), status(a[6], data),
                                   handle(a[7], data)));
    END_HANDLE_TH_ERRORS
}

// (q, bounds, page_table, cache_len, page_size, node_count, out, dev_status, stream) -> scores
PyObject *scores(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 9);
    const at::Tensor &from = tensor(a[1], "bounds"), &q = rows16(a[0], "q", from, -1);
    bounds_of(a[1], q, -1, -1, q.size(3));
    TORCH_CHECK_VALUE(q.scalar_type() == from.scalar_type(), "q and bounds must be of one dtype");
    TORCH_CHECK_VALUE(from.size(0) <= INT_MAX && from.size(1) <= INT_MAX, "bounds are too large");
    const int64_t B = q.size(0), H = from.size(1);
    const at::Tensor &table = ints(a[2], "page_table", &q, B, -1), &len = ints(a[3], "cache_len", &q, B);
    const int *nodes = a[5] == Py_None ? nullptr : ints(a[5], "node_count", &q, B).data_ptr<int>();
    const c10::DeviceGuard guard(q.device());
    at::Tensor out;
    if (a[6] != Py_None) {
        out = tensor(a[6], "out");
        TORCH_CHECK_VALUE(out.sizes() == at::IntArrayRef({B, H, table.size(1)}) && out.scalar_type() == at::kFloat &&
                              out.is_cuda() && out.is_contiguous() && out.device() == q.device(),
                          "out must be a contiguous float32 CUDA tensor [B, kv_heads, max_pages]");
        no_gradient(out, "out");
    } else {
        out = at::empty({B, H, table.size(1)}, q.options().dtype(at::kFloat));
    }
    const spec_status_t st = spec_page_scores(
        q.data_ptr(), dtype16(q, "q"), stride(q, 0), stride(q, 1), stride(q, 2), from.data_ptr(), table.data_ptr<int>(),
        len.data_ptr<int>(), nodes, out.data_ptr<float>(), (int)B, (int)q.size(1), (int)q.size(2), (int)H,
        (int)q.size(3), (int)table.size(1), (int)from.size(0), small(a[4], "page_size"), status(a[7], q),
        handle(a[8], q));
    return st == SPEC_OK ? THPVariable_Wrap(out) : done(st);
    END_HANDLE_TH_ERRORS
}

// (scores, page_table, cache_len, page_size, keep, first, recent, extra, dev_status, stream) -> (table, len)
PyObject *select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const at::Tensor &from = tensor(a[0], "scores");
    TORCH_CHECK_VALUE(from.dim() == 3 && from.scalar_type() == at::kFloat && from.is_cuda() && from.is_contiguous(),
                      "scores must be a contiguous float32 CUDA tensor [B, kv_heads, max_pages]");
    no_gradient(from, "scores");
    const int64_t B = from.size(0), H = from.size(1), P = from.size(2);
    TORCH_CHECK_VALUE(B <= INT_MAX && H <= INT_MAX && P <= INT_MAX, "scores are too large");
    const at::Tensor &table = ints(a[1], "page_table", &from, B, P), &len = ints(a[2], "cache_len", &from, B);
    const int page = small(a[3], "page_size"), keep = small(a[4], "keep"), extra = small(a[7], "extra");
    TORCH_CHECK_VALUE(page >= 8 && keep >= 1 && keep <= SPEC_MAX_SELECT && extra >= 0 && extra <= (1 << 20),
                      "page_size must be at least 8, keep 1 to ", SPEC_MAX_SELECT, ", extra 0 to ", 1 << 20);
    const c10::DeviceGuard guard(from.device());
    const at::Tensor out = at::empty({B, H, keep + ((int64_t)extra + page - 1) / page}, table.options()),
                     kept = at::empty({B}, table.options());
    const spec_status_t st = spec_page_select(
        from.data_ptr<float>(), table.data_ptr<int>(), len.data_ptr<int>(), out.data_ptr<int>(), kept.data_ptr<int>(),
        (int)B, (int)H, (int)P, page, keep, small(a[5], "first"), small(a[6], "recent"), extra, status(a[8], from),
        handle(a[9], from));
    return st == SPEC_OK ? pair(out, kept) : done(st);
    END_HANDLE_TH_ERRORS
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(resize), ENTRY(fork), ENTRY(copy), ENTRY(append), ENTRY(commit),
                         ENTRY(tree_attention), ENTRY(tree_attention4), ENTRY(append4), ENTRY(read4), ENTRY(commit4),
                         ENTRY(copy4), ENTRY(fork4), ENTRY(bounds), ENTRY(bounds4), ENTRY(scores), ENTRY(select),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
