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

// (q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out, return_lse, workspace,
//  dev_status, stream) -> out, or (out, lse)
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 15);
    const spec_pages_t p = pool(a[1], a[2], false);
    const at::Tensor &k = tensor(a[1], "k"), &q = rows(a[0], "q", k, -1);
    const int64_t B = q.size(0), N = q.size(1), Hq = q.size(2), D = q.size(3);
    const at::Tensor &table = ints(a[3], "page_table", &k, B, -1), &len = ints(a[4], "cache_len", &k, B);
    const int *parent = a[5] == Py_None ? nullptr : ints(a[5], "parent", &k, B, N).data_ptr<int>();
    const int *nodes = a[6] == Py_None ? nullptr : ints(a[6], "node_count", &k, B).data_ptr<int>();
    double scale = 1.0 / std::sqrt((double)D);
    if (a[7] != Py_None) {
        scale = PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred()) return nullptr;
    }
    const int window = small(a[8], "window"), sinks = small(a[9], "sinks");
    at::Tensor out, lse;
    if (a[10] != Py_None) {
        out = tensor(a[10], "out");
        TORCH_CHECK_VALUE(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() && out.is_cuda() &&
                              out.is_contiguous() && out.device() == q.device(),
                          "out must be a contiguous CUDA tensor of q's shape and dtype");
        no_gradient(out, "out");
    } else {
        out = at::empty(q.sizes(), q.options());
    }
    const int with_lse = PyObject_IsTrue(a[11]);
    if (with_lse < 0) return nullptr;
    if (with_lse) lse = at::empty({B, N, Hq}, q.options().dtype(at::kFloat));
    const c10::DeviceGuard guard(q.device());
    const at::Tensor ws =
        workspace(a[12], k, spec_tree_attention_workspace_bytes((int)B, (int)N, (int)Hq, p.heads, (int)D));
    const spec_status_t st = spec_tree_attention(
        q.data_ptr(), stride(q, 0), stride(q, 1), stride(q, 2), &p, table.data_ptr<int>(), len.data_ptr<int>(),
        parent, nodes, (int)B, (int)N, (int)Hq, (int)table.size(1), (float)scale, window, sinks, out.data_ptr(),
        with_lse ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), (size_t)ws.nbytes(),
        status(a[13], k), handle(a[14], k));
    if (st != SPEC_OK) return done(st);
    PyObject *o = THPVariable_Wrap(out);
    if (!with_lse || !o) return o;
    PyObject *l = THPVariable_Wrap(lse);
    PyObject *both = l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_DECREF(o);
    Py_XDECREF(l);
    return both;
    END_HANDLE_TH_ERRORS
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(resize), ENTRY(fork), ENTRY(copy), ENTRY(append), ENTRY(commit),
                         ENTRY(tree_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
