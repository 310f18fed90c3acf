"""Paged key/value cache and tree attention (include/spec_cache.h).

A step of a model that verifies drafted trees:

    cache = PagedCache(layers, num_pages, page_size, kv_heads, head_dim, slots, max_pages)
    cache.reserve(N)                                  # pages for the drafted tokens
    for layer in range(layers):
        cache.append(layer, k_new, v_new)             # [slots, N, kv_heads, head_dim]
        o = cache.attention(layer, q, parent)         # [slots, N, q_heads, head_dim]
    out_tokens, out_nodes, accept_len = verify_tree(...)
    cache.commit(out_nodes, accept_len)               # accepted nodes behind the root
    cache.trim()                                      # pages past the new lengths returned

The functions below the class are the same operators on plain tensors.  Pools
of pages are [num_pages, page_size, kv_heads, head_dim] (one layer) or [layers,
num_pages, ...] tensors of any strides that leave head_dim contiguous; a pool
stored heads first is passed as its transpose.  As everywhere in this package
every step runs in the library's kernels, on torch's current stream or the
`stream` given, and nothing falls back to torch.
"""
import ctypes
import functools
import math
import struct

import torch

DEV_BAD_PAGE, DEV_NO_PAGES, DEV_BAD_SLOT = 16, 32, 64
DTYPE_F16 = 2
MAX_SLOTS, MAX_TREE, MAX_HEAD_DIM = 8192, 64, 128

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: DTYPE_F16}


# spec_pages_t: k, v, dtype, layers, num_pages, page_size, heads, head_dim, and
# the strides of layers, pages, tokens and heads
_PAGES = struct.Struct("PPiiiiiiqqqq")


def declare(L):
    """argtypes of the entry points of include/spec_cache.h."""
    vp, i, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    L.spec_cache_resize.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp]
    L.spec_cache_fork_workspace_bytes.argtypes = [i]
    L.spec_cache_fork_workspace_bytes.restype = sz
    L.spec_cache_fork.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, vp, sz, vp, vp]
    L.spec_cache_copy.argtypes = [vp, vp, vp, i, vp, vp]
    L.spec_cache_append.argtypes = [vp, vp, vp, vp, vp, ll, ll, ll, vp, i, i, i, vp, vp]
    L.spec_cache_commit.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, vp, vp]
    L.spec_tree_attention_workspace_bytes.argtypes = [i] * 5
    L.spec_tree_attention_workspace_bytes.restype = sz
    L.spec_tree_attention.argtypes = [vp, ll, ll, ll, vp, vp, vp, vp, vp, i, i, i, i, ctypes.c_float, i, i,
                                      vp, vp, vp, sz, vp, vp]
    for name in ("resize", "fork", "copy", "append", "commit"):
        getattr(L, "spec_cache_" + name).restype = i
    L.spec_tree_attention.restype = i


EXPORTED = ["spec_cache_resize", "spec_cache_fork_workspace_bytes", "spec_cache_fork", "spec_cache_copy",
            "spec_cache_append", "spec_cache_commit", "spec_tree_attention_workspace_bytes",
            "spec_tree_attention"]


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import load_library
        _loaded = load_library()
    return _loaded


def _check(status):
    if status != 0:
        from . import SpecVerifyError
        raise SpecVerifyError("%s (%d)" % (_lib().spec_status_str(status).decode(), status))


# The handle of torch's current stream on a device, without the Python object
# that torch.cuda.current_stream makes around it (3 us a call).
_current_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream, t):
    return _current_stream(t.get_device()) if stream is None else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(shape, strides, step):
    """Strides of a tensor's dimensions; a dimension of one element is never
    stepped over, so its stride is any valid one."""
    return [st if n > 1 else step for n, st in zip(shape, strides)] if 1 in shape else strides


def _pages(k, v, layered):
    """spec_pages_t of a pool, and its shape."""
    sh, st = k.shape, k.stride()
    if len(sh) != (5 if layered else 4) or v.shape != sh or v.dtype is not k.dtype:
        raise ValueError("k and v must be alike, [%snum_pages, page_size, kv_heads, head_dim]"
                         % ("layers, " if layered else ""))
    code = _CODES.get(k.dtype)
    if code is None:
        raise TypeError("a cache is bfloat16, float16 or float32, got %s" % k.dtype)
    if not k.is_cuda or not v.is_cuda:
        raise ValueError("k and v must be CUDA tensors")
    other = v.stride()
    if 1 in sh:
        st, other = _strides(sh, st, sh[-1]), _strides(sh, other, sh[-1])
    if st != other or k.stride(-1) != 1:
        raise ValueError("k and v need the same strides and a contiguous head_dim")
    n, page, heads, dim = sh[-4:]
    if layered:
        return _PAGES.pack(k.data_ptr(), v.data_ptr(), code, sh[0], n, page, heads, dim, *st[:4]), sh
    return _PAGES.pack(k.data_ptr(), v.data_ptr(), code, 1, n, page, heads, dim, 0, *st[:3]), sh


_I32 = torch.int32


def _ints(name, t, shape):
    """An int32 CUDA tensor, contiguous, of this shape."""
    if t.dtype is not _I32 or not t.is_cuda or not t.is_contiguous() or t.shape != shape:
        raise ValueError("%s must be a contiguous int32 CUDA tensor %s" % (name, list(shape)))


def _table(t, slots=None):
    if (t.dtype is not _I32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 2
            or (slots is not None and t.shape[0] != slots)):
        raise ValueError("page_table must be a contiguous int32 CUDA tensor [%s, max_pages]"
                         % ("slots" if slots is None else slots))
    return t.shape


_scratch = {}


def _workspace(n, t, handle, stream):
    """Scratch that one stream's calls share: they never overlap."""
    key = (t.get_device(), handle)
    ws = _scratch.get(key)
    if ws is None or ws.numel() < n:
        if stream is None:
            ws = torch.empty(n, dtype=torch.uint8, device=t.device)
        else:
            with torch.cuda.stream(stream):
                ws = torch.empty(n, dtype=torch.uint8, device=t.device)
        _scratch[key] = ws
    return ws


@functools.lru_cache(maxsize=4096)
def _attention_bytes(B, N, Hq, heads, D):
    return max(256, _lib().spec_tree_attention_workspace_bytes(B, N, Hq, heads, D))


def cache_resize(page_table, page_count, page_ref, want_len, page_size, *, extra=0, dev_status=None, stream=None):
    """Pages for want_len + extra tokens per slot (spec_cache_resize): the pages
    past that given back, then the missing ones taken, lowest free page first.
    page_table int32 [slots, max_pages], page_count [slots] and page_ref
    [num_pages] are updated; want_len int32 [slots], negative: left as it is."""
    B, P = _table(page_table)
    _ints("page_count", page_count, (B,))
    _ints("want_len", want_len, (B,))
    pages = page_ref.numel()
    _ints("page_ref", page_ref, (pages,))
    _check(_lib().spec_cache_resize(page_table.data_ptr(), page_count.data_ptr(), page_ref.data_ptr(),
                                    want_len.data_ptr(), extra, page_size, B, P, pages, _ptr(dev_status),
                                    _stream(stream, page_table)))


def cache_fork(k, v, page_table, page_count, page_ref, cache_len, src, dst, *, dev_status=None, stream=None):
    """Slots dst (int32 [F]) continued from slots src (spec_cache_fork): full
    pages shared, the last partial page copied in every layer.  k, v [layers,
    num_pages, page_size, kv_heads, head_dim]; page_table, page_count, page_ref
    and cache_len are updated."""
    pages, shape = _pages(k, v, True)
    S, P = _table(page_table)
    _ints("page_count", page_count, (S,))
    _ints("cache_len", cache_len, (S,))
    _ints("page_ref", page_ref, (shape[1],))
    F = src.numel()
    _ints("src", src, (F,))
    _ints("dst", dst, (F,))
    handle = _stream(stream, k)
    ws = _workspace(max(256, _lib().spec_cache_fork_workspace_bytes(F)), k, handle, stream)
    _check(_lib().spec_cache_fork(pages, page_table.data_ptr(), page_count.data_ptr(), page_ref.data_ptr(),
                                  cache_len.data_ptr(), src.data_ptr(), dst.data_ptr(), F, S, P, ws.data_ptr(),
                                  ws.numel(), _ptr(dev_status), handle))


def cache_copy(k, v, src_pages, dst_pages, *, dev_status=None, stream=None):
    """Whole pages copied in every layer (spec_cache_copy): k, v [layers,
    num_pages, ...], src_pages and dst_pages int32 [n]."""
    pages, _ = _pages(k, v, True)
    n = src_pages.numel()
    _ints("src_pages", src_pages, (n,))
    _ints("dst_pages", dst_pages, (n,))
    _check(_lib().spec_cache_copy(pages, src_pages.data_ptr(), dst_pages.data_ptr(), n, _ptr(dev_status),
                                  _stream(stream, k)))


def _rows(name, t, like, last, heads=None):
    """Shape and strides of a [B, N, heads, head_dim] tensor of the cache's dtype."""
    sh = t.shape
    if (len(sh) != 4 or t.dtype is not like.dtype or not t.is_cuda or sh[3] != last or t.stride(3) != 1
            or (heads is not None and sh[2] != heads)):
        raise ValueError("%s must be a CUDA tensor [B, N, %s, %d] of the cache's dtype, its last dimension contiguous"
                         % (name, "heads" if heads is None else heads, last))
    return sh, _strides(sh, t.stride(), last)


def cache_append(k, v, page_table, cache_len, k_new, v_new, *, count=None, dev_status=None, stream=None):
    """New keys and values of one layer written behind the committed positions
    (spec_cache_append): k, v [num_pages, page_size, kv_heads, head_dim];
    k_new, v_new [B, N, kv_heads, head_dim] of equal strides; count int32 [B]
    tokens of each request, None: all N.  cache_len is not changed."""
    pages, shape = _pages(k, v, False)
    new = _rows("k_new", k_new, k, shape[3], shape[2])
    if _rows("v_new", v_new, k, shape[3], shape[2]) != new:
        raise ValueError("k_new and v_new need the same shape and strides")
    (B, N, _, _), st = new
    _, P = _table(page_table, B)
    _ints("cache_len", cache_len, (B,))
    if count is not None:
        _ints("count", count, (B,))
    _check(_lib().spec_cache_append(pages, page_table.data_ptr(), cache_len.data_ptr(), k_new.data_ptr(),
                                    v_new.data_ptr(), st[0], st[1], st[2], _ptr(count), B, N, P, _ptr(dev_status),
                                    _stream(stream, k)))


def cache_commit(k, v, page_table, cache_len, out_nodes, accept_len, *, new_len=None, nodes=None, dev_status=None,
                 stream=None):
    """The accepted path of every tree moved behind its root in every layer and
    the lengths advanced (spec_cache_commit): k, v [layers, num_pages, ...];
    out_nodes int32 [B, N] and accept_len int32 [B] as verify_tree returns them.
    out_nodes None: linear drafts (nodes: their number with the root), whose
    accepted tokens lie in place.  new_len int32 [B] receives the lengths; None:
    cache_len itself is updated.  Returns the tensor that holds them."""
    pages, _ = _pages(k, v, True)
    B, P = _table(page_table)
    if out_nodes is not None:
        nodes = out_nodes.shape[-1]
        _ints("out_nodes", out_nodes, (B, nodes))
    elif nodes is None:
        raise ValueError("linear drafts need their number of nodes")
    _ints("cache_len", cache_len, (B,))
    _ints("accept_len", accept_len, (B,))
    if new_len is None:
        new_len = cache_len
    else:
        _ints("new_len", new_len, (B,))
    _check(_lib().spec_cache_commit(pages, page_table.data_ptr(), cache_len.data_ptr(), _ptr(out_nodes),
                                    accept_len.data_ptr(), new_len.data_ptr(), B, nodes, P, _ptr(dev_status),
                                    _stream(stream, k)))
    return new_len


def tree_attention(q, k, v, page_table, cache_len, parent=None, *, node_count=None, scale=None, window=0, sinks=0,
                   out=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """Attention of drafted trees over one layer of a paged cache
    (spec_tree_attention): q [B, N, q_heads, head_dim], k, v [num_pages,
    page_size, kv_heads, head_dim], bfloat16 or float16; parent int32 [B, N]
    (None: chains, N = 1 being the decoding of single tokens); node n of request
    b sees the positions [0, cache_len[b]), its ancestors and itself, with a
    window only the last `window` of them along its path and the first `sinks`
    tokens.  Returns out [B, N, q_heads, head_dim], with return_lse also the log
    of the softmax sums, float32 [B, N, q_heads]."""
    pages, shape = _pages(k, v, False)
    qshape, st = _rows("q", q, k, shape[3])
    B, N, Hq, D = qshape
    _, P = _table(page_table, B)
    _ints("cache_len", cache_len, (B,))
    if parent is not None:
        _ints("parent", parent, (B, N))
    if node_count is not None:
        _ints("node_count", node_count, (B,))
    handle = _stream(stream, q)
    if out is not None and (out.shape != qshape or out.dtype is not q.dtype or not out.is_cuda
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous CUDA tensor of q's shape and dtype")
    if stream is None:
        out, lse = _outputs(q, qshape, out, return_lse)
    else:
        with torch.cuda.stream(stream):
            out, lse = _outputs(q, qshape, out, return_lse)
    if workspace is None:
        workspace = _workspace(_attention_bytes(B, N, Hq, shape[2], D), q, handle, stream)
    _check(_lib().spec_tree_attention(q.data_ptr(), st[0], st[1], st[2], pages, page_table.data_ptr(),
                                      cache_len.data_ptr(), _ptr(parent), _ptr(node_count), B, N, Hq, P,
                                      1.0 / math.sqrt(D) if scale is None else scale, window, sinks, out.data_ptr(),
                                      _ptr(lse), workspace.data_ptr(), workspace.numel(), _ptr(dev_status), handle))
    return (out, lse) if return_lse else out


def _outputs(q, shape, out, return_lse):
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    return out, torch.empty(shape[:3], dtype=torch.float32, device=q.device) if return_lse else None


class PagedCache:
    """The cache of a batch of `slots` requests: pools of pages for every layer,
    the page table, the lengths, and the status word the calls report in."""

    def __init__(self, layers, num_pages, page_size, kv_heads, head_dim, slots, max_pages, *,
                 dtype=torch.bfloat16, device="cuda"):
        shape = (layers, num_pages, page_size, kv_heads, head_dim)
        self.page_size = page_size
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self._layers = list(zip(self.k.unbind(0), self.v.unbind(0)))
        i32 = dict(dtype=torch.int32, device=device)
        self.page_table = torch.full((slots, max_pages), -1, **i32)
        self.page_count = torch.zeros((slots,), **i32)
        self.page_ref = torch.zeros((num_pages,), **i32)
        self.cache_len = torch.zeros((slots,), **i32)
        self.status = torch.zeros((1,), **i32)

    def reserve(self, tokens, stream=None):
        """Room for `tokens` more tokens in every slot."""
        cache_resize(self.page_table, self.page_count, self.page_ref, self.cache_len, self.page_size, extra=tokens,
                     dev_status=self.status, stream=stream)

    def trim(self, stream=None):
        """The pages past every slot's length given back."""
        self.reserve(0, stream=stream)

    def append(self, layer, k_new, v_new, count=None, stream=None):
        k, v = self._layers[layer]
        cache_append(k, v, self.page_table, self.cache_len, k_new, v_new, count=count,
                     dev_status=self.status, stream=stream)

    def attention(self, layer, q, parent=None, **kw):
        k, v = self._layers[layer]
        return tree_attention(q, k, v, self.page_table, self.cache_len, parent, dev_status=self.status, **kw)

    def commit(self, out_nodes, accept_len, nodes=None, stream=None):
        cache_commit(self.k, self.v, self.page_table, self.cache_len, out_nodes, accept_len, nodes=nodes,
                     dev_status=self.status, stream=stream)

    def fork(self, src, dst, stream=None):
        cache_fork(self.k, self.v, self.page_table, self.page_count, self.page_ref, self.cache_len, src, dst,
                   dev_status=self.status, stream=stream)
