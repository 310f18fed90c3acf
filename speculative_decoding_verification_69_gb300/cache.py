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
`stream` given, and nothing falls back to torch.  The calls can be captured in a
CUDA graph: a call without a `workspace` (a uint8 tensor, 256-byte aligned) takes
one from torch's allocator, in a capture from the graph's own memory.  Nothing here
has a backward pass: with gradients enabled, tensors that require one are refused.
"""
import ctypes
import importlib.util
import subprocess

import torch

from . import _build

DEV_BAD_PAGE, DEV_NO_PAGES, DEV_BAD_SLOT = 16, 32, 64
DTYPE_F16 = 2


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


def _native():
    """The compiled binding (csrc/binding.cpp), which checks its arguments; built
    first if it is missing or stale."""
    global _loaded
    if _loaded is None:
        from . import SpecVerifyError, load_library
        load_library()
        try:
            path = _build.build_binding()
        except (OSError, subprocess.CalledProcessError) as e:
            raise SpecVerifyError("the binding of the paged cache is not built, and building it failed: %s" % e) from e
        spec = importlib.util.spec_from_file_location("_native", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _loaded = module
    return _loaded


def _handle(stream):
    return None if stream is None else stream.cuda_stream  # None: torch's current stream


def cache_resize(page_table, page_count, page_ref, want_len, page_size, *, extra=0, dev_status=None, stream=None):
    """Pages for want_len + extra tokens per slot (spec_cache_resize): the pages
    past that given back, then the missing ones taken, lowest free page first.
    page_table int32 [slots, max_pages], page_count [slots] and page_ref
    [num_pages] are updated; want_len int32 [slots], negative: left as it is."""
    _native().resize(page_table, page_count, page_ref, want_len, page_size, extra, dev_status,
                     _handle(stream))


def cache_fork(k, v, page_table, page_count, page_ref, cache_len, src, dst, *, workspace=None, dev_status=None,
               stream=None):
    """Slots dst (int32 [F]) continued from slots src (spec_cache_fork): full
    pages shared, the last partial page copied in every layer.  k, v [layers,
    num_pages, page_size, kv_heads, head_dim]; page_table, page_count, page_ref
    and cache_len are updated."""
    args = (k, v, page_table, page_count, page_ref, cache_len, src, dst, workspace, dev_status, None)
    if stream is None:
        _native().fork(*args)
    else:
        with torch.cuda.stream(stream):  # a workspace of the call's own belongs to that stream
            _native().fork(*args)


def cache_copy(k, v, src_pages, dst_pages, *, dev_status=None, stream=None):
    """Whole pages copied in every layer (spec_cache_copy): k, v [layers,
    num_pages, ...], src_pages and dst_pages int32 [n]."""
    _native().copy(k, v, src_pages, dst_pages, dev_status, _handle(stream))


def cache_append(k, v, page_table, cache_len, k_new, v_new, *, count=None, dev_status=None, stream=None):
    """New keys and values of one layer written behind the committed positions
    (spec_cache_append): k, v [num_pages, page_size, kv_heads, head_dim];
    k_new, v_new [B, N, kv_heads, head_dim] of equal strides; count int32 [B]
    tokens of each request, None: all N.  cache_len is not changed."""
    _native().append(k, v, page_table, cache_len, k_new, v_new, count, dev_status, _handle(stream))


def cache_commit(k, v, page_table, cache_len, out_nodes, accept_len, *, new_len=None, nodes=None, dev_status=None,
                 stream=None):
    """The accepted path of every tree moved behind its root in every layer and
    the lengths advanced (spec_cache_commit): k, v [layers, num_pages, ...];
    out_nodes int32 [B, N] and accept_len int32 [B] as verify_tree returns them.
    out_nodes None: linear drafts (nodes: their number with the root), whose
    accepted tokens lie in place.  new_len int32 [B] receives the lengths; None:
    cache_len itself is updated.  Returns the tensor that holds them."""
    if new_len is None:
        new_len = cache_len
    _native().commit(k, v, page_table, cache_len, out_nodes, accept_len, new_len, nodes, dev_status,
                     _handle(stream))
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
    if stream is None:
        return _native().tree_attention(q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out,
                                        return_lse, workspace, dev_status, None)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().tree_attention(q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out,
                                        return_lse, workspace, dev_status, None)


class PagedCache:
    """The cache of a batch of `slots` requests: pools of pages for every layer,
    the page table, the lengths, and the status word the calls report in.  The
    methods work on all slots; single slots are filled, kept or released with
    cache_resize and want_len (0: released, negative: left alone).  dtype:
    bfloat16 or float16, or float32 for the pages alone (attention refuses it)."""

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

    def fork(self, src, dst, workspace=None, stream=None):
        cache_fork(self.k, self.v, self.page_table, self.page_count, self.page_ref, self.cache_len, src, dst,
                   workspace=workspace, dev_status=self.status, stream=stream)
