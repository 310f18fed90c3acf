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

A long cache that is read once per token, as a drafter's, can be made cheap in two
ways.  PagedCache4 holds it in 4 bits: the same methods, its attention called
tree_attention4.  Attention over selected pages reads only the pages that a
cheap score picks, of either cache:

    bounds = cache.new_bounds()                       # of one layer
    cache.append(layer, k_new, v_new)
    pages = cache.select(layer, q, bounds, keep=64, start=start)
    o = cache.attention(layer, q, parent, pages=pages)

`start` int32 [slots]: the lengths up to which the bounds have been formed (None:
not at all); the pages that hold positions from there on are summarised first.
"""
import ctypes
import importlib.util
import subprocess

import torch

from . import _build

DEV_BAD_PAGE, DEV_NO_PAGES, DEV_BAD_SLOT, DEV_BAD_VALUE = 16, 32, 64, 128
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
    L.spec_sparse_attention.argtypes = L.spec_tree_attention.argtypes
    L.spec_cache4_page_bytes.argtypes = [i, i]
    L.spec_cache4_page_bytes.restype = sz
    L.spec_cache4_append.argtypes = [vp, vp, vp, vp, vp, i, ll, ll, ll, vp, i, i, i, vp, vp]
    L.spec_cache4_read.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, vp, vp]
    L.spec_cache4_commit.argtypes = L.spec_cache_commit.argtypes
    L.spec_cache4_copy.argtypes = L.spec_cache_copy.argtypes
    L.spec_cache4_fork.argtypes = L.spec_cache_fork.argtypes
    L.spec_tree_attention4_workspace_bytes.argtypes = [i] * 5
    L.spec_tree_attention4_workspace_bytes.restype = sz
    L.spec_tree_attention4.argtypes = [vp, i, ll, ll, ll, vp, vp, i, vp, vp, vp, i, i, i, i, ctypes.c_float, i, i,
                                       vp, vp, vp, sz, vp, vp]
    L.spec_cache_bounds.argtypes = [vp, vp, vp, vp, vp, i, i, vp, vp]
    L.spec_cache4_bounds.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, vp]
    L.spec_page_scores.argtypes = [vp, i, ll, ll, ll, vp, vp, vp, vp, vp] + [i] * 8 + [vp, vp]
    L.spec_page_select.argtypes = [vp] * 5 + [i] * 8 + [vp, vp]
    for name in EXPORTED:
        if not name.endswith("_bytes"):
            getattr(L, name).restype = i


EXPORTED = ["spec_cache_resize", "spec_cache_fork_workspace_bytes", "spec_cache_fork", "spec_cache_copy",
            "spec_cache_append", "spec_cache_commit", "spec_tree_attention_workspace_bytes",
            "spec_tree_attention", "spec_sparse_attention", "spec_cache4_page_bytes", "spec_cache4_append",
            "spec_cache4_read", "spec_cache4_commit", "spec_cache4_copy", "spec_cache4_fork",
            "spec_tree_attention4_workspace_bytes", "spec_tree_attention4", "spec_cache_bounds", "spec_cache4_bounds",
            "spec_page_scores", "spec_page_select"]


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
    tokens.  page_table [B, max_pages], or [B, kv_heads, max_pages] (with cache_len as
    page_select returns them): a list of pages for every key head, in whose positions
    window and sinks then count, not in the sequence's.  Returns out [B, N, q_heads, head_dim], with
    return_lse also the log of the softmax sums, float32 [B, N, q_heads]."""
    if stream is None:
        return _native().tree_attention(q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out,
                                        return_lse, workspace, dev_status, None)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().tree_attention(q, k, v, page_table, cache_len, parent, node_count, scale, window, sinks, out,
                                        return_lse, workspace, dev_status, None)


def cache4_page_bytes(page_size, head_dim):
    """Bytes of one page and head of a 4-bit pool (spec_cache4_page_bytes)."""
    from . import load_library
    n = load_library().spec_cache4_page_bytes(page_size, head_dim)
    if n == 0:
        raise ValueError("page_size must be a power of two of at least 8, head_dim a multiple of 8 up to 128")
    return n


def cache4_append(pool, page_table, cache_len, k_new, v_new, page_size, *, count=None, dev_status=None, stream=None):
    """New keys and values of one layer quantised into a 4-bit pool (spec_cache4_append): pool uint8
    [num_pages, kv_heads, cache4_page_bytes(page_size, head_dim)]; the rest as for cache_append,
    k_new and v_new bfloat16 or float16.  A pool's bytes tell neither its page_size nor its head_dim: every call
    has to give it the same ones (PagedCache4 sees to that)."""
    _native().append4(pool, page_table, cache_len, k_new, v_new, page_size, count, dev_status, _handle(stream))


def cache4_read(pool, page_table, start, n, page_size, head_dim, *, count=None, dtype=torch.bfloat16, dev_status=None,
                stream=None):
    """The numbers that a 4-bit pool stands for (spec_cache4_read): positions start[b] + i, i < count[b] (None: n)
    of every request b.  start and count int32 [B].  Returns k and v [B, n, kv_heads, head_dim], for a pool
    [layers, num_pages, ...] with the layers in front; rows from count[b] on are 0."""
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("the numbers come as bfloat16 or float16")
    args = (pool, page_table, start, n, page_size, head_dim, count, dtype == torch.float16, dev_status, None)
    if stream is None:
        return _native().read4(*args)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().read4(*args)


def cache4_commit(pool, page_table, cache_len, out_nodes, accept_len, page_size, head_dim, *, new_len=None, nodes=None,
                  dev_status=None, stream=None):
    """cache_commit for a 4-bit pool [layers, num_pages, ...] (spec_cache4_commit)."""
    if new_len is None:
        new_len = cache_len
    _native().commit4(pool, page_table, cache_len, out_nodes, accept_len, page_size, head_dim, new_len, nodes,
                      dev_status, _handle(stream))
    return new_len


def cache4_copy(pool, src_pages, dst_pages, page_size, head_dim, *, dev_status=None, stream=None):
    """cache_copy for a 4-bit pool [layers, num_pages, ...] (spec_cache4_copy)."""
    _native().copy4(pool, src_pages, dst_pages, page_size, head_dim, dev_status, _handle(stream))


def cache4_fork(pool, page_table, page_count, page_ref, cache_len, src, dst, page_size, head_dim, *, workspace=None,
                dev_status=None, stream=None):
    """cache_fork for a 4-bit pool [layers, num_pages, ...] (spec_cache4_fork)."""
    args = (pool, page_table, page_count, page_ref, cache_len, src, dst, page_size, head_dim, workspace, dev_status,
            None)
    if stream is None:
        _native().fork4(*args)
    else:
        with torch.cuda.stream(stream):  # a workspace of the call's own belongs to that stream
            _native().fork4(*args)


def tree_attention4(q, pool, page_table, cache_len, page_size, parent=None, *, node_count=None, scale=None, window=0,
                    sinks=0, out=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """tree_attention over one layer of a 4-bit cache (spec_tree_attention4): pool uint8 [num_pages,
    kv_heads, page_bytes], q [B, N, q_heads, head_dim] bfloat16 or float16; all else as there."""
    args = (q, pool, page_table, cache_len, page_size, parent, node_count, scale, window, sinks, out, return_lse,
            workspace, dev_status, None)
    if stream is None:
        return _native().tree_attention4(*args)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().tree_attention4(*args)


def cache_bounds(k, bounds, page_table, cache_len, *, start=None, dev_status=None, stream=None):
    """Smallest and largest key of each channel (spec_cache_bounds) of the pages that hold positions [start[b],
    cache_len[b]): bounds [num_pages, kv_heads, 2, head_dim] of the keys' dtype, updated; k [num_pages,
    page_size, kv_heads, head_dim] bfloat16 or float16, start int32 [B], None: 0."""
    _native().bounds(k, bounds, page_table, cache_len, start, dev_status, _handle(stream))


def cache4_bounds(pool, bounds, page_table, cache_len, page_size, *, start=None, dev_status=None, stream=None):
    """cache_bounds for one layer of a 4-bit pool (spec_cache4_bounds), bounds bfloat16 or float16."""
    _native().bounds4(pool, bounds, page_table, cache_len, page_size, start, dev_status, _handle(stream))


def page_scores(q, bounds, page_table, cache_len, page_size, *, node_count=None, out=None, dev_status=None, stream=None):
    """An upper bound of q . k over every page (spec_page_scores), the largest over the nodes and query heads of
    a key head: q [B, N, q_heads, head_dim] of the bounds' dtype.  Returns float32 [B, kv_heads,
    max_pages], -inf where a place holds no committed position."""
    args = (q, bounds, page_table, cache_len, page_size, node_count, out, dev_status, None)
    if stream is None:
        return _native().scores(*args)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().scores(*args)


def page_select(scores, page_table, cache_len, page_size, keep, *, first=1, recent=1, extra=0, dev_status=None,
                stream=None):
    """The `keep` pages of each request and key head that rank highest (spec_page_select), the first `first` and
    last `recent` ones before all others, and behind them the pages of `extra` drafted tokens: of all nodes of the
    attention that follows, since it looks them up behind the selected positions.  Returns
    (table, length): int32 [B, kv_heads, keep + ceil(extra / page_size)] and [B], the page_table
    and cache_len of attention over these pages."""
    args = (scores, page_table, cache_len, page_size, keep, first, recent, extra, dev_status, None)
    if stream is None:
        return _native().select(*args)
    with torch.cuda.stream(stream):  # what the call allocates belongs to that stream
        return _native().select(*args)


class _Slots:
    """The page table, the lengths and the status word of a batch of `slots` requests."""

    def _slots(self, num_pages, page_size, slots, max_pages, device):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
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

    def select(self, layer, q, bounds, keep, *, start=None, first=1, recent=1, extra=None, node_count=None,
               stream=None):
        """Pages for attention(..., pages=): the bounds of the pages written since `start` formed, all pages
        scored and the best `keep` of each key head taken, and behind them the pages of `extra` drafted tokens
        (None: the nodes of q, which that attention looks up there).  node_count int32 [slots]: the nodes
        that each slot has; rows of q past them, which that attention leaves out, have no part in the scores."""
        if extra is None:
            extra = q.shape[1]
        self.summarise(layer, bounds, start=start, stream=stream)
        scores = page_scores(q, bounds, self.page_table, self.cache_len, self.page_size, node_count=node_count,
                             dev_status=self.status, stream=stream)
        return page_select(scores, self.page_table, self.cache_len, self.page_size, keep, first=first, recent=recent,
                           extra=extra, dev_status=self.status, stream=stream)

    def _lists(self, pages):
        return (self.page_table, self.cache_len) if pages is None else pages


class PagedCache(_Slots):
    """The cache of a batch of `slots` requests: pools of pages for every layer,
    the page table, the lengths, and the status word the calls report in.  The
    methods work on all slots; single slots are filled, kept or released with
    cache_resize and want_len (0: released, negative: left alone).  dtype:
    bfloat16 or float16, or float32 for the pages alone (attention refuses it)."""

    def __init__(self, layers, num_pages, page_size, kv_heads, head_dim, slots, max_pages, *,
                 dtype=torch.bfloat16, device="cuda"):
        shape = (layers, num_pages, page_size, kv_heads, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self._layers = list(zip(self.k.unbind(0), self.v.unbind(0)))
        self._slots(num_pages, page_size, slots, max_pages, device)

    def new_bounds(self):
        """Bounds of one layer's pages, for select."""
        _, num_pages, _, heads, head_dim = self.k.shape
        return torch.zeros((num_pages, heads, 2, head_dim), dtype=self.k.dtype, device=self.k.device)

    def summarise(self, layer, bounds, start=None, stream=None):
        cache_bounds(self._layers[layer][0], bounds, self.page_table, self.cache_len, start=start,
                     dev_status=self.status, stream=stream)

    def append(self, layer, k_new, v_new, count=None, stream=None):
        k, v = self._layers[layer]
        cache_append(k, v, self.page_table, self.cache_len, k_new, v_new, count=count,
                     dev_status=self.status, stream=stream)

    def attention(self, layer, q, parent=None, pages=None, **kw):
        k, v = self._layers[layer]
        table, length = self._lists(pages)
        return tree_attention(q, k, v, table, length, parent, dev_status=self.status, **kw)

    def commit(self, out_nodes, accept_len, nodes=None, stream=None):
        cache_commit(self.k, self.v, self.page_table, self.cache_len, out_nodes, accept_len, nodes=nodes,
                     dev_status=self.status, stream=stream)

    def fork(self, src, dst, workspace=None, stream=None):
        cache_fork(self.k, self.v, self.page_table, self.page_count, self.page_ref, self.cache_len, src, dst,
                   workspace=workspace, dev_status=self.status, stream=stream)


class PagedCache4(_Slots):
    """PagedCache held in 4 bits: 17/64 of the bytes of bfloat16.  dtype: bfloat16 or float16, that of the
    queries, of new keys and values and of what is read back."""

    def __init__(self, layers, num_pages, page_size, kv_heads, head_dim, slots, max_pages, *, dtype=torch.bfloat16,
                 device="cuda"):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("a 4-bit cache serves bfloat16 or float16")
        self.head_dim, self.dtype = head_dim, dtype
        self.pool = torch.empty((layers, num_pages, kv_heads, cache4_page_bytes(page_size, head_dim)),
                                dtype=torch.uint8, device=device)
        self._layers = list(self.pool.unbind(0))
        self._slots(num_pages, page_size, slots, max_pages, device)

    def new_bounds(self):
        """Bounds of one layer's pages, for select."""
        _, num_pages, heads, _ = self.pool.shape
        return torch.zeros((num_pages, heads, 2, self.head_dim), dtype=self.dtype, device=self.pool.device)

    def _own(self, x, name):
        """(A pool's bytes do not tell: pages have the same for heads of 72, 80, 88 and 96.)"""
        if x.shape[-1] != self.head_dim:
            raise ValueError("%s has heads of %d, the cache of %d" % (name, x.shape[-1], self.head_dim))
        return x

    def summarise(self, layer, bounds, start=None, stream=None):
        self._own(bounds, "bounds")
        cache4_bounds(self._layers[layer], bounds, self.page_table, self.cache_len, self.page_size, start=start,
                      dev_status=self.status, stream=stream)

    def append(self, layer, k_new, v_new, count=None, stream=None):
        cache4_append(self._layers[layer], self.page_table, self.cache_len, self._own(k_new, "k_new"), v_new,
                      self.page_size, count=count, dev_status=self.status, stream=stream)

    def read(self, start, n, layer=None, count=None, stream=None):
        """Keys and values of `n` positions from `start` on (int32 [slots]), of one layer or of all."""
        pool = self.pool if layer is None else self._layers[layer]
        return cache4_read(pool, self.page_table, start, n, self.page_size, self.head_dim, count=count,
                           dtype=self.dtype, dev_status=self.status, stream=stream)

    def attention(self, layer, q, parent=None, pages=None, **kw):
        table, length = self._lists(pages)
        return tree_attention4(self._own(q, "q"), self._layers[layer], table, length, self.page_size, parent,
                               dev_status=self.status, **kw)

    def commit(self, out_nodes, accept_len, nodes=None, stream=None):
        cache4_commit(self.pool, self.page_table, self.cache_len, out_nodes, accept_len, self.page_size, self.head_dim,
                      nodes=nodes, dev_status=self.status, stream=stream)

    def fork(self, src, dst, workspace=None, stream=None):
        cache4_fork(self.pool, self.page_table, self.page_count, self.page_ref, self.cache_len, src, dst,
                    self.page_size, self.head_dim, workspace=workspace, dev_status=self.status, stream=stream)
