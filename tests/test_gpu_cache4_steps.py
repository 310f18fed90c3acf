"""The 4-bit cache and the selection of pages in whole steps, in CUDA graphs and in calls that are refused."""
import pytest
import torch

import cache4_helpers as c4
import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _sv():
    import speculative_decoding_verification_69_gb300 as sv
    return sv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(g, shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _filled(g, lens, *, layers=2, pages=90, page=8, hkv=2, D=64, slots=None, max_pages=24):
    """A PagedCache4 whose first slots hold prompts of these lengths."""
    sv = _sv()
    cache = sv.PagedCache4(layers, pages, page, hkv, D, slots or len(lens), max_pages)
    want = _i32(list(lens) + [0] * ((slots or len(lens)) - len(lens)))
    sv.cache_resize(cache.page_table, cache.page_count, cache.page_ref, want, page, dev_status=cache.status)
    for i in range(layers):
        x = _rows(g, (want.numel(), max(lens), 2 * hkv, D))
        cache.append(i, x[:, :, :hkv], x[:, :, hkv:], count=want)
    cache.cache_len.copy_(want)
    return cache


def test_steps_of_drafted_trees():
    """Prompts, a fork, and three steps of trees of seven nodes: after each, attention is that of the numbers the pool
    holds, and the accepted nodes are those that were appended, behind their root."""
    g = torch.Generator(device="cuda").manual_seed(21)
    hkv, hq, D, N, page, slots = 2, 8, 64, 7, 8, 4
    cache = _filled(g, [30, 61], slots=slots)
    cache.fork(_i32([0, 1]), _i32([2, 3]))
    assert cache.cache_len.tolist() == [30, 61, 30, 61]
    k0, v0 = cache.read(_i32([0] * slots), 61, count=cache.cache_len)
    assert torch.equal(k0[:, 0], k0[:, 2]) and torch.equal(v0[:, 1], v0[:, 3])
    rows = [k0[:, b, :n].clone() for b, n in enumerate(cache.cache_len.tolist())]
    paths = [[[1, 2, 3], [4], [], [2, 5, 6]], [[3], [1, 6], [2, 4, 5], []], [[], [1, 2, 3, 4, 5, 6], [6], [5]]]
    for step in range(3):
        parent = ch.random_parents(g, slots, N)
        lens = cache.cache_len.tolist()
        cache.reserve(N)
        new = []
        for i in range(2):
            x = _rows(g, (slots, N, hq + 2 * hkv, D))
            q = x[:, :, :hq]
            cache.append(i, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:])
            new.append(c4.values(x[:, :, hq:hq + hkv]).bfloat16())
            o, l = cache.attention(i, q, parent, return_lse=True)
            ref = c4.ref_attention(q, cache.pool[i], page, cache.page_table, cache.cache_len, parent)
            ch.check_attention(o, l, ref, torch.bfloat16, D)
        nodes = torch.full((slots, N), -1, dtype=torch.int32, device="cuda")
        for b, path in enumerate(paths[step]):
            if path:
                nodes[b, :len(path)] = _i32(path)
            rows[b] = torch.cat([rows[b]] + [torch.stack([new[i][b, n] for i in range(2)]).unsqueeze(1)
                                             for n in [0] + path], 1)
        cache.commit(nodes, _i32([len(p) for p in paths[step]]))
        cache.trim()
        assert cache.cache_len.tolist() == [n + 1 + len(p) for n, p in zip(lens, paths[step])]
        most = max(cache.cache_len.tolist())
        k, _ = cache.read(_i32([0] * slots), most, count=cache.cache_len)
        for b, n in enumerate(cache.cache_len.tolist()):
            assert torch.equal(k[:, b, :n], rows[b]) and (k[:, b, n:] == 0).all()
        k1, _ = cache.read(_i32([5] * slots), 9, layer=1)
        assert torch.equal(k1, k[1][:, 5:14])
    assert int(cache.status) == 0


def test_a_captured_step_replayed_after_other_calls():
    """Append, attention, selection, attention over the selected pages and the commit in one graph: what it works in is
    not given to later calls, and every replay is a step further."""
    hkv, hq, D, N, keep = 2, 8, 64, 3, 4
    caches, outs = [], []
    for captured in (False, True):
        g = torch.Generator(device="cuda").manual_seed(5)
        cache = _filled(g, [40, 7, 101])
        cache.reserve(4 * N)
        bounds = cache.new_bounds()
        x = _rows(g, (3, N, hq + 2 * hkv, D))
        acc = _i32([1, 0, 2])

        def step():
            cache.append(0, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:])
            cache.append(1, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:])
            a = cache.attention(0, x[:, :, :hq])
            pages = cache.select(1, x[:, :, :hq], bounds, keep, extra=N)
            b = cache.attention(1, x[:, :, :hq], pages=pages)
            cache.commit(None, acc, nodes=N)
            return a, b

        res = []
        torch.cuda.synchronize()
        if captured:
            s = torch.cuda.Stream()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = step()
            assert cache.cache_len.tolist() == [40, 7, 101]
            other = _filled(torch.Generator(device="cuda").manual_seed(6), [90, 100], D=128, layers=1)
            fills = []
            for k in range(4):
                with torch.cuda.stream(s):
                    graph.replay()
                    res.append([t.clone() for t in out])
                s.synchronize()
                other.reserve(9)
                other.append(0, *(_rows(g, (2, 9, 2, 128)) for _ in range(2)))
                other.attention(0, _rows(g, (2, 9, 8, 128)))
                fills += [torch.full((n,), 90, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 20)]
                torch.cuda.synchronize()
            assert all(bool((t == 90).all()) for t in fills) and int(other.status) == 0
        else:
            for k in range(4):
                res.append([t.clone() for t in step()])
        torch.cuda.synchronize()
        assert int(cache.status) == 0 and cache.cache_len.tolist() == [48, 11, 113]
        caches.append(cache)
        outs.append(res)
    used = caches[0].page_table[caches[0].page_table >= 0].long()
    assert torch.equal(caches[0].page_table, caches[1].page_table)
    k, v = zip(*(c.read(_i32([0, 0, 0]), 113, count=c.cache_len) for c in caches))
    assert torch.equal(*k) and torch.equal(*v) and used.numel() > 0
    for a, b in zip(*outs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tensors_that_require_a_gradient_are_refused():
    sv = _sv()
    page, D = 8, 32
    pool = c4.make_pool(torch.Generator(device="cuda").manual_seed(1), 4, 1, page, D)
    table, one, zero = _i32([[0, 1]]), _i32([1]), _i32([0])
    x = torch.randn((1, 2, 1, D), device="cuda").bfloat16()
    k = torch.randn((4, page, 1, D), device="cuda").bfloat16()
    bounds = torch.zeros((4, 1, 2, D), device="cuda", dtype=torch.bfloat16)
    scores = torch.zeros((1, 1, 2), device="cuda")
    lists = table.view(1, 1, 2)

    def grad(t):
        return t.detach().clone().requires_grad_(True)
    calls = [(lambda t: sv.cache4_append(pool, table, one, t, x, page), x),
             (lambda t: sv.cache4_append(pool, table, one, x, t, page), x),
             (lambda t: sv.tree_attention4(t, pool, table, one, page), x),
             (lambda t: sv.tree_attention4(x, pool, table, one, page, out=t), x),
             (lambda t: sv.tree_attention(t, k, k, lists, one), x),
             (lambda t: sv.tree_attention(x, t, k, lists, one), k),
             (lambda t: sv.cache_bounds(t, bounds, table, one), k),
             (lambda t: sv.cache_bounds(k, t, table, one), bounds),
             (lambda t: sv.cache4_bounds(pool, t, table, one, page), bounds),
             (lambda t: sv.page_scores(t, bounds, table, one, page), x),
             (lambda t: sv.page_scores(x, t, table, one, page), bounds),
             (lambda t: sv.page_scores(x, bounds, table, one, page, out=t), scores),
             (lambda t: sv.page_select(t, table, one, page, 1, first=0), scores)]
    for call, t in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(grad(t))
        with torch.no_grad():
            call(grad(t))
        call(t)
    torch.cuda.synchronize()


def test_shapes_that_are_refused():
    sv = _sv()
    page, D, hkv, B, N = 16, 64, 2, 2, 3
    pool = c4.make_pool(torch.Generator(device="cuda").manual_seed(1), 6, hkv, page, D)
    table, lens = _i32([[0, 1, 2], [3, 4, 5]]), _i32([4, 5])
    q, x = (torch.randn((B, N, h, D), device="cuda").bfloat16() for h in (4, hkv))
    bounds = torch.zeros((6, hkv, 2, D), device="cuda", dtype=torch.bfloat16)
    scores = torch.zeros((B, hkv, 3), device="cuda")
    lists = table.unsqueeze(1).expand(B, hkv, 3).contiguous()
    refused = [
        lambda: sv.tree_attention4(q, pool, table, lens, 32),                         # pages of another size
        lambda: sv.tree_attention4(q, pool[:, :, :-16], table, lens, page),
        lambda: sv.tree_attention4(q, pool.unsqueeze(0), table, lens, page),          # layers
        lambda: sv.tree_attention4(q[:, :, :3], pool, table, lens, page),             # 3 heads over 2
        lambda: sv.tree_attention4(q, pool, lists[:, :1].contiguous(), lens, page),   # one list for two heads
        lambda: sv.tree_attention4(q, pool, lists.transpose(0, 2), lens, page),
        lambda: sv.tree_attention4(q, pool, table.long(), lens, page),
        lambda: sv.tree_attention4(q, pool, table, lens[:1], page),
        lambda: sv.tree_attention4(q, pool, table, lens.cpu(), page),
        lambda: sv.tree_attention4(q, pool, table, lens, page, scale=0.0),
        lambda: sv.tree_attention4(q, pool, table, lens, page, window=-1),
        lambda: sv.tree_attention4(q, pool, table, lens, page, out=q.half()),
        lambda: sv.tree_attention4(q, pool, table, lens, page, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: sv.tree_attention4(torch.zeros((B, 65, 4, D), device="cuda").bfloat16(), pool, table, lens, page),
        lambda: sv.cache4_append(pool, table, lens, x, x.half(), page),
        lambda: sv.cache4_append(pool, table, lens, x[:, :, :1], x[:, :, :1], page),
        lambda: sv.cache4_append(pool, table, lens, x[:1], x[:1], page),
        lambda: sv.cache4_read(pool, table, lens, 0, page, D),
        lambda: sv.cache4_commit(pool.unsqueeze(0), table, lens, None, lens, page, D),  # how many nodes?
        lambda: sv.cache4_copy(pool.unsqueeze(0), _i32([0]), _i32([1, 2]), page, D),
        lambda: sv.cache4_bounds(pool, bounds[:, :1].contiguous(), table, lens, page),
        lambda: sv.cache_bounds(x.view(6, 1, 2, D).contiguous(), bounds.half(), table, lens),
        lambda: sv.page_scores(q.half(), bounds, table, lens, page),
        lambda: sv.page_scores(q[..., :32], bounds, table, lens, page),
        lambda: sv.page_scores(q, bounds, table, lens, 12),
        lambda: sv.page_scores(q, bounds, table, lens, page, out=scores[:, :1]),
        lambda: sv.page_select(scores, table[:, :2].contiguous(), lens, page, 2),
        lambda: sv.page_select(scores, table, lens, page, 0),
        lambda: sv.page_select(scores, table, lens, page, 2, first=2, recent=1),
        lambda: sv.page_select(scores, table, lens, page, 2, recent=0),
        lambda: sv.page_select(scores.double(), table, lens, page, 2),
    ]
    before = pool.clone()
    for i, call in enumerate(refused):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
            pytest.fail("call %d was taken" % i)
    torch.cuda.synchronize()
    assert torch.equal(pool, before) and lens.tolist() == [4, 5]
