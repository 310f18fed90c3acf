"""The cache operators in CUDA graphs: what a captured call works in is not given
to anything else, whatever is called and allocated before the replays."""
import pytest
import torch

import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _sv():
    import speculative_decoding_verification_69_gb300 as sv
    return sv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(seed, lens, N, hq=8, hkv=2, D=64, page=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    P = max(-(-(n + N) // page) for n in lens)
    pages = sum(-(-(n + N) // page) for n in lens)
    table, _, _, cl = ch.make_table(g, lens, N, page, P, pages)
    k, v = (ch.make_pool(g, pages, page, hkv, D, torch.bfloat16) for _ in range(2))
    q = torch.randn((len(lens), N, hq, D), generator=g, device="cuda").bfloat16()
    return dict(q=q, k=k, v=v, table=table, len=cl, parent=ch.random_parents(g, len(lens), N))


def _call(c, **kw):
    return _sv().tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], return_lse=True, **kw)


def _stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    return s


def _larger_call_and_fills(s, sizes):
    """A call of many rows on the stream, and then tensors of the sizes that the
    calls before it worked in, full of a pattern."""
    big = _case(99, [700, 90], 64)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _call(big)
        fills = [torch.full((n,), 90, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(40)]
    s.synchronize()
    return fills


def _untouched(fills):
    return all(bool((x == 90).all()) for x in fills)


@pytest.mark.parametrize("N,lens", [(1, [3000]), (9, [700, 40]), (4, [0, 5000, 3])])
def test_attention_replayed_after_a_larger_call(N, lens):
    c = _case(N, lens, N)
    n = _sv().load_library().spec_tree_attention_workspace_bytes(len(lens), N, 8, 2, 64)
    s = _stream()
    with torch.cuda.stream(s):
        _call(c)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, l = _call(c)
    fills = _larger_call_and_fills(s, [n])
    for scale in (1.0, 0.5):
        c["q"].mul_(scale)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert _untouched(fills)
        ref = ch.ref_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"])
        ch.check_attention(o, l, ref, torch.bfloat16, 64)


def test_fork_replayed_after_a_larger_call():
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(5)
    page, lens = 16, [37, 16, 5] + [0] * 9
    table, count, ref, cl = ch.make_table(g, lens, 0, page, 6, 40)
    k, v = (ch.make_pool(g, 40, page, 2, 64, torch.bfloat16, layers=2) for _ in range(2))
    src, dst = [0, 0, 1, 2, 2, 0, 2], [3, 4, 5, 6, 7, 8, 9]
    s, a, b = _stream(), _i32(src), _i32(dst)
    st = _i32([0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sv.cache_fork(k, v, table, count, ref, cl, a, b, dev_status=st)
    fills = _larger_call_and_fills(s, [256, 512])
    for _ in range(3):  # from the second time on the destinations give back what they got
        model = ch.Pages(table.cpu(), count.cpu(), ref.cpu(), cl.cpu())
        ek, ev = k.clone(), v.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        copies, missed = model.fork(src, dst, page)
        assert not missed and len(copies) == 6
        for x, y, n in copies:
            ek[:, y, :n], ev[:, y, :n] = ek[:, x, :n], ev[:, x, :n]
        model.check(table.cpu(), count.cpu(), ref.cpu(), cl.cpu())
        assert torch.equal(k, ek) and torch.equal(v, ev) and int(st) == 0 and _untouched(fills)


def test_two_graphs_replayed_side_by_side():
    """Captured on one stream, replayed on two and beside calls on that stream."""
    cases = [_case(20, [9000], 5), _case(21, [4000, 4100], 5)]
    want = [_call(c) for c in cases]
    capture = _stream()
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            got.append(_call(c))
        graphs.append(graph)
    other = _case(22, [8000], 5)
    streams = [_stream(), _stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(capture):
            _call(other)
        torch.cuda.synchronize()
        for (o, l), (eo, el) in zip(got, want):
            assert torch.equal(o, eo) and torch.equal(l, el)
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()


def test_a_whole_step_replayed():
    """Pages, new keys, attention, the accepted path and the pages returned: the
    replays continue the sequence as the same calls do outside a graph."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(7)
    slots, N, layers, hkv, D = 3, 6, 2, 2, 64
    parent = ch.random_parents(g, slots, N)
    nodes = _i32([[1, 3, -1, -1, -1, -1], [-1] * 6, [2, 4, 5, -1, -1, -1]])
    accept = _i32([2, 0, 3])
    kv = torch.randn((layers, slots, N, 2 * hkv, D), generator=g, device="cuda").bfloat16()
    q = torch.randn((layers, slots, N, 8, D), generator=g, device="cuda").bfloat16()

    def step(cache):
        cache.reserve(N)
        out = []
        for layer in range(layers):
            cache.append(layer, kv[layer, :, :, :hkv], kv[layer, :, :, hkv:])
            out.append(cache.attention(layer, q[layer], parent))
        cache.commit(nodes, accept)
        cache.trim()
        return out

    caches = [sv.PagedCache(layers, 30, 8, hkv, D, slots, 10) for _ in range(2)]
    for c in caches:
        c.k.zero_()
        c.v.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for _ in range(8):
        graph.replay()
        want = step(caches[1])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("k", "v", "page_table", "page_count", "page_ref", "cache_len", "status"):
            assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    assert caches[0].cache_len.tolist() == [24, 8, 32] and int(caches[0].status) == 0


def test_fork_in_a_given_workspace():
    sv = _sv()
    k = torch.randn((1, 8, 8, 1, 8), device="cuda").bfloat16()
    state = [_i32([[0, 1], [-1, -1]]), _i32([2, 0]), _i32([1, 1, 0, 0, 0, 0, 0, 0]), _i32([11, 0])]

    def fork(ws):
        sv.cache_fork(k, k.clone(), *state, _i32([0]), _i32([1]), workspace=ws)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    fork(ws)
    assert state[0].tolist() == [[0, 1], [0, 2]] and state[3].tolist() == [11, 11]
    assert torch.equal(k[:, 2, :3], k[:, 1, :3]) and ws.view(torch.int32)[:3].tolist() == [1, 2, 3]
    with pytest.raises(sv.SpecVerifyError):
        fork(ws[:128])
    with pytest.raises(ValueError):
        fork(ws.cpu())
    with pytest.raises(TypeError):
        fork(256)
