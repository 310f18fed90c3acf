"""Tree attention over a 4-bit cache against the definition in 64 bits."""
import pytest
import torch

import cache4_helpers as c4
import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _sv():
    import speculative_decoding_verification_69_gb300 as sv
    return sv


def _case(seed, lens, N, hq, hkv, D, page, dtype, *, tree=True, qscale=2.0, spare=3, per_head=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    P = max(-(-(n + N) // page) for n in lens) + 1
    pages = sum(-(-(n + N) // page) for n in lens) + spare
    table, _, _, cl = ch.make_table(g, lens, N, page, P, pages)
    if per_head:  # every key head its own order of pages
        table = torch.stack([torch.cat([ch.make_table(g, lens, N, page, P, pages)[0][b:b + 1] for _ in range(hkv)])
                             for b in range(B)]).contiguous()
    pool = c4.make_pool(g, pages, hkv, page, D)
    q = (torch.randn((B, N, hq, D), generator=g, device="cuda") * qscale).to(dtype)
    return dict(q=q, pool=pool, page=page, table=table, len=cl, parent=ch.random_parents(g, B, N) if tree else None)


def _run(c, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = _sv().tree_attention4(c["q"], c["pool"], c["table"], c["len"], c["page"], c["parent"], return_lse=True,
                                 dev_status=st, **kw)
    torch.cuda.synchronize()
    return o, l, int(st.item())


def _check(c, status=0, **kw):
    o, l, st = _run(c, **kw)
    assert st == status
    ref = c4.ref_attention(c["q"], c["pool"], c["page"], c["table"], c["len"], c["parent"], **kw)
    ch.check_attention(o, l, ref, c["q"].dtype, c["q"].shape[-1])
    return o, l


LENS = [0, 1, 7, 8, 63, 64, 127, 128, 129, 200, 255, 256, 257, 511, 640]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page", [
    (1, 8, 8, 64, 16),       # single tokens, a key head each
    (1, 8, 1, 128, 8),       # one key head for all
    (1, 32, 8, 128, 16),
    (2, 4, 4, 8, 8),         # the smallest head
    (1, 5, 5, 32, 32),       # an odd number of small heads
    (4, 6, 3, 64, 64),       # and of heads of 64
    (9, 8, 2, 128, 16),      # linear-draft size
    (16, 14, 2, 128, 32),    # a group of 7
    (16, 16, 4, 128, 128),   # 64 rows exactly
    (17, 12, 3, 96, 16),     # just past
    (33, 4, 1, 96, 64),
    (64, 4, 2, 64, 128),
    (64, 8, 2, 128, 256),    # pages longer than a tile of keys
    (63, 10, 2, 72, 16),     # 315 rows, a head of 72
    (3, 128, 2, 40, 8),      # a group of 64
    (64, 64, 1, 40, 8),      # 4096 rows of one key head
])
def test_lengths_heads_layouts(N, hq, hkv, D, page, dtype):
    lens = LENS if hq < 64 else [0, 5, 130, 300]
    _check(_case(N * 131 + D, lens, N, hq, hkv, D, page, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page", [(1, 8, 2, 128, 16), (5, 12, 3, 64, 8), (9, 8, 4, 64, 64),
                                             (40, 8, 2, 80, 16), (2, 16, 16, 32, 128), (3, 8, 4, 64, 256)])
def test_a_list_of_pages_for_every_key_head(N, hq, hkv, D, page, dtype):
    _check(_case(N + D, LENS[:12], N, hq, hkv, D, page, dtype, per_head=True))


@pytest.mark.parametrize("N", [1, 9, 33])
def test_chain_is_causal(N):
    c = _case(7, [0, 3, 100, 700], N, 8, 2, 128, 16, torch.bfloat16, tree=False)
    o, l = _check(c)
    c["parent"] = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(4, 1)
    o2, l2, _ = _run(c)
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (17, 0), (64, 3), (128, 130), (129, 128),
                                          (300, 1), (5000, 4), (700, 0)])
@pytest.mark.parametrize("N,hq,hkv,D,page", [(1, 8, 1, 64, 16), (12, 8, 2, 64, 16), (40, 8, 2, 128, 64),
                                             (5, 8, 2, 128, 8)])
def test_window_and_sinks(N, hq, hkv, D, page, window, sinks):
    _check(_case(window * 7 + N, [0, 1, 5, 127, 128, 300, 513, 1000], N, hq, hkv, D, page, torch.bfloat16),
           window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window", [0, 100])
def test_unseen_positions_hold_anything(window, dtype):
    """The largest scales at every position of the pool that no node sees; rubbish in the table's entries for pages
    that no node sees; counts of nodes, 0 among them."""
    page, N, lens, D = 16, 11, [0, 4, 37, 250, 260, 385], 64
    c = _case(91, lens, N, 8, 2, D, page, dtype)
    cnt = torch.tensor([11, 3, 11, 0, 7, 10], dtype=torch.int32, device="cuda")
    sinks = 3 if window else 0
    seen = torch.zeros((c["pool"].shape[0], page), dtype=torch.bool)
    for b, n0 in enumerate(lens):
        used = set()
        for p in ch.paths(c["parent"][b].tolist(), int(cnt[b])):
            used |= set(ch.seen_positions(n0, p, window, sinks))
        row = c["table"][b].tolist()
        for j in used:
            seen[row[j // page], j % page] = True
        for i in range(c["table"].shape[1]):
            if not any(j // page == i for j in used):
                c["table"][b, i] = [-1, 2 ** 31 - 1, -2 ** 31][i % 3]
    for kind in "kv":
        sc = c4.places(page, D, kind)[2]
        for p, t in (~seen).nonzero().tolist():
            c["pool"][p][:, sc[t].cuda()] = 255
    o, l = _check(c, node_count=cnt, window=window, sinks=sinks)
    for b in range(len(lens)):  # rows past the count see nothing
        assert (o[b, int(cnt[b]):] == 0).all() and torch.isneginf(l[b, int(cnt[b]):]).all()


@pytest.mark.parametrize("N,hq,hkv,D,ctx", [(1, 8, 1, 128, 70001), (16, 8, 2, 128, 20000), (64, 8, 2, 64, 9999),
                                            (5, 4, 4, 64, 33333), (1, 4, 4, 128, 12345)])
def test_long_contexts(N, hq, hkv, D, ctx):
    _check(_case(ctx, [ctx], N, hq, hkv, D, 64, torch.bfloat16))


def test_many_requests_of_mixed_lengths():
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in (torch.rand(300, generator=g) ** 3 * 900).tolist()] + [4000, 0, 0, 0]
    _check(_case(17, lens, 5, 8, 4, 64, 16, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,G,hkv,D,page,window,sinks", [
    (1, 1, 80, 64, 16, 0, 0),
    (9, 8, 40, 64, 16, 128, 0),
    (16, 8, 38, 128, 32, 0, 0),
    (13, 3, 63, 72, 8, 50, 2),
    (7, 5, 102, 40, 256, 700, 1),
])
def test_many_heads(N, G, hkv, D, page, window, sinks, dtype):
    lens = [0, 3, 127, 128, 129, 300, 1000, 64][:8 if hkv < 100 else 3]
    _check(_case(D + N, lens, N, G * hkv, hkv, D, page, dtype), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_that_grow(dtype):
    """Keys whose scores rise and fall by orders of magnitude along the sequence: the running reference moves."""
    D, page = 128, 16
    c = _case(5, [900, 2000], 3, 8, 2, D, page, dtype, qscale=1.0)
    sc = c4.places(page, D, "k")[2].cuda()
    for b, n0 in enumerate((900, 2000)):
        for i in range(-(-(n0 + 3) // page)):
            c["pool"][int(c["table"][b, i])][:, sc] = 112 + (i * 37 % 48) if b else 112 + min(48, i)
    _check(c)


def test_rows_that_are_not_finite():
    """q with NaN or infinities: those rows come out NaN, the others as they were."""
    c = _case(8, [0, 40, 300], 4, 8, 2, 64, 16, torch.bfloat16)
    o, l = _check(c)
    c["q"][1, 2, 3, 5] = float("nan")
    c["q"][2, 0, 7, 0] = float("inf")
    o2, l2, st = _run(c)
    bad = torch.zeros(o.shape[:3], dtype=torch.bool, device="cuda")
    bad[1, 2, 3] = bad[2, 0, 7] = True
    assert st == 0 and torch.isnan(l2[bad]).all() and torch.isnan(o2[bad]).all()
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(l2[~bad], l[~bad])


def test_scores_of_minus_infinity():
    """A row whose scores are all -inf is NaN; one whose scores are -inf in some places has no weight there."""
    sv = _sv()
    D, page = 32, 8
    pool = torch.zeros((2, 1, c4.page_bytes(page, D)), dtype=torch.uint8, device="cuda")
    x = torch.full((1, 12, 1, D), 1.0, device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = torch.arange(12, device="cuda").view(1, 12, 1, 1).expand(1, 12, 1, D).bfloat16()
    x[0, 5:] = 0.0
    sv.cache4_append(pool, table, zero, x, v, page)
    q = torch.full((1, 1, 2, D), 3.0e38, device="cuda", dtype=torch.bfloat16)
    q[:, :, 1] = -3.0e38
    o, l = sv.tree_attention4(q, pool, table, zero + 4, page, return_lse=True)
    assert torch.isnan(o).all() and torch.isnan(l).all()              # +inf; all -inf
    o, l = sv.tree_attention4(q, pool, table, zero + 11, page, return_lse=True)
    assert torch.isnan(o[:, :, 0]).all()
    k, vv = sv.cache4_read(pool, table, zero, 12, page, D)
    want = vv[0, 5:12, 0].double().mean(0)
    assert (o[0, 0, 1].double() - want).abs().max() <= 2 ** -7 * 11 and abs(float(l[0, 0, 1]) - 1.9459101) < 1e-5


@pytest.mark.parametrize("dtype,power", [(torch.bfloat16, 10), (torch.bfloat16, 14), (torch.bfloat16, 30),
                                         (torch.bfloat16, 90), (torch.float16, 10), (torch.float16, 14)])
@pytest.mark.parametrize("N,hq,hkv,D", [(1, 4, 2, 128), (8, 4, 1, 128), (40, 2, 1, 128), (9, 4, 2, 64)])
def test_scores_as_large_as_float32_holds(power, N, hq, hkv, D, dtype):
    """One key twice as large as all others, and scores so large that it takes all the weight: the result is its value,
    which the formats hold, but for the roundings of that weight 2^z to float16 (the sum takes it unrounded, and z is
    whole only where the scores are less their reference exactly) and of the result, each half a step.  The key lies
    in the first tile or in a later one."""
    page, lens = 16, [5, 130, 700, 2000]
    c = _case(power + N, lens, N, hq, hkv, D, page, dtype, tree=False)
    sc = c4.places(page, D, "k")[2].cuda()
    at = c4.places(page, D, "k")[0].cuda()
    c["pool"][..., sc] = 248 if power > 10 else 152                   # 2^12 and 1
    c["pool"][..., :page * D // 2] = 0xBB                             # all keys 3 scales
    for b, (n0, j) in enumerate(zip(lens, (3, 129, 0, 1777))):
        p = int(c["table"][b, j // page])
        byte = torch.unique(at[j % page])
        c["pool"][p, :, byte] = 0xEE                                  # and one of 6
    c["q"].fill_(2.0 ** power)
    o, l, st = _run(c, scale=1.0)
    k, v = c4.decode(c["pool"], page, D)
    for b, j in enumerate((3, 129, 0, 1777)):
        p = int(c["table"][b, j // page])
        want = v[p, j % page].to(dtype).repeat_interleave(hq // hkv, 0)
        score = float(k[p, j % page, 0].sum()) * 2.0 ** power
        assert ((o[b] - want).double().abs() <= want.double().abs() * (2 ** -11 + torch.finfo(dtype).eps / 2 + 2 ** -18)).all()
        assert (l[b].double() - score).abs().max() <= score * 2 ** -20
    assert st == 0


def test_bad_inputs_are_reported():
    sv = _sv()
    c = _case(12, [20, 50], 6, 4, 2, 64, 16, torch.bfloat16)
    c["parent"][0, 3] = 5                                              # not an earlier node
    _check(c, status=sv.DEV_BAD_TREE)
    c = _case(12, [20, 50], 6, 4, 2, 64, 16, torch.bfloat16)
    c["len"][1] = 16 * c["table"].shape[1] - 3                         # three nodes past the row's reach
    assert _run(c)[2] & sv.DEV_BAD_LEN
    c["len"][1] = -4
    assert _run(c)[2] == sv.DEV_BAD_LEN
    c["len"][1] = 50
    c["table"][1, 1] = 10 ** 6
    assert _run(c)[2] == sv.DEV_BAD_PAGE


@pytest.mark.parametrize("N,hq,hkv,D", [(1, 8, 2, 128), (12, 8, 4, 64)])
def test_same_results_every_time(N, hq, hkv, D):
    c = _case(3, [3000, 17, 900], N, hq, hkv, D, 16, torch.bfloat16)
    o, l, _ = _run(c)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127):
        ws.fill_(fill)
        o2, l2, _ = _run(c, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_streams_out_and_graphs():
    sv = _sv()
    c = _case(4, [700, 40, 0], 5, 8, 2, 128, 16, torch.bfloat16)
    o, l, _ = _run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(o)
    got = sv.tree_attention4(c["q"], c["pool"], c["table"], c["len"], c["page"], c["parent"], out=out, stream=s)
    s.synchronize()
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, o)
    graphs = []
    for lens in ([700, 40, 0], [300, 500, 64]):                        # two graphs, each with a workspace of its own
        d = _case(4, lens, 5, 8, 2, 128, 16, torch.bfloat16)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            res = sv.tree_attention4(d["q"], d["pool"], d["table"], d["len"], d["page"], d["parent"], return_lse=True)
        graphs.append((graph, d, res))
    for _ in range(2):
        for graph, d, res in graphs:
            d["q"].mul_(0.5)
            torch.cuda.synchronize()
            graph.replay()
        torch.cuda.synchronize()
        for graph, d, res in graphs:
            ref = c4.ref_attention(d["q"], d["pool"], d["page"], d["table"], d["len"], d["parent"])
            ch.check_attention(res[0], res[1], ref, torch.bfloat16, 128)


@pytest.mark.parametrize("N,hq,hkv,D", [(1, 8, 2, 128), (9, 8, 2, 64), (8, 8, 2, 128), (64, 16, 2, 128), (40, 4, 1, 64)])
def test_wait_that_runs_out_is_reported(N, hq, hkv, D):
    """Every wait between the kernel's roles gives up at once: the call reports it and ends, the next one is right."""
    sv = _sv()
    c = _case(N, [900, 300, 5], N, hq, hkv, D, 16, torch.bfloat16)
    try:
        sv.force_wait_timeout(True)
        _, _, st = _run(c)
    finally:
        sv.force_wait_timeout(False)
    assert st == sv.DEV_TIMEOUT
    _check(c)


@pytest.mark.parametrize("N,hq,hkv,D", [(1, 8, 2, 128), (9, 12, 3, 64), (5, 8, 1, 64), (64, 8, 2, 96)])
def test_exact_workspace_and_two_calls_at_once(N, hq, hkv, D):
    """The workspace that the library asks for, full of a pattern, suffices; calls on two streams, each with its own,
    do not disturb each other."""
    sv = _sv()
    cs = [_case(N + i, [700, 90, 0, 2000 * i], N, hq, hkv, D, 16, torch.bfloat16) for i in range(2)]
    want = [_check(c) for c in cs]
    n = sv.load_library().spec_tree_attention4_workspace_bytes(4, N, hq, hkv, D)
    guard = [torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for c, w, s in zip(cs, guard, streams):
            got.append(sv.tree_attention4(c["q"], c["pool"], c["table"], c["len"], c["page"], c["parent"],
                                          return_lse=True, workspace=w[:n], stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    assert all(bool((w[n:] == 255).all()) for w in guard)
