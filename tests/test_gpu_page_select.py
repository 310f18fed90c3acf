"""Attention over selected pages: bounds, scores, selection and the attention, against plain 64-bit steps."""
import math

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


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _case(seed, lens, N, hq, hkv, D, page, dtype, *, four=False, hnd=False, extra_places=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    P = max(-(-(n + N) // page) for n in lens) + extra_places
    pages = sum(-(-(n + N) // page) for n in lens) + 3
    table, _, _, cl = ch.make_table(g, lens, N, page, P, pages)
    c = dict(table=table, len=cl, page=page, lens=lens)
    if four:
        c["pool"] = c4.make_pool(g, pages, hkv, page, D)
        c["k"], c["v"] = (x.to(dtype) for x in c4.decode(c["pool"], page, D))
    else:
        c["k"], c["v"] = (ch.make_pool(g, pages, page, hkv, D, dtype, hnd=hnd) for _ in range(2))
    qkv = (torch.randn((B, N, hq + 3, D), generator=g, device="cuda") * 2).to(dtype)
    c["q"] = qkv[:, :, :hq]
    return c


def _ref_bounds(c, bounds, start):
    out, page = bounds.clone(), c["page"]
    for b, n0 in enumerate(c["lens"]):
        s = max(0, start[b])
        if s >= n0:
            continue
        for i in range(s // page, -(-n0 // page)):
            k = c["k"][int(c["table"][b, i])][:min(page, n0 - i * page)]
            out[int(c["table"][b, i])] = torch.stack((k.amin(0), k.amax(0)), 1)
    return out


def _ref_scores(c, bounds, count=None):
    """Scores in 64 bits, and the sums of the magnitudes that were added."""
    B, N, hq, D = c["q"].shape
    hkv, P = c["k"].shape[2], c["table"].shape[1]
    out = torch.full((B, hkv, P), -math.inf, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for b, n0 in enumerate(c["lens"]):
        n, cnt = -(-n0 // c["page"]), N if count is None else count[b]
        if n == 0 or cnt == 0:
            continue
        q = c["q"][b, :cnt].double().view(cnt, hkv, -1, D)
        bd = bounds[c["table"][b, :n].long()].double()                 # [n, hkv, 2, D]
        lo, hi = (torch.einsum("nhgd,phd->hpng", f(q), bd[:, :, i]).flatten(2)
                  for i, f in ((0, lambda x: x.clamp(max=0)), (1, lambda x: x.clamp(min=0))))
        al, ah = (torch.einsum("nhgd,phd->hpng", f(q).abs(), bd[:, :, i].abs()).flatten(2)
                  for i, f in ((0, lambda x: x.clamp(max=0)), (1, lambda x: x.clamp(min=0))))
        out[b, :, :n] = (lo + hi).amax(-1)
        mag[b, :, :n] = (al + ah).amax(-1)
    return out, mag


def _ref_select(scores, table, lens, page, keep, first=1, recent=1, extra=0):
    B, H, P = scores.shape
    tail = -(-extra // page)
    rows, kept = [], []
    for b, n0 in enumerate(lens):
        n = -(-n0 // page)
        row = table[b].tolist()
        m = min(n, keep)
        per_head = []
        for h in range(H):
            val = [math.nan if math.isnan(x) else x for x in scores[b, h, :n].tolist()]
            must = [p for p in range(n) if p < first or p >= n - recent]
            rest = sorted((p for p in range(n) if p not in set(must)),
                          key=lambda p: (0 if math.isnan(val[p]) else 1, -val[p] if not math.isnan(val[p]) else 0, p))
            chosen = sorted((must + rest)[:m]) if n > keep else list(range(n))
            behind = [row[n + i] if n + i < P else -1 for i in range(tail)]
            per_head.append([row[p] for p in chosen] + behind + [-1] * (keep - m))
        rows.append(per_head)
        kept.append(n0 - (n - m) * page)
    return torch.tensor(rows, dtype=torch.int32), kept


LENS = [0, 1, 7, 8, 16, 100, 255, 256, 257, 700]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hkv,D,page,hnd,four", [(8, 128, 16, False, False), (2, 64, 8, True, False), (1, 8, 64, False, False),
                                                 (33, 80, 16, True, False), (3, 96, 256, False, False),
                                                 (8, 128, 16, False, True), (3, 72, 8, False, True), (1, 32, 256, False, True)])
@pytest.mark.parametrize("where", ["all", "last", "mixed"])
def test_bounds(hkv, D, page, hnd, four, where, dtype):
    sv = _sv()
    c = _case(hkv + D, LENS, 1, hkv, hkv, D, page, dtype, four=four, hnd=hnd)
    bounds = torch.full((c["k"].shape[0], hkv, 2, D), 77.0, dtype=dtype, device="cuda")
    start = {"all": [0] * len(LENS), "last": [max(0, n - 1) for n in LENS],
             "mixed": [-3 if i % 3 == 0 else n * (i % 3) // 2 for i, n in enumerate(LENS)]}[where]
    want = _ref_bounds(c, bounds, start)
    st = _status()
    kw = dict(start=None if where == "all" else _i32(start), dev_status=st)
    if four:
        sv.cache4_bounds(c["pool"], bounds, c["table"], c["len"], page, **kw)
    else:
        sv.cache_bounds(c["k"], bounds, c["table"], c["len"], **kw)
    assert torch.equal(bounds, want) and int(st) == 0


def test_bounds_of_keys_that_are_not_finite():
    sv = _sv()
    c = _case(2, [20], 1, 2, 2, 16, 8, torch.bfloat16)
    p = int(c["table"][0, 1])
    c["k"][p, 2, 0, 3], c["k"][p, 4, 1, 5], c["k"][int(c["table"][0, 2]), 6, 0, 0] = float("nan"), float("inf"), float("nan")
    bounds = torch.zeros((c["k"].shape[0], 2, 2, 16), dtype=torch.bfloat16, device="cuda")
    sv.cache_bounds(c["k"], bounds, c["table"], c["len"])
    assert torch.isnan(bounds[p, 0, :, 3]).all() and torch.isinf(bounds[p, 1, 1, 5])
    assert int(torch.isnan(bounds).sum()) == 2                         # a position past the length has no part


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page", [(1, 8, 2, 128, 8), (1, 1, 1, 8, 16), (3, 12, 4, 64, 16), (16, 14, 2, 96, 32),
                                             (64, 8, 8, 72, 8), (5, 64, 1, 40, 8), (9, 10, 5, 128, 256)])
def test_scores(N, hq, hkv, D, page, dtype):
    """Sums of 2 D exact products in 32 bits."""
    sv = _sv()
    c = _case(N + D, LENS, N, hq, hkv, D, page, dtype)
    bounds = torch.zeros((c["k"].shape[0], hkv, 2, D), dtype=dtype, device="cuda")
    sv.cache_bounds(c["k"], bounds, c["table"], c["len"])
    count = [N if i % 4 else N // 2 for i in range(len(LENS))]
    st = _status()
    for cnt in (None, count):
        got = sv.page_scores(c["q"], bounds, c["table"], c["len"], page, node_count=None if cnt is None else _i32(cnt),
                             dev_status=st)
        want, mag = _ref_scores(c, bounds, cnt)
        none = torch.isneginf(want)
        assert torch.equal(torch.isneginf(got), none) and int(st) == 0
        err = (got.double() - want).abs()[~none]
        assert (err <= (2 * D + 2) * 2.0 ** -24 * mag[~none] + 1e-30).all()


def test_scores_bound_the_products():
    sv = _sv()
    c = _case(1, [500, 64], 4, 8, 2, 64, 16, torch.bfloat16)
    bounds = torch.zeros((c["k"].shape[0], 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    sv.cache_bounds(c["k"], bounds, c["table"], c["len"])
    got = sv.page_scores(c["q"], bounds, c["table"], c["len"], 16)
    for b, n0 in enumerate(c["lens"]):
        for j in range(n0):
            k = c["k"][int(c["table"][b, j // 16]), j % 16].double()
            top = torch.einsum("nhgd,hd->hng", c["q"][b].double().view(4, 2, 4, 64), k).flatten(1).amax(1)
            assert (top <= got[b, :, j // 16].double() + 1e-3).all()


def test_scores_that_are_not_numbers():
    sv = _sv()
    c = _case(1, [60], 2, 4, 2, 16, 8, torch.float16)
    bounds = torch.zeros((c["k"].shape[0], 2, 2, 16), dtype=torch.float16, device="cuda")
    sv.cache_bounds(c["k"], bounds, c["table"], c["len"])
    bounds[int(c["table"][0, 3]), 1, 0, 2] = float("nan")
    got = sv.page_scores(c["q"], bounds, c["table"], c["len"], 8)
    assert torch.isnan(got[0, 1, 3]) and int(torch.isnan(got).sum()) == 1
    c["q"][0, 1, 0, 4] = float("nan")
    got = sv.page_scores(c["q"], bounds, c["table"], c["len"], 8)
    assert torch.isnan(got[0, 0, :8]).all()


@pytest.mark.parametrize("keep,first,recent,extra", [(1, 0, 1, 0), (2, 1, 1, 0), (5, 1, 1, 9), (8, 3, 2, 1), (40, 0, 1, 17),
                                                     (64, 30, 34, 3), (200, 1, 1, 64)])
@pytest.mark.parametrize("kind", ["normal", "ties", "odd"])
def test_select(keep, first, recent, extra, kind):
    sv = _sv()
    page, H, lens = 8, 3, [0, 1, 8, 9, 100, 333, 800, 801, 1500]
    c = _case(keep, lens, extra + 1, H, H, 8, page, torch.bfloat16, extra_places=0)
    g = torch.Generator(device="cuda").manual_seed(keep)
    scores = torch.randn((len(lens), H, c["table"].shape[1]), generator=g, device="cuda")
    if kind == "ties":
        scores = (scores * 2).round() / 2 * torch.tensor([1.0, 0.0, -1.0], device="cuda").view(1, 3, 1)
    if kind == "odd":
        u = torch.randint(0, 12, scores.shape, generator=g, device="cuda")
        for i, x in enumerate((math.nan, math.inf, -math.inf, -0.0, 0.0, 1e-42, -1e-42)):
            scores = torch.where(u == i, torch.full_like(scores, x), scores)
    st = _status()
    got, kept = sv.page_select(scores, c["table"], c["len"], page, keep, first=first, recent=recent, extra=extra,
                               dev_status=st)
    want, want_len = _ref_select(scores.cpu(), c["table"].cpu(), lens, page, keep, first, recent, extra)
    assert torch.equal(got.cpu(), want) and kept.tolist() == want_len and int(st) == 0


@pytest.mark.parametrize("places", [1024, 1025, 2048, 2049, 8192, 8193, 16384, 16390, 40000])
def test_select_from_many(places):
    sv = _sv()
    page, keep = 8, 333
    n0 = places * page - 3
    table = torch.randperm(places, device="cuda").int().view(1, -1)
    scores = torch.randn((1, 2, places), device="cuda")
    scores[0, 1] = (scores[0, 1] * 3).round()
    got, kept = sv.page_select(scores, table, _i32([n0]), page, keep, extra=2)
    want, want_len = _ref_select(scores.cpu(), table.cpu(), [n0], page, keep, extra=2)
    assert torch.equal(got.cpu(), want) and kept.tolist() == want_len


def test_lengths_out_of_range():
    sv = _sv()
    table = _i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    lens = _i32([-4, 25, 24])
    scores = torch.arange(9, device="cuda", dtype=torch.float32).view(3, 1, 3)
    st = _status()
    got, kept = sv.page_select(scores, table, lens, 8, 2, dev_status=st)
    assert kept.tolist() == [0, 16, 16] and int(st) == sv.DEV_BAD_LEN
    assert got.tolist() == [[[-1, -1]], [[3, 5]], [[6, 8]]]
    k = torch.randn((9, 8, 1, 8), device="cuda").bfloat16()
    bounds = torch.zeros((9, 1, 2, 8), dtype=torch.bfloat16, device="cuda")
    st.zero_()
    sv.cache_bounds(k, bounds, table, lens, dev_status=st)
    assert int(st) == sv.DEV_BAD_LEN and (bounds[:3] == 0).all()
    assert torch.equal(bounds[3:, :, 0], k[3:].amin(1)) and torch.equal(bounds[3:, :, 1], k[3:].amax(1))
    q = torch.ones((3, 1, 1, 8), device="cuda").bfloat16()
    st.zero_()
    got = sv.page_scores(q, bounds, table, lens, 8, dev_status=st)
    assert int(st) == sv.DEV_BAD_LEN and torch.isneginf(got[0]).all() and torch.isfinite(got[1:]).all()
    table[1, 1] = 9
    st.zero_()
    got = sv.page_scores(q, bounds, table, lens, 8, dev_status=st)
    sv.cache_bounds(k, bounds, table, lens, dev_status=st)
    assert int(st) == sv.DEV_BAD_LEN | sv.DEV_BAD_PAGE and torch.isneginf(got[1, 0, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page,hnd", [(1, 8, 2, 128, 16, False), (9, 8, 4, 64, 8, True), (33, 8, 2, 128, 32, False),
                                                 (4, 80, 80, 64, 16, False), (20, 128, 16, 96, 128, False), (3, 6, 3, 72, 256, True)])
def test_attention_over_lists(N, hq, hkv, D, page, hnd, dtype):
    """tree_attention with a list of pages for every key head."""
    sv = _sv()
    lens = [0, 3, 127, 129, 300, 700][:6 if hkv < 16 else 4]
    c = _case(N, lens, N, hq, hkv, D, page, dtype, hnd=hnd)
    g = torch.Generator(device="cuda").manual_seed(9)
    tables = [c["table"]] + [c["table"].gather(1, torch.stack([
        torch.cat([torch.randperm(-(-(n + N) // page), generator=g, device="cuda"),
                   torch.arange(-(-(n + N) // page), c["table"].shape[1], device="cuda")]) for n in lens]))
        for _ in range(hkv - 1)]
    table = torch.stack(tables, 1).contiguous()
    parent = ch.random_parents(g, len(lens), N)
    st = _status()
    for kw in (dict(), dict(window=70, sinks=2)):
        o, l = sv.tree_attention(c["q"], c["k"], c["v"], table, c["len"], parent, return_lse=True, dev_status=st, **kw)
        ref = c4.ref_lists(c["q"], c["k"], c["v"], table, c["len"], parent, **kw)
        ch.check_attention(o, l, ref, dtype, D)
    assert int(st) == 0


def test_lists_that_are_all_alike_change_nothing():
    sv = _sv()
    c = _case(3, [0, 50, 900], 7, 8, 2, 64, 16, torch.bfloat16)
    o, l = sv.tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], return_lse=True)
    table = c["table"].unsqueeze(1).expand(-1, 2, -1).contiguous()
    o2, l2 = sv.tree_attention(c["q"], c["k"], c["v"], table, c["len"], return_lse=True)
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("four", [False, True])
def test_a_step_on_a_cache(four):
    """Two layers of a PagedCache: append, select, attention over the selected pages, commit, and another step whose
    bounds continue from the first; captured and replayed too."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(11)
    layers, slots, hkv, hq, D, page, N, keep = 2, 3, 2, 8, 64, 16, 5, 6
    cls = sv.PagedCache4 if four else sv.PagedCache
    cache = cls(layers, 120, page, hkv, D, slots, 40)
    prompt = [40, 333, 200]
    want = _i32(prompt)
    sv.cache_resize(cache.page_table, cache.page_count, cache.page_ref, want, page)
    for i in range(layers):
        x = torch.randn((slots, 333, 2 * hkv, D), generator=g, device="cuda").bfloat16()
        cache.append(i, x[:, :, :hkv], x[:, :, hkv:], count=want)
    cache.cache_len.copy_(want)
    bounds = [cache.new_bounds() for _ in range(layers)]
    start = torch.zeros_like(want)
    for step in range(2):
        cache.reserve(N)
        for i in range(layers):
            x = torch.randn((slots, N, hq + 2 * hkv, D), generator=g, device="cuda").bfloat16()
            q = x[:, :, :hq]
            cache.append(i, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:])
            pages = cache.select(i, q, bounds[i], keep, start=start, extra=N)
            o, l = cache.attention(i, q, pages=pages, return_lse=True)
            if four:
                k, v = c4.decode(cache.pool[i], page, D)
            else:
                k, v = cache.k[i], cache.v[i]
            lens = cache.cache_len.tolist()
            c = dict(k=k.bfloat16(), table=cache.page_table, lens=lens, page=page)
            every = _ref_bounds(c, torch.zeros_like(bounds[i]), [0] * slots)
            for b, n0 in enumerate(lens):
                used = cache.page_table[b, :-(-n0 // page)].long()
                assert torch.equal(bounds[i][used], every[used])
            scores = sv.page_scores(q, bounds[i], cache.page_table, cache.cache_len, page)
            want_table, want_len = _ref_select(scores.cpu(), cache.page_table.cpu(), lens, page, keep, extra=N)
            assert torch.equal(pages[0].cpu(), want_table) and pages[1].tolist() == want_len
            ch.check_attention(o, l, c4.ref_lists(q, k, v, pages[0], pages[1], None), torch.bfloat16, D)
        start = cache.cache_len.clone()
        cache.commit(None, _i32([2, 0, 4]), nodes=N)
        cache.trim()
    cache.reserve(N)
    cache.append(0, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:])         # (what the drafted positions hold is read)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pages = cache.select(0, q, bounds[0], keep, start=start, extra=N)
        o = cache.attention(0, q, pages=pages)
    eager = cache.attention(0, q, pages=cache.select(0, q, bounds[0], keep, start=start, extra=N))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager) and int(cache.status) == 0
