"""Steps that attend to selected pages, through the caches' own calls."""
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


def _cache(four, lens, N, seed, hkv=2, D=64, page=16, max_pages=40):
    """A cache of one layer whose slots hold prompts of these lengths, and have pages for N tokens more."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = (sv.PagedCache4 if four else sv.PagedCache)(1, 150, page, hkv, D, len(lens), max_pages)
    want = _i32(lens)
    sv.cache_resize(cache.page_table, cache.page_count, cache.page_ref, want, page, extra=N, dev_status=cache.status)
    x = torch.randn((len(lens), max(lens), 2 * hkv, D), generator=g, device="cuda").bfloat16()
    cache.append(0, x[:, :, :hkv], x[:, :, hkv:], count=want)
    cache.cache_len.copy_(want)
    x = torch.randn((len(lens), N, 8 + 2 * hkv, D), generator=g, device="cuda").bfloat16()
    cache.append(0, x[:, :, 8:8 + hkv], x[:, :, 8 + hkv:])
    return cache, x[:, :, :8], g


def _numbers(cache, four, D=64, page=16):
    k, v = c4.decode(cache.pool[0], page, D) if four else (cache.k[0], cache.v[0])
    return k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("N", [1, 3, 20])
def test_the_pages_of_the_nodes_follow_the_selected_ones(N, four):
    """Lengths at the end of a page, below and above `keep` pages: the nodes see themselves without being asked for."""
    keep = 4
    cache, q, g = _cache(four, [0, 16, 30, 64, 96, 320, 333], N, 3 + N)
    for cls_kw in (dict(), dict(extra=N)):
        pages = cache.select(0, q, cache.new_bounds(), keep, **cls_kw)
        assert pages[0].shape[2] == keep + -(-N // 16)
        parent = ch.random_parents(g, 7, N)
        o, l = cache.attention(0, q, parent, pages=pages, return_lse=True)
        assert int(cache.status) == 0
        k, v = _numbers(cache, four)
        ch.check_attention(o, l, c4.ref_lists(q, k, v, *pages, parent), torch.bfloat16, 64)
    none = cache.select(0, q, cache.new_bounds(), keep, extra=0)       # pages for no node, when that is asked for
    assert none[0].shape[2] == keep and torch.equal(none[1], pages[1])


@pytest.mark.parametrize("four", [False, True])
def test_rows_past_the_node_counts_have_no_say(four):
    """Rows past a request's count hold NaN: its lists are those of the rows before."""
    N, keep, cnt = 5, 4, _i32([5, 1, 3, 2])
    cache, q, _ = _cache(four, [200, 320, 333, 100], N, 8)
    past = torch.arange(N, device="cuda").view(1, N, 1, 1) >= cnt.view(4, 1, 1, 1)
    alike = torch.where(past, q[:, :1], q)                             # in their place the first row once more
    want = cache.select(0, alike, cache.new_bounds(), keep)
    other = cache.select(0, q, cache.new_bounds(), keep)
    got = cache.select(0, torch.where(past, torch.full_like(q, float("nan")), q), cache.new_bounds(), keep,
                       node_count=cnt)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not torch.equal(other[0], want[0])                          # (they would have had one)
    o = cache.attention(0, torch.where(past, torch.full_like(q, float("nan")), q), pages=got, node_count=cnt)
    ref = cache.attention(0, alike, pages=want, node_count=cnt)
    assert torch.equal(o, ref) and torch.isfinite(o).all() and int(cache.status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page", [(1, 8, 2, 128, 16), (9, 12, 3, 64, 8), (40, 8, 2, 80, 16), (6, 16, 16, 32, 128)])
@pytest.mark.parametrize("window,sinks,counts", [(70, 2, False), (0, 0, True), (130, 0, True), (7, 140, True)])
def test_lists_in_4_bits_with_windows_and_counts(window, sinks, counts, N, hq, hkv, D, page, dtype):
    """Windows and sinks count the positions of the lists."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(N * 7 + window)
    lens = [0, 3, 127, 129, 300, 700]
    P = max(-(-(n + N) // page) for n in lens) + 1
    pages = sum(-(-(n + N) // page) for n in lens) + 3
    table = torch.stack([ch.make_table(g, lens, N, page, P, pages)[0] for _ in range(hkv)], 1).contiguous()
    pool = c4.make_pool(g, pages, hkv, page, D)
    q = (torch.randn((len(lens), N, hq, D), generator=g, device="cuda") * 2).to(dtype)
    parent, cl, st = ch.random_parents(g, len(lens), N), _i32(lens), _i32([0])
    kw = dict(window=window, sinks=sinks, node_count=_i32([N, 1, 0, N, N // 2, N]) if counts else None)
    o, l = sv.tree_attention4(q, pool, table, cl, page, parent, return_lse=True, dev_status=st, **kw)
    ch.check_attention(o, l, c4.ref_attention(q, pool, page, table, cl, parent, **kw), dtype, D)
    assert int(st) == 0


@pytest.mark.parametrize("four", [False, True])
def test_a_selection_on_a_stream_that_is_given(four):
    """Every call of it behind the work that its stream has to do, with the results of the current stream."""
    sv = _sv()
    cache, q, _ = _cache(four, [200, 320, 0, 100], 2, 9)
    bounds = cache.new_bounds()
    want = cache.select(0, q, bounds, 4)
    scores = sv.page_scores(q, bounds, cache.page_table, cache.cache_len, 16)
    s = torch.cuda.Stream()
    late, x = torch.zeros_like(bounds), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                                  # about 10 ms
        x.copy_(q)
    got = cache.select(0, x, late, 4, stream=s)
    again = sv.page_scores(x, late, cache.page_table, cache.cache_len, 16, stream=s)
    table, length = sv.page_select(again, cache.page_table, cache.cache_len, 16, 4, extra=2, stream=s)
    s.synchronize()
    assert torch.equal(late, bounds) and torch.equal(again, scores)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(table, want[0]) and torch.equal(length, want[1]) and int(cache.status) == 0


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("N,hq,hkv,D,page,slots", [
    (1, 8, 2, 128, 16, 4),       # a stream's keys
    (5, 16, 8, 64, 8, 24),       # heads in pairs
    (3, 12, 3, 64, 32, 4),       # an odd one left
    (40, 16, 2, 96, 64, 3),      # many rows
    (2, 40, 40, 72, 16, 6),
])
def test_lists_of_pages_in_another_order_change_nothing(N, hq, hkv, D, page, slots, four):
    """Each head's pages moved to other places of the pool and listed there, in 16 bits with values and keys that are
    not finite at the nodes of a branch: the same bits as with one table for all heads."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(N + D)
    lens = [(7, 300, 0, 133)[b % 4] + b for b in range(slots)]
    P = -(-(max(lens) + N) // page)
    pages = slots * P + 2
    table, _, _, cl = ch.make_table(g, lens, N, page, P, pages)
    q = torch.randn((slots, N, hq, D), generator=g, device="cuda").bfloat16()
    parent = ch.random_parents(g, slots, N)
    if four:
        pools = [c4.make_pool(g, pages, hkv, page, D)]
    else:
        pools = [torch.randn((pages, page, hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
        for b in range(0, slots, 2):
            at = lens[b] + N - 1
            pools[1][int(table[b, at // page]), at % page, b % hkv, 3] = (float("inf"), float("nan"))[b // 2 % 2]
            if N > 2:
                at -= 1
                pools[0][int(table[b, at // page]), at % page, (b + 1) % hkv, 5] = float("nan")
    moved = [p.clone() for p in pools]
    lists = table.unsqueeze(1).repeat(1, hkv, 1)
    for h in range(hkv):
        perm = torch.randperm(pages, generator=g, device="cuda")
        for p, m in zip(pools, moved):
            if four:
                m[perm, h] = p[:, h]
            else:
                m[perm, :, h] = p[:, :, h]
        held = lists[:, h] >= 0
        lists[:, h][held] = perm[lists[:, h][held].long()].int()
    st = _i32([0])
    for kw in (dict(), dict(window=100, sinks=3), dict(node_count=_i32([N - b % 2 for b in range(slots)]))):
        kw.update(return_lse=True, dev_status=st)
        if four:
            a = sv.tree_attention4(q, pools[0], table, cl, page, parent, **kw)
            b = sv.tree_attention4(q, moved[0], lists, cl, page, parent, **kw)
        else:
            a = sv.tree_attention(q, *pools, table, cl, parent, **kw)
            b = sv.tree_attention(q, *moved, lists, cl, parent, **kw)
        for x, y in zip(a, b):
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
    assert int(st) == 0
