"""Page operators of the paged cache against plain Python bookkeeping: integers
and moved bytes have to be equal."""
import random

import pytest
import torch

import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _sv():
    import speculative_decoding_verification_69_gb300 as sv
    return sv


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("slots,pages,page,P", [(1, 1, 8, 1), (3, 40, 8, 20), (33, 500, 16, 30), (1000, 9000, 64, 12),
                                                (8192, 70000, 8, 9), (5, 300001, 16, 70000)])
def test_resize_random_walk(slots, pages, page, P):
    sv = _sv()
    r = random.Random(slots + pages)
    table, count = torch.full((slots, P), -1, dtype=torch.int32, device="cuda"), torch.zeros(slots, dtype=torch.int32,
                                                                                          device="cuda")
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    model = ch.Pages(table.cpu(), count.cpu(), ref.cpu())
    for step in range(12):
        top = [1, 2 * pages * page // slots, pages * page // slots][step % 3]
        want = [r.choice([-1, 0, r.randint(0, max(1, top)), r.randint(0, max(1, top))]) for _ in range(slots)]
        extra = r.choice([0, 1, 9, page])
        st = _status()
        sv.cache_resize(table, count, ref, _i32(want), page, extra=extra, dev_status=st)
        torch.cuda.synchronize()
        missed = model.resize(want, extra, page)
        assert int(st.item()) == (sv.DEV_NO_PAGES if missed else 0)
        model.check(table.cpu(), count.cpu(), ref.cpu())


@pytest.mark.parametrize("slots,pages,page", [(3, 40, 8), (33, 500, 16), (1000, 9000, 64)])
def test_resize_with_too_few_pages(slots, pages, page):
    """Every slot asks for twice its share: those served come first, the others
    keep what they had, and after some are freed the rest are served."""
    sv = _sv()
    P = 2 * pages // slots + 1
    table, count = _i32([[-1] * P] * slots), _i32([0] * slots)
    ref = _i32([0] * pages)
    model = ch.Pages(table.cpu(), count.cpu(), ref.cpu())
    first = [page] * slots
    double = [2 * pages * page // slots] * slots
    for want, missed in ((first, False), (double, True), ([-1 if i % 2 else 0 for i in range(slots)], False),
                         ([-1 if i % 2 == 0 else 5 * page for i in range(slots)], None), (double, True)):
        st = _status()
        sv.cache_resize(table, count, ref, _i32(want), page, dev_status=st)
        got = model.resize(want, 0, page)
        assert missed is None or got == missed
        assert int(st.item()) == (sv.DEV_NO_PAGES if got else 0)
        model.check(table.cpu(), count.cpu(), ref.cpu())


def test_resize_huge_wants():
    """Lengths near 2^31 need no more than max_pages, and sums of needs do not wrap."""
    sv = _sv()
    slots, pages, P = 4096, 64, 1 << 15
    table = torch.full((slots, P), -1, dtype=torch.int32, device="cuda")
    count, ref = torch.zeros(slots, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    st = _status()
    sv.cache_resize(table, count, ref, _i32([2 ** 31 - 1] * slots), 8, extra=2 ** 31 - 1, dev_status=st)
    assert int(st.item()) == sv.DEV_NO_PAGES and int(count.sum()) == 0 and int(ref.sum()) == 0
    want = [-1] * slots
    want[-1] = 64 * 8
    st.zero_()
    sv.cache_resize(table, count, ref, _i32(want), 8, dev_status=st)
    assert int(st.item()) == 0 and table[-1, :64].tolist() == list(range(64))


def test_resize_bad_pages():
    """A held page outside the pool, or one that nobody counted, is reported."""
    sv = _sv()
    table = _i32([[3, 99, -7, 1]])
    count, ref = _i32([4]), _i32([0, 0, 0, 1])
    st = _status()
    sv.cache_resize(table, count, ref, _i32([0]), 8, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_PAGE
    assert ref.tolist() == [0, 0, 0, 0] and count.tolist() == [0] and table.tolist() == [[-1] * 4]


@pytest.mark.parametrize("layers,heads,D,page,dtype,hnd", [(1, 1, 8, 8, torch.float32, False),
                                                           (3, 2, 64, 16, torch.bfloat16, True),
                                                           (2, 16, 96, 32, torch.float16, False),
                                                           (2, 40, 128, 8, torch.float32, False),
                                                           (5, 8, 128, 128, torch.bfloat16, False)])
@pytest.mark.parametrize("tight", [False, True])
def test_fork(layers, heads, D, page, dtype, hnd, tight):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(page + heads)
    lens = [0, 1, page - 1, page, page + 1, 5 * page + 3, 3 * page, 7]
    slots, P = 24, 8
    lens += [9, 2 * page] + [0] * (slots - 10)
    pages = sum(-(-n // page) for n in lens) + (2 if tight else 30)
    table, count, ref, cl = ch.make_table(g, lens, 0, page, P, pages)
    k = ch.make_pool(g, pages, page, heads, D, dtype, layers=layers, hnd=hnd)
    v = ch.make_pool(g, pages, page, heads, D, dtype, layers=layers, hnd=hnd)
    # slot 9 held pages before; void forks: a dst that is a source, a dst used twice, slots out of range
    src = [0, 1, 2, 3, 4, 5, 5, 5, 6, 5, 4, 99, 2, -1, 7]
    dst = [10, 11, 12, 13, 14, 15, 16, 9, 17, 7, 14, 18, 2 ** 30, 19, 20]
    for rep in range(2):  # the second time the destinations give back what they got
        model = ch.Pages(table.cpu(), count.cpu(), ref.cpu(), cl.cpu())
        ek, ev = k.clone(), v.clone()
        st = _status()
        sv.cache_fork(k, v, table, count, ref, cl, _i32(src), _i32(dst), dev_status=st)
        torch.cuda.synchronize()
        copies, missed = model.fork(src, dst, page)
        for a, b, n in copies:
            ek[:, b, :n] = ek[:, a, :n]
            ev[:, b, :n] = ev[:, a, :n]
        model.check(table.cpu(), count.cpu(), ref.cpu(), cl.cpu())
        assert torch.equal(k, ek) and torch.equal(v, ev)
        assert int(st.item()) & ~sv.DEV_NO_PAGES == sv.DEV_BAD_SLOT
        assert (int(st.item()) & sv.DEV_NO_PAGES != 0) == missed == tight
    if not tight:
        assert len(copies) >= 7


def test_fork_of_a_slot_without_its_pages():
    sv = _sv()
    k = torch.zeros((1, 8, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    table, count, ref, cl = _i32([[0, 1], [2, -1], [-1, -1]]), _i32([2, 1, 0]), _i32([1, 1, 1, 0, 0, 0, 0, 0]), _i32(
        [17, 8, 0])
    before = [x.clone() for x in (table, count, ref, cl)]
    st = _status()
    sv.cache_fork(k, k.clone(), table, count, ref, cl, _i32([0]), _i32([2]), dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_LEN
    assert all(torch.equal(a, b) for a, b in zip(before, (table, count, ref, cl)))


@pytest.mark.parametrize("dtype,hnd", [(torch.bfloat16, False), (torch.float32, True)])
def test_copy_pages(dtype, hnd):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(3)
    k = ch.make_pool(g, 20, 32, 3, 40, dtype, layers=4, hnd=hnd)
    v = ch.make_pool(g, 20, 32, 3, 40, dtype, layers=4, hnd=hnd)
    ek, ev = k.clone(), v.clone()
    src, dst = [0, 0, 5, -1, 7, 3], [1, 2, 19, 4, 20, 6]
    st = _status()
    sv.cache_copy(k, v, _i32(src), _i32(dst), dev_status=st)
    for a, b in ((0, 1), (0, 2), (5, 19), (3, 6)):
        ek[:, b], ev[:, b] = ek[:, a], ev[:, a]
    assert torch.equal(k, ek) and torch.equal(v, ev) and int(st.item()) == sv.DEV_BAD_PAGE


@pytest.mark.parametrize("N,heads,D,page,dtype,hnd", [(1, 1, 8, 8, torch.float32, False),
                                                      (9, 8, 128, 16, torch.bfloat16, False),
                                                      (200, 3, 72, 32, torch.float16, True),
                                                      (64, 40, 128, 64, torch.bfloat16, False)])
def test_append(N, heads, D, page, dtype, hnd):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(N)
    lens = [0, 1, page - 1, page, 3 * page + 5]
    pages = sum(-(-(n + N) // page) for n in lens) + 2
    P = max(-(-(n + N) // page) for n in lens)
    table, count, ref, cl = ch.make_table(g, lens, N, page, P, pages)
    k = ch.make_pool(g, pages, page, heads, D, dtype, hnd=hnd)
    v = ch.make_pool(g, pages, page, heads, D, dtype, hnd=hnd)
    kv = torch.randn((5, N, 2 * heads + 1, D), generator=g, device="cuda").to(dtype)
    kn, vn = kv[:, :, :heads], kv[:, :, heads + 1:]
    for cnt in (None, [N, 0, N + 7, -3, (N + 1) // 2]):
        ek, ev = k.clone(), v.clone()
        for b, n0 in enumerate(lens):
            m = N if cnt is None else max(0, min(N, cnt[b]))
            for n in range(m):
                p = int(table[b, (n0 + n) // page])
                ek[p, (n0 + n) % page], ev[p, (n0 + n) % page] = kn[b, n], vn[b, n]
        st = _status()
        sv.cache_append(k, v, table, cl, kn, vn, count=None if cnt is None else _i32(cnt), dev_status=st)
        assert torch.equal(k, ek) and torch.equal(v, ev) and int(st.item()) == 0
        kv.mul_(-1)


def test_append_reports_what_it_skips():
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.zeros((6, 8, 2, 8), device="cuda"), torch.zeros((6, 8, 2, 8), device="cuda")
    kn = torch.randn((3, 10, 2, 8), generator=g, device="cuda")
    st = _status()
    sv.cache_append(k, v, _i32([[0, 1], [2, 77], [-1, 3]]), _i32([9, 3, 0]), kn, kn, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_LEN | sv.DEV_BAD_PAGE
    e = torch.zeros_like(k)
    e[1, 1:8] = kn[0, :7]              # the rest of request 0 is past its row
    e[2, 3:8] = kn[1, :5]              # page 77 is none
    e[3, 0:2] = kn[2, 8:]              # page -1 is none
    assert torch.equal(k, e) and torch.equal(v, e)
    st.zero_()
    sv.cache_append(k, v, _i32([[0, 1], [2, 4], [5, 3]]), _i32([-1, 2 ** 31 - 3, 16]), kn, kn, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_LEN and torch.equal(k, e)


def _paths(r, B, N):
    out = []
    for _ in range(B):
        par = [-1] + [n - 1 if r.random() < 0.5 else r.randrange(n) for n in range(1, N)]
        n, p = r.randrange(N), []
        while n > 0:
            p.append(n)
            n = par[n]
        out.append(p[::-1])
    return out


@pytest.mark.parametrize("layers,heads,D,page,dtype,hnd", [(1, 1, 8, 8, torch.float32, False),
                                                           (3, 2, 64, 16, torch.bfloat16, True),
                                                           (2, 16, 96, 32, torch.float16, False),
                                                           (2, 40, 128, 8, torch.float32, False),
                                                           (5, 8, 128, 64, torch.bfloat16, False)])
@pytest.mark.parametrize("N", [1, 2, 9, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(layers, heads, D, page, dtype, hnd, N, in_place):
    sv = _sv()
    r = random.Random(N * 100 + page)
    g = torch.Generator(device="cuda").manual_seed(page + heads)
    B = 9
    lens = [r.choice([0, page - 1, page, r.randint(0, 3 * page)]) for _ in range(B)]
    pages = sum(-(-(n + N) // page) for n in lens) + 2
    P = max(-(-(n + N) // page) for n in lens)
    table, count, ref, cl = ch.make_table(g, lens, N, page, P, pages)
    k = ch.make_pool(g, pages, page, heads, D, dtype, layers=layers, hnd=hnd)
    v = ch.make_pool(g, pages, page, heads, D, dtype, layers=layers, hnd=hnd)
    paths = _paths(r, B, N)
    paths[0], paths[1] = list(range(1, N)), list(range(1, N))[-1:]      # all in place; the last node alone
    nodes = _i32([p + [-1] * (N - len(p)) for p in paths])
    acc = _i32([len(p) for p in paths])
    ek, ev = k.clone(), v.clone()
    for b, p in enumerate(paths):
        for i, n in enumerate(p):
            a, z = lens[b] + n, lens[b] + 1 + i
            fa, fz = int(table[b, a // page]), int(table[b, z // page])
            ek[:, fz, z % page] = k[:, fa, a % page]
            ev[:, fz, z % page] = v[:, fa, a % page]
    st = _status()
    new = None if in_place else torch.empty_like(cl)
    got = sv.cache_commit(k, v, table, cl, nodes, acc, new_len=new, dev_status=st)
    torch.cuda.synchronize()
    assert got is (cl if in_place else new)
    assert got.tolist() == [n + 1 + len(p) for n, p in zip(lens, paths)]
    if not in_place:
        assert cl.tolist() == lens
    assert torch.equal(k, ek) and torch.equal(v, ev) and int(st.item()) == 0


def test_commit_of_linear_drafts():
    sv = _sv()
    k = torch.zeros((2, 4, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    table, cl, acc = _i32([[0], [1], [2]]), _i32([3, 0, 5]), _i32([0, 4, 9])
    assert sv.cache_commit(k, k, table, cl, None, acc, nodes=5).tolist() == [4, 5, 10]
    new = torch.empty_like(cl)
    assert sv.cache_commit(k, k, table, cl, None, acc, nodes=9, new_len=new).tolist() == [5, 10, 19]
    assert cl.tolist() == [4, 5, 10]


@pytest.mark.parametrize("in_place", [False, True])
def test_commit_cuts_bad_paths(in_place):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn((2, 8, 8, 2, 8), generator=g, device="cuda")
    v = torch.randn((2, 8, 8, 2, 8), generator=g, device="cuda")
    table, cl = _i32([[0, 1], [2, 3], [4, 50], [6, 7]]), _i32([0, 2, 5, 13])
    nodes = _i32([[2, 1, 3, 4, 5, -1], [3, 9, -1, -1, -1, -1], [1, 4, 5, -1, -1, -1], [2, 3, -1, -1, -1, -1]])
    acc = _i32([5, 2, 3, 2])
    ek, ev = k.clone(), v.clone()
    for e, x in ((ek, k), (ev, v)):
        e[:, 0, 1] = x[:, 0, 2]            # request 0: node 1 cannot be the second of a path
        e[:, 2, 3] = x[:, 2, 5]            # request 1: node 9 of 6
        # request 2: node 1 is in place, node 4 lies in page 50
        e[:, 7, 6] = x[:, 7, 7]            # request 3: node 2 moves, node 3 is past the table
    st = _status()
    got = sv.cache_commit(k, v, table, cl, nodes, acc, new_len=None if in_place else torch.empty_like(cl), dev_status=st)
    assert got.tolist() == [2, 4, 7, 15]
    assert int(st.item()) == sv.DEV_BAD_TREE | sv.DEV_BAD_PAGE
    assert torch.equal(k, ek) and torch.equal(v, ev)


def test_pools_past_32_bit_offsets():
    """Pages whose elements lie past 2^31 are written, moved and copied where they are."""
    sv = _sv()
    page, heads, D = 64, 8, 128
    pages = (1 << 31) // (page * heads * D) + 9
    k = torch.empty((1, pages, page, heads, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    a, b = pages - 1, pages - 3
    g = torch.Generator(device="cuda").manual_seed(3)
    kn = torch.randn((1, 20, heads, D), generator=g, device="cuda").bfloat16()
    table, cl = _i32([[a, b, -1]]), _i32([60])
    sv.cache_append(k[0], v[0], table, cl, kn, -kn)
    assert torch.equal(k[0, a, 60:], kn[0, :4]) and torch.equal(v[0, b, :16], -kn[0, 4:])
    nodes = _i32([[3, 10, 19] + [-1] * 17])
    sv.cache_commit(k, v, table, cl, nodes, _i32([3]))
    assert torch.equal(k[0, a, 61:], kn[0, [3, 10, 19]]) and torch.equal(v[0, a, 61:], -kn[0, [3, 10, 19]])
    sv.cache_copy(k, v, _i32([a]), _i32([0]))
    assert torch.equal(k[:, 0], k[:, a]) and torch.equal(v[:, 0], v[:, a])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("linear", [False, True])
def test_commit_stops_where_pages_end(linear, in_place):
    """Neither a tree's path nor linear drafts are kept past the slot's pages, and a
    root without a page leaves the length alone."""
    sv = _sv()
    k = torch.randn((2, 6, 8, 1, 8), device="cuda")
    v = torch.randn_like(k)
    ek, ev = k.clone(), v.clone()
    table = _i32([[0, -1, -1], [-1, -1, -1], [1, -1, -1], [2, 6, -1], [3, -1, 4], [5, -1, -1]])
    lens, acc = [6, 0, 8, 5, 7, 3], _i32([3, 2, 0, 3, 3, 1])
    nodes = None if linear else _i32([[1, 2, 3, -1]] * 6)
    new = None if in_place else torch.full((6,), -9, dtype=torch.int32, device="cuda")
    st = _status()
    got = sv.cache_commit(k, v, table, _i32(lens), nodes, acc, new_len=new, nodes=4, dev_status=st)
    assert got.tolist() == [8, 0, 8, 8, 8, 5]
    assert int(st) == sv.DEV_BAD_PAGE
    assert torch.equal(k, ek) and torch.equal(v, ev)
    st.zero_()
    got = sv.cache_commit(k, v, table, _i32([-3, 2, 0, 0, 0, 0]), nodes, acc, new_len=new, nodes=4, dev_status=st)
    assert got.tolist()[:2] == [-3, 2] and int(st) == sv.DEV_BAD_PAGE | sv.DEV_BAD_LEN


def test_linear_drafts_past_the_row_are_reported():
    sv = _sv()
    k = torch.zeros((1, 4, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    for new in (None, _i32([0, 0])):
        st = _status()
        got = sv.cache_commit(k, k, _i32([[0], [1]]), _i32([3, 2 ** 31 - 3]), None, _i32([4, 4]), nodes=5, new_len=new,
                              dev_status=st)
        assert got.tolist() == [8, 2 ** 31 - 1] and int(st) == sv.DEV_BAD_LEN
        st.zero_()
        got = sv.cache_commit(k, k, _i32([[0], [1]]), _i32([3, 6]), None, _i32([4, 4]), nodes=5, new_len=new,
                              dev_status=st)
        assert got.tolist() == [8, 11] and int(st) == sv.DEV_BAD_LEN


@pytest.mark.parametrize("linear", [False, True])
def test_a_slot_without_pages_for_its_step_loses_nothing(linear):
    """While a third request holds the pages, one slot gets none for its step: its
    length stays at what was written, and it goes on from there when there are some."""
    sv = _sv()
    c = sv.PagedCache(1, 6, 8, 1, 8, 3, 4, dtype=torch.bfloat16)
    c.k.fill_(7.0)
    c.v.fill_(7.0)
    N = 6
    kv = torch.randn((3, 8, 1, 8), device="cuda").bfloat16()

    def resize(want):
        sv.cache_resize(c.page_table, c.page_count, c.page_ref, _i32(want), 8, dev_status=c.status)

    def append(n):
        c.append(0, kv[:, :n], kv[:, :n], count=_i32([n, n, 0]))

    def commit(nodes, accept):
        c.commit(nodes, _i32(accept + [0]), nodes=N)
        c.cache_len[2] = 0  # the third request does not take part

    path = None if linear else _i32([[1, 2, 3, 4, 5, -1]] * 3)
    resize([8, 8, 24])
    append(8)
    c.cache_len[:2] = 8
    resize([14, 14, -1])
    assert int(c.status) == sv.DEV_NO_PAGES and c.page_count.tolist() == [2, 1, 3]
    c.status.zero_()
    append(N)
    commit(path, [5, 5])
    assert int(c.status) == sv.DEV_BAD_PAGE and c.cache_len.tolist() == [14, 8, 0]
    c.status.zero_()
    c.trim()  # the third request is done
    assert int(c.status) == 0 and c.page_count.tolist() == [2, 1, 0]
    c.reserve(N)
    append(N)
    commit(path, [1, 5])
    assert int(c.status) == 0 and c.cache_len.tolist() == [16, 14, 0]
    for b, want in ((0, [kv[0], kv[0, :N], kv[0, :2]]), (1, [kv[1], kv[1, :N]])):
        want = torch.cat(want)
        at = torch.arange(len(want), device="cuda")
        pages = c.page_table[b].long()[at // 8]
        assert torch.equal(c.k[0, pages, at % 8], want) and torch.equal(c.v[0, pages, at % 8], want)


def test_tensors_that_require_a_gradient_are_refused():
    """There is no backward pass: instead of a result cut off from the graph, an error."""
    sv = _sv()
    k = torch.randn((1, 4, 8, 1, 8), device="cuda").bfloat16()
    v = k.clone()
    table, one = _i32([[0, 1]]), _i32([1])
    count, ref, zero = _i32([2]), _i32([1, 1, 0, 0]), _i32([0])
    new = torch.randn((1, 2, 1, 8), device="cuda").bfloat16()

    def grad(t):
        return t.detach().clone().requires_grad_(True)
    calls = [lambda k, v, x: sv.tree_attention(x, k[0], v[0], table, one),
             lambda k, v, x: sv.cache_append(k[0], v[0], table, one, x, x),
             lambda k, v, x: sv.cache_append(k[0], v[0], table, one, new, x),
             lambda k, v, x: sv.cache_commit(k, v, table, one.clone(), _i32([[1, -1]]), one),
             lambda k, v, x: sv.cache_copy(k, v, zero, _i32([3])),
             lambda k, v, x: sv.cache_fork(k, v, table, count, ref, one, zero, _i32([5]))]
    for i, call in enumerate(calls):
        for args in ((grad(k), v, new), (k, grad(v), new)) + (((k, v, grad(new)),) if i < 3 else ()):
            with pytest.raises(ValueError, match="gradient"):
                call(*args)
            with torch.no_grad():
                call(*args)
        call(k, v, new)
    out = sv.tree_attention(new.detach(), k[0], v[0], table, one)
    with torch.no_grad():
        assert torch.equal(sv.tree_attention(grad(new), k[0], v[0], table, one), out)


def test_an_output_that_requires_a_gradient_is_refused():
    sv = _sv()
    k = torch.randn((2, 8, 1, 8), device="cuda").bfloat16()
    q = torch.randn((1, 2, 1, 8), device="cuda").bfloat16()
    out = torch.zeros_like(q).requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        sv.tree_attention(q, k, k, _i32([[0, 1]]), _i32([1]), out=out)
    with torch.no_grad():
        assert sv.tree_attention(q, k, k, _i32([[0, 1]]), _i32([1]), out=out).data_ptr() == out.data_ptr()
