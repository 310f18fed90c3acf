"""The 4-bit cache: writing, reading back, committing, copying and forking, against the format in 64 bits."""
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


def _slots(g, lens, N, page, spare=3):
    P = max(-(-(n + N) // page) for n in lens) + 1
    pages = sum(-(-(n + N) // page) for n in lens) + spare
    table, count, ref, cl = ch.make_table(g, lens, N, page, P, pages)
    return table, count, ref, cl, pages


LENS = [0, 1, 5, 7, 8, 9, 63, 64, 65, 100, 127, 128, 129, 250]


def _at(table, page, b, pos):
    pos = torch.tensor(pos, device=table.device)
    return table[b].long()[pos // page], pos % page


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,heads,D,page", [(1, 1, 8, 8), (1, 8, 128, 16), (9, 2, 64, 16), (13, 3, 80, 8), (7, 5, 96, 32),
                                            (40, 1, 24, 256), (130, 2, 128, 128), (300, 16, 128, 64), (17, 33, 72, 16)])
def test_append_and_read(N, heads, D, page, dtype):
    """Every byte of the pool is what the format says; what is not written stays."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(N * 7 + D)
    table, _, _, cl, pages = _slots(g, LENS, N, page)
    B = len(LENS)
    pool = c4.make_pool(g, pages, heads, page, D)
    before = pool.clone()
    kv = (torch.randn((B, N, 2 * heads, D), generator=g, device="cuda") * 3).to(dtype)
    kn, vn = kv[:, :, :heads], kv[:, :, heads:]                       # a fused projection's slices
    count = _i32([N if b % 3 else N // 2 for b in range(B)])
    st = _status()
    sv.cache4_append(pool, table, cl, kn, vn, page, count=count, dev_status=st)
    want = before.cpu()
    for x, kind in ((kn, "k"), (vn, "v")):
        at, shift, sc = c4.places(page, c4.channels(D), kind)
        code, byte = (y.cpu() for y in c4.kept(x))
        for b, n0 in enumerate(LENS):
            for n in range(int(count[b])):
                p, t = int(table[b, (n0 + n) // page]), (n0 + n) % page
                row = want[p].to(torch.int64)
                for c in range(2):  # both nibbles of a byte
                    m = shift[t] == 4 * c
                    row[:, at[t][m]] = (row[:, at[t][m]] & (240 if c == 0 else 15)) | (code[b, n][:, m] << (4 * c))
                row[:, sc[t]] = byte[b, n]
                want[p] = row.to(torch.uint8)
    assert torch.equal(pool.cpu(), want)
    k, v = sv.cache4_read(pool, table, cl, N, page, D, count=count, dtype=dtype, dev_status=st)
    for got, x in ((k, kn), (v, vn)):
        ref = c4.values(x)
        for b in range(B):
            c = int(count[b])
            assert torch.equal(got[b, :c].double(), ref[b, :c]) and (got[b, c:] == 0).all()
    assert int(st) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounding(dtype):
    """Ties of scales and of codes, subnormal numbers, groups of zeros, the ends of the scales' range."""
    sv = _sv()
    D, page = 64, 16
    s = [2.0 ** -19, 2.0 ** -10, 1.0, 1.125, 1.375, 1.875] + ([7680.0] if dtype == torch.bfloat16 else [5120.0])
    rows = []
    for x in s:
        half = [(i - 15.5) / 2.0 for i in range(32)]                  # codes in the middle, up to 7.75
        rows.append([7.0 * x] + [h * x for h in half[1:]] + [7.0 * x, -7.0 * x] + [i * x / 4.0 for i in range(30)])
    for t in range(16, 32):                                           # amax / 7 in the middle between two scales
        rows.append([7.0 * (t + 0.5) / 16.0 * 2.0 ** -3] + [0.0] * 31 + [7.0 * (t + 0.25) / 16.0] + [0.1] * 31)
    rows += [[0.0] * 64, [2.0 ** -24] * 64, [2.0 ** -17] * 32 + [-2.0 ** -16] * 32, [-65504.0] * 32 + [60000.0, 1.0] * 16]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda().view(1, len(rows), 1, D)
    pool = torch.full((4, 1, c4.page_bytes(page, D)), 255, dtype=torch.uint8, device="cuda")
    table, zero = _i32([[2, 0, 3]]), _i32([0])
    st = _status()
    sv.cache4_append(pool, table, zero, x, -x, page, dev_status=st)
    k, v = sv.cache4_read(pool, table, zero, len(rows), page, D, dtype=dtype)
    assert torch.equal(k.double(), c4.values(x)) and torch.equal(v.double(), c4.values(-x)) and int(st) == 0


def test_values_that_are_not_finite():
    """A NaN is kept as 0 and an infinity as the largest number of its sign; both are reported."""
    sv = _sv()
    inf, nan = float("inf"), float("nan")
    for value, want in ((nan, 0.0), (inf, 7.0 * 7680.0), (-inf, -8.0 * 7680.0)):
        x = torch.ones((1, 1, 1, 32), device="cuda", dtype=torch.bfloat16)
        y = x.clone()
        y[..., 3] = value
        for kn, vn in ((x, y), (y, x)):
            pool = torch.zeros((1, 1, c4.page_bytes(8, 32)), dtype=torch.uint8, device="cuda")
            st = _status()
            sv.cache4_append(pool, _i32([[0]]), _i32([0]), kn, vn, 8, dev_status=st)
            assert int(st) == sv.DEV_BAD_VALUE
            k, v = sv.cache4_read(pool, _i32([[0]]), _i32([0]), 1, 8, 32)
            assert float((v if kn is x else k)[..., 3]) == torch.tensor(want).bfloat16()
            assert torch.isfinite(k).all() and torch.isfinite(v).all()


@pytest.mark.parametrize("byte", range(0, 256, 5))
def test_every_byte_stands_for_a_finite_number(byte):
    sv = _sv()
    pool = torch.full((1, 1, c4.page_bytes(8, 32)), byte, dtype=torch.uint8, device="cuda")
    for dtype in (torch.bfloat16, torch.float16):
        k, v = sv.cache4_read(pool, _i32([[0]]), _i32([0]), 8, 8, 32, dtype=dtype)
        rk, rv = c4.decode(pool, 8, 32)
        assert torch.equal(k[0].double(), rk[0]) and torch.equal(v[0].double(), rv[0])
        assert torch.isfinite(k).all()


@pytest.mark.parametrize("N,heads,D,page,layers", [(2, 2, 64, 8, 3), (9, 3, 128, 16, 2), (64, 2, 96, 16, 2),
                                                   (33, 1, 24, 256, 1), (64, 8, 128, 64, 1)])
def test_commit(N, heads, D, page, layers):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(N + D)
    table, _, _, cl, pages = _slots(g, LENS, N, page)
    B = len(LENS)
    pool = c4.make_pool(g, pages, heads, page, D, layers=layers)
    k0, v0 = c4.decode(pool, page, D)
    parent = ch.random_parents(g, B, N)
    nodes, accept = torch.full((B, N), -1, dtype=torch.int32), []
    for b in range(B):
        path = ch.paths(parent[b].tolist(), N)[(b * 5) % N][1:] if b else list(range(1, N))
        nodes[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        accept.append(len(path))
    nodes, acc, new = nodes.cuda(), _i32(accept), torch.full_like(cl, -9)
    second = pool.clone()
    st = _status()
    sv.cache4_commit(pool, table, cl, nodes, acc, page, D, new_len=new, dev_status=st)
    for b, n0 in enumerate(LENS):
        for i in range(accept[b]):
            (p,), (t,) = _at(table, page, b, [n0 + int(nodes[b, i])])
            (r,), (u,) = _at(table, page, b, [n0 + 1 + i])
            for x in (k0, v0):
                x[:, r, u] = x[:, p, t]
    k, v = c4.decode(pool, page, D)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    assert new.tolist() == [n + 1 + a for n, a in zip(LENS, accept)] and int(st) == 0
    lens = cl.clone()
    sv.cache4_commit(second, table, lens, nodes, acc, page, D, dev_status=st)  # lengths in place
    assert torch.equal(second, pool) and torch.equal(lens, new) and int(st) == 0


def test_commit_of_linear_drafts_and_of_paths_that_are_none():
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(3)
    page, D, lens = 8, 32, [3, 6, 20, 5]
    table, _, _, cl, pages = _slots(g, lens, 9, page)
    pool = c4.make_pool(g, pages, 2, page, D, layers=2)
    before = pool.clone()
    new, st = torch.empty_like(cl), _status()
    sv.cache4_commit(pool, table, cl, None, _i32([0, 8, 3, 20]), page, D, new_len=new, nodes=9, dev_status=st)
    assert torch.equal(pool, before) and new.tolist() == [4, 15, 24, 14] and int(st) == 0
    table[2, :] = -1                                                   # no pages: nothing is counted
    k0, v0 = c4.decode(pool, page, D)
    # (trees of three nodes: a node 3 is none, and its path ends there)
    nodes = _i32([[1, 3, -1], [3, 2, -1], [1, 2, -1], [2, 9, -1]])
    sv.cache4_commit(pool, table, cl, nodes, _i32([2, 2, 2, 2]), page, D, new_len=new, dev_status=st)
    assert new.tolist() == [5, 7, 20, 7] and int(st) == sv.DEV_BAD_PAGE | sv.DEV_BAD_TREE
    # trees of nine nodes, and a path that is not in order
    wide = torch.full((4, 9), -1, dtype=torch.int32, device="cuda")
    wide[0, :3], wide[1, :3], wide[3, :1] = _i32([1, 8, 4]), _i32([5, 2, 7]), _i32([2])
    for path, b in (([2], 3), ([1, 8, 4], 0), ([5, 2, 7], 1), ([2], 3)):
        for i, n in enumerate(path):
            (p,), (t,) = _at(table, page, b, [lens[b] + n])
            (r,), (u,) = _at(table, page, b, [lens[b] + 1 + i])
            for x in (k0, v0):
                x[:, r, u] = x[:, p, t]
    st.zero_()
    sv.cache4_commit(pool, table, cl, wide, _i32([3, 3, 0, 1]), page, D, new_len=new, dev_status=st)
    assert new.tolist() == [7, 10, 20, 7] and int(st) == sv.DEV_BAD_PAGE
    k, v = c4.decode(pool, page, D)
    assert torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("page,D,heads", [(8, 32, 1), (16, 128, 8), (64, 80, 3), (256, 64, 2), (8, 96, 5)])
def test_copy_and_fork(page, D, heads):
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(page)
    lens = [3 * page + 3, 2 * page, 0]
    slots = 8
    P = 6
    table, count, ref, cl = ch.make_table(g, lens + [0] * (slots - 3), 0, page, P, 40)
    pool = c4.make_pool(g, 40, heads, page, D, layers=3)
    before, st = pool.clone(), _status()
    book = ch.Pages(table, count, ref, cl)
    src, dst = [0, 1, 0, 2, 0], [4, 3, 7, 5, 6]
    sv.cache4_fork(pool, table, count, ref, cl, _i32(src), _i32(dst), page, D, dev_status=st)
    copies, missing = book.fork(src, dst, page)
    assert not missing and int(st) == 0
    book.check(table, count, ref, cl)
    for a, b, _ in copies:
        before[:, b] = before[:, a]
    assert torch.equal(pool, before)
    free = [p for p, r in enumerate(ref.tolist()) if r == 0]
    sv.cache4_copy(pool, _i32([1, 2, 99]), _i32([free[0], free[1], free[2]]), page, D, dev_status=st)
    before[:, free[0]], before[:, free[1]] = before[:, 1], before[:, 2]
    assert torch.equal(pool, before) and int(st) == sv.DEV_BAD_PAGE


def test_bad_lengths_and_pages_are_skipped():
    sv = _sv()
    page, D = 8, 32
    pool = c4.make_pool(torch.Generator(device="cuda").manual_seed(1), 4, 1, page, D)
    before = pool.clone()
    x = torch.ones((3, 4, 1, D), device="cuda", dtype=torch.bfloat16)
    st = _status()
    table = _i32([[0, 1], [-1, 9], [2, 3]])
    sv.cache4_append(pool, table, _i32([-5, 6, 14]), x, x, page, dev_status=st)
    assert int(st) == sv.DEV_BAD_LEN | sv.DEV_BAD_PAGE
    assert torch.equal(pool[:3], before[:3])
    st.zero_()
    k, v = sv.cache4_read(pool, table, _i32([-5, 6, 14]), 4, page, D, dev_status=st)
    assert int(st) == sv.DEV_BAD_LEN | sv.DEV_BAD_PAGE
    # (the scale nearest to 1 / 7 is 9 / 64, so a group of ones is kept as 63 / 64)
    assert (k[:2] == 0).all() and (k[2, :2] == 63.0 / 64.0).all() and (k[2, 2:] == 0).all() and torch.equal(k, v)


def test_rows_without_tokens_touch_and_report_nothing():
    """count 0 in a row whose pages are gone, its length in the middle of a block of 8 tokens."""
    sv = _sv()
    page, D = 8, 32
    pool = c4.make_pool(torch.Generator(device="cuda").manual_seed(1), 4, 1, page, D)
    before = pool.clone()
    x = torch.ones((3, 4, 1, D), device="cuda", dtype=torch.bfloat16)
    table, lens, count, st = _i32([[-1, -1], [0, 99], [2, 3]]), _i32([5, 11, 13]), _i32([0, 0, -2]), _status()
    sv.cache4_append(pool, table, lens, x, x, page, count=count, dev_status=st)
    k, v = sv.cache4_read(pool, table, lens, 4, page, D, count=count, dev_status=st)
    assert int(st) == 0 and torch.equal(pool, before) and (k == 0).all() and (v == 0).all()


def test_pools_with_strides():
    """A pool inside a larger tensor, heads and pages in any order."""
    sv = _sv()
    g = torch.Generator(device="cuda").manual_seed(5)
    page, D, heads, N = 16, 64, 3, 5
    lens = [0, 9, 30]
    table, _, _, cl, pages = _slots(g, lens, N, page)
    big = torch.zeros((heads, pages, 2, c4.page_bytes(page, D) + 16), dtype=torch.uint8, device="cuda")
    pool = big[:, :, 1, :-16].transpose(0, 1)
    dense = torch.zeros(pool.shape, dtype=torch.uint8, device="cuda")
    x = torch.randn((3, N, heads, D), generator=g, device="cuda").bfloat16()
    for t in (pool, dense):
        sv.cache4_append(t, table, cl, x, x, page)
    assert torch.equal(pool, dense) and (big[:, :, 0] == 0).all() and (big[..., -16:] == 0).all()
    q = torch.randn((3, N, 6, D), generator=g, device="cuda").bfloat16()
    a, b = (sv.tree_attention4(q, t, table, cl, page) for t in (pool, dense))
    assert torch.equal(a, b)


def test_long_offsets():
    """A pool of more than 2^32 bytes: its last pages."""
    sv = _sv()
    page, D, heads = 128, 128, 8
    each = heads * c4.page_bytes(page, D)
    pages = (1 << 32) // each + 8
    pool = torch.empty((pages, heads, c4.page_bytes(page, D)), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((1, 300, heads, D), generator=g, device="cuda").bfloat16()
    table, zero = _i32([[pages - 1, 0, pages - 3]]), _i32([0])
    sv.cache4_append(pool, table, zero, x, x, page)
    k, v = sv.cache4_read(pool, table, zero, 300, page, D)
    assert torch.equal(k.double(), c4.values(x)) and torch.equal(k, v)
    q = torch.randn((1, 1, heads, D), generator=g, device="cuda").bfloat16()
    o, l = sv.tree_attention4(q, pool, table, _i32([299]), page, return_lse=True)
    few = pool[[pages - 1, 0, pages - 3]]
    ref = c4.ref_attention(q, few, page, _i32([[0, 1, 2]]), _i32([299]), None)
    ch.check_attention(o, l, ref, torch.bfloat16, D)
