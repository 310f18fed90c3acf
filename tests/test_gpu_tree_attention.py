"""Tree attention over a paged cache against the definition in 64 bits."""
import math

import pytest
import torch

import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _sv():
    import speculative_decoding_verification_69_gb300 as sv
    return sv


def _case(seed, lens, N, hq, hkv, D, page, dtype, *, tree=True, hnd=False, qscale=2.0, spare=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    P = max(-(-(n + N) // page) for n in lens) + 1
    pages = sum(-(-(n + N) // page) for n in lens) + spare
    table, count, ref, cl = ch.make_table(g, lens, N, page, P, pages)
    k = ch.make_pool(g, pages, page, hkv, D, dtype, hnd=hnd)
    v = ch.make_pool(g, pages, page, hkv, D, dtype, hnd=hnd)
    q = (torch.randn((B, N, hq, D), generator=g, device="cuda") * qscale).to(dtype)
    parent = ch.random_parents(g, B, N) if tree else None
    return dict(q=q, k=k, v=v, table=table, len=cl, parent=parent)


def _run(c, **kw):
    sv = _sv()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = sv.tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], return_lse=True,
                             dev_status=st, **kw)
    torch.cuda.synchronize()
    return o, l, int(st.item())


def _check(c, status=0, **kw):
    o, l, st = _run(c, **kw)
    assert st == status
    ref = ch.ref_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], **kw)
    ch.check_attention(o, l, ref, c["q"].dtype, c["q"].shape[-1])
    return o, l


LENS = [0, 1, 7, 8, 63, 64, 127, 128, 129, 200, 255, 256, 257, 511, 640]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page,hnd", [
    (1, 8, 8, 64, 16, False),      # single tokens, a key head each
    (1, 8, 1, 128, 8, True),       # one key head for all
    (2, 4, 4, 8, 8, False),        # the smallest head
    (9, 8, 2, 128, 16, False),     # linear-draft size
    (16, 14, 2, 128, 32, True),    # a group of 7
    (33, 4, 1, 96, 64, False),     # 132 rows of one key head: just past 128
    (64, 4, 2, 64, 128, False),    # 128 rows exactly
    (64, 8, 2, 128, 256, True),    # 256 rows, pages longer than a tile of keys
    (63, 10, 2, 72, 16, False),    # 315 rows, a head of 72
    (64, 64, 1, 40, 8, False),     # 4096 rows of one key head
])
def test_lengths_heads_layouts(N, hq, hkv, D, page, hnd, dtype):
    lens = LENS if hq < 64 else [0, 5, 130, 300]
    _check(_case(N * 131 + D, lens, N, hq, hkv, D, page, dtype, hnd=hnd))


@pytest.mark.parametrize("N", [1, 9, 33])
def test_chain_is_causal(N):
    c = _case(7, [0, 3, 100, 700], N, 8, 2, 128, 16, torch.bfloat16, tree=False)
    o, l = _check(c)
    c["parent"] = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(4, 1)
    o2, l2, _ = _run(c)
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (17, 0), (64, 3), (128, 130), (129, 128),
                                          (300, 1), (5000, 4), (700, 0)])
@pytest.mark.parametrize("N,hq,hkv,D,page", [(1, 8, 1, 64, 16), (12, 8, 2, 64, 16), (40, 8, 2, 128, 64)])
def test_window_and_sinks(N, hq, hkv, D, page, window, sinks):
    _check(_case(window * 7 + N, [0, 1, 5, 127, 128, 300, 513, 1000], N, hq, hkv, D, page, torch.bfloat16),
           window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window", [0, 100])
def test_unseen_positions_hold_anything(window, dtype):
    """Stale pages: every position of the pool that no node sees is NaN or
    infinite, and the table's entries for pages that no node sees are rubbish."""
    page, N, lens = 16, 11, [0, 4, 37, 250, 260, 385]
    c = _case(91, lens, N, 8, 2, 64, page, dtype)
    cnt = torch.tensor([11, 3, 11, 0, 7, 10], dtype=torch.int32, device="cuda")
    sinks = 3 if window else 0
    seen = torch.zeros(c["k"].shape[:2], dtype=torch.bool)
    P = c["table"].shape[1]
    for b, n0 in enumerate(lens):
        used = set()
        for p in ch.paths(c["parent"][b].tolist(), int(cnt[b])):
            used |= set(ch.seen_positions(n0, p, window, sinks))
        row = c["table"][b].tolist()
        for j in used:
            seen[row[j // page], j % page] = True
        for i in range(P):
            if not any(j // page == i for j in used):
                c["table"][b, i] = [-1, 2 ** 31 - 1, -2 ** 31][i % 3]
    bad = ~seen.cuda().unsqueeze(-1).unsqueeze(-1).expand_as(c["k"])
    fill = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda", dtype=dtype)
    noise = fill[torch.randint(0, 3, c["k"].shape, device="cuda")]
    c["k"] = torch.where(bad, noise, c["k"])
    c["v"] = torch.where(bad, noise, c["v"])
    o, l = _check(c, node_count=cnt, window=window, sinks=sinks)
    for b in range(len(lens)):  # rows past the count see nothing
        assert (o[b, int(cnt[b]):] == 0).all() and torch.isneginf(l[b, int(cnt[b]):]).all()


@pytest.mark.parametrize("N,hq,hkv,D,ctx", [(1, 8, 1, 128, 70001), (16, 8, 2, 128, 20000), (64, 8, 2, 64, 9999),
                                            (5, 4, 4, 64, 33333)])
def test_long_contexts(N, hq, hkv, D, ctx):
    _check(_case(ctx, [ctx], N, hq, hkv, D, 64, torch.bfloat16))


def test_many_requests_of_mixed_lengths():
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in (torch.rand(300, generator=g) ** 3 * 900).tolist()] + [4000, 0, 0, 0]
    _check(_case(17, lens, 5, 8, 4, 64, 16, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,G,hkv,D,page,window,sinks", [
    (1, 1, 80, 64, 16, 0, 0),
    (9, 8, 40, 64, 16, 128, 0),       # 72 rows
    (9, 8, 40, 64, 16, 100, 130),     # sinks past a tile
    (16, 8, 38, 128, 32, 0, 0),       # 128 rows, at one head per CTA
    (13, 3, 64, 72, 8, 50, 2),
    (64, 2, 44, 128, 128, 0, 0),      # a node per row pair
    (7, 5, 102, 40, 256, 700, 1),
])
def test_many_heads(N, G, hkv, D, page, window, sinks, dtype):
    """More (request, key head) pairs than CTAs: each softmax stream has a head of its own."""
    lens = [0, 3, 127, 128, 129, 300, 1000, 64][:8 if hkv < 100 else 3]
    c = _case(N * 17 + hkv, lens, N, hkv * G, hkv, D, page, dtype)
    _check(c, window=window, sinks=sinks)
    r = torch.Generator().manual_seed(N)
    cnt = torch.randint(0, N + 1, (len(lens),), generator=r, dtype=torch.int32).cuda()
    # positions that no node sees hold NaN
    live = torch.zeros((c["k"].shape[0], page), dtype=torch.bool, device="cuda")
    for b, n0 in enumerate(lens):
        seen = set()
        for path in ch.paths(c["parent"][b].tolist(), int(cnt[b])):
            seen |= set(ch.seen_positions(n0, path, window, sinks))
        for j in seen:
            live[int(c["table"][b, j // page]), j % page] = True
    for x in (c["k"], c["v"]):
        x[~live] = float("nan")
    _check(c, node_count=cnt, window=window, sinks=sinks)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    import random
    r = random.Random(1000 + seed)
    hkv, G = r.choice([1, 2, 3, 8]), r.choice([1, 2, 3, 5, 8, 16])
    N, D = r.randint(1, 64), 8 * r.randint(1, 16)
    page = r.choice([8, 16, 32, 64, 128, 256])
    B = r.randint(1, 6)
    lens = [r.choice([0, r.randint(0, 40), r.randint(0, 1500)]) for _ in range(B)]
    window = r.choice([0, 0, r.randint(1, 600)])
    c = _case(seed, lens, N, hkv * G, hkv, D, page, r.choice([torch.bfloat16, torch.float16]),
              hnd=r.random() < 0.5, tree=r.random() < 0.7)
    cnt = torch.tensor([r.randint(0, N) for _ in range(B)], dtype=torch.int32, device="cuda")
    _check(c, node_count=cnt, window=window, sinks=r.choice([0, 2, 200]) if window else 0,
           scale=r.choice([None, 0.05]))


@pytest.mark.parametrize("N,hq,ctx", [(4, 4, 300), (64, 8, 500), (2, 2, 60000)])
def test_nan_and_infinite_scores_show(N, hq, ctx):
    """A NaN or an infinity that a row does see makes that row NaN, and no other."""
    c = _case(N + ctx, [ctx, 200], N, hq, 2, 64, 16, torch.bfloat16)
    ref_o, ref_l, _ = _run(c)
    bad = c["q"].clone()
    bad[0, 1, 0, 3] = float("nan")
    bad[1, 0, hq - 1] = float("inf")  # scores of both infinities
    o, l, st = _run(dict(c, q=bad))
    assert st == 0
    for b, n, h in ((0, 1, 0), (1, 0, hq - 1)):
        assert o[b, n, h].isnan().all() and l[b, n, h].isnan()
        o[b, n, h], l[b, n, h] = ref_o[b, n, h], ref_l[b, n, h]
    assert torch.equal(o, ref_o) and torch.equal(l, ref_l)
    # all scores of a row NaN, in every key tile and every part
    c["k"][c["table"][0, :-(-(ctx + N) // 16)].long()] = float("nan")
    o, l, st = _run(c)
    assert st == 0 and o[0].isnan().all() and l[0].isnan().all()
    assert torch.equal(o[1], ref_o[1]) and torch.equal(l[1], ref_l[1])


@pytest.mark.parametrize("N,hq,hkv,ctx", [(1, 8, 2, 3000), (9, 8, 2, 700), (64, 16, 2, 900), (4, 64, 64, 250)])
def test_nothing_unwritten_is_read(N, hq, hkv, ctx):
    """A workspace and outputs full of NaN and -1 make no difference, and every output is written."""
    sv = _sv()
    c = _case(N + hq, [ctx, 0, 40], N, hq, hkv, 64, 16, torch.bfloat16)
    cnt = torch.tensor([N, N, N // 2], dtype=torch.int32, device="cuda")
    o, l, _ = _run(c, node_count=cnt)
    n = sv.load_library().spec_tree_attention_workspace_bytes(3, N, hq, hkv, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    o2, l2, st = _run(c, node_count=cnt, workspace=ws, out=torch.full_like(o, float("nan")))
    assert st == 0 and torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("N,hq,hkv,D", [(1, 8, 2, 128), (9, 8, 2, 64), (64, 16, 2, 128), (4, 64, 64, 64)])
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


def test_large_scores():
    """Sharp distributions whose maximum grows along the keys (the running
    maximum moves many times) and falls (it never moves again)."""
    for sign in (1.0, -1.0):
        c = _case(3, [1500, 900], 4, 4, 1, 64, 64, torch.bfloat16, qscale=1.0)
        kk, page = c["k"], 64
        for b, n0 in enumerate([1500, 900]):
            j = torch.arange(n0 + 4, device="cuda")
            pg = c["table"][b].long()[j // page]
            ramp = (sign * (j.float() / 100 - 5)).view(-1, 1, 1)
            kk[pg, j % page] = (kk[pg, j % page].float() * 0.5 + ramp).bfloat16()
        c["q"] = c["q"].abs() * 4 + 1
        _check(c)


def test_strided_queries_and_single_extents():
    """Queries that are a slice of a fused projection, batches of one, and
    dimensions of one element with odd strides."""
    g = torch.Generator(device="cuda").manual_seed(2)
    c = _case(2, [77], 9, 8, 2, 64, 16, torch.bfloat16)
    qkv = torch.randn((1, 9, 12, 64), generator=g, device="cuda").bfloat16()
    c["q"] = qkv[:, :, 2:10]
    _check(c)
    c["q"] = torch.as_strided(qkv, (1, 9, 8, 64), (3, 12 * 64, 64, 1))
    _check(c)


def test_pool_past_32_bit_offsets():
    """A pool of more than 2^31 elements: pages at both of its ends."""
    page, hkv, D, N = 64, 8, 128, 4
    pages = (1 << 31) // (page * hkv * D) + 40
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.empty((pages, page, hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = [pages - 1, 0, pages - 7, pages - 30, 5]
    for p in ids:
        k[p].normal_(generator=g)
        v[p].normal_(generator=g)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    q = torch.randn((1, N, 16, D), generator=g, device="cuda").bfloat16()
    _check(dict(q=q, k=k, v=v, table=table, len=torch.tensor([300], dtype=torch.int32, device="cuda"),
                parent=ch.random_parents(g, 1, N)))


def test_bad_data_is_reported_and_survived():
    sv = _sv()
    c = _case(4, [40, 100], 6, 4, 2, 64, 16, torch.bfloat16)
    c["parent"][1] = torch.tensor([-1, 0, 5, -3, 2 ** 31 - 1, 4], device="cuda")
    _check(c, status=sv.DEV_BAD_TREE)
    c = _case(4, [40, 100], 6, 4, 2, 64, 16, torch.bfloat16)
    c["table"][0, 1] = 10 ** 6
    o, l, st = _run(c)
    assert st == sv.DEV_BAD_PAGE
    ref = ch.ref_attention(c["q"][1:], c["k"], c["v"], c["table"][1:], c["len"][1:], c["parent"][1:])
    ch.check_attention(o[1:], l[1:], ref, torch.bfloat16, 64)
    c = _case(4, [40, 100], 6, 4, 2, 64, 16, torch.bfloat16)
    P = c["table"].shape[1]
    for bad in (-5, P * 16 + 1, 2 ** 31 - 1):
        c["len"][0] = bad
        o, l, st = _run(c)
        assert st & sv.DEV_BAD_LEN
        ref = ch.ref_attention(c["q"][1:], c["k"], c["v"], c["table"][1:], c["len"][1:], c["parent"][1:])
        ch.check_attention(o[1:], l[1:], ref, torch.bfloat16, 64)


def test_length_up_to_the_last_place_of_the_table():
    """The tree fills the row of the table to its end; one token more is cut."""
    sv = _sv()
    page, N = 16, 8
    c = _case(6, [page * 5 - N], N, 4, 2, 64, page, torch.bfloat16, tree=False)
    c["table"] = c["table"][:, :5].contiguous()
    o, l = _check(c)
    c["len"] += 1
    o2, l2, st = _run(c)
    assert st == sv.DEV_BAD_LEN
    ref = ch.ref_attention(c["q"], c["k"], c["v"], c["table"], c["len"], None, node_count=[N - 1])
    ch.check_attention(o2, l2, ref, torch.bfloat16, 64)


def test_same_inputs_same_bits_on_any_stream():
    c = _case(8, [1000, 3, 5000], 16, 8, 2, 128, 32, torch.bfloat16)
    o, l, _ = _run(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv = _sv()
    for _ in range(3):
        o2, l2 = sv.tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], return_lse=True, stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("N,hq,hkv,D", [(1, 5, 1, 8), (1, 4, 4, 128), (3, 14, 2, 64), (9, 24, 4, 128), (33, 20, 4, 64)])
def test_same_bits_whatever_ran_before(N, hq, hkv, D):
    """What earlier calls left in shared and tensor memory, under rows that the next call does not have, is not seen."""
    lens = [(i * 613) % 4001 for i in range(100)]
    c = _case(31 + N, lens, N, hq, hkv, D, 256, torch.bfloat16, qscale=0.3)
    others = [_case(32 + i, [700, 90], 64, 8, 2, 64 + 64 * (i % 2), 16, dt, qscale=30.0)
              for i, dt in enumerate((torch.bfloat16, torch.float16))]
    o, l, _ = _run(c)
    for i in range(12):
        _run(others[i % 2])
        o2, l2, _ = _run(c)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_captured_in_a_graph():
    """One captured call follows the lengths and the data of later replays."""
    c = _case(9, [600, 30], 7, 8, 2, 64, 16, torch.bfloat16)
    sv = _sv()
    out = torch.empty_like(c["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def call():
        sv.tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c["len"][0] = 333
    c["q"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    ref = ch.ref_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"])
    ch.check_attention(out, None, ref, torch.bfloat16, 64)


def test_refusals():
    sv = _sv()
    c = _case(1, [20, 30], 4, 4, 2, 64, 16, torch.bfloat16)

    def call(**kw):
        x = dict(c, **{a: b for a, b in kw.items() if a in c})
        opt = {a: b for a, b in kw.items() if a not in c}
        return sv.tree_attention(x["q"], x["k"], x["v"], x["table"], x["len"], x["parent"], **opt)

    with pytest.raises(ValueError):
        call(q=c["q"].half())
    with pytest.raises(ValueError):
        call(q=c["q"][..., :32])
    with pytest.raises(ValueError):
        call(q=c["q"].cpu())
    with pytest.raises(ValueError):
        call(v=c["v"][:-1])
    with pytest.raises(ValueError):
        call(v=c["v"].transpose(1, 2).contiguous().transpose(1, 2))    # other strides than k
    with pytest.raises(ValueError):
        call(table=c["table"].long())
    with pytest.raises(ValueError):
        call(len=c["len"][:1])
    with pytest.raises(ValueError):
        call(parent=c["parent"][:, :3])
    with pytest.raises(ValueError):
        call(out=torch.empty_like(c["q"]).half())
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
               dict(scale=math.inf)):
        with pytest.raises(sv.SpecVerifyError):
            call(**kw)
    with pytest.raises(sv.SpecVerifyError):                             # 3 query heads on 2 key heads
        call(q=c["q"][:, :, :3])
    with pytest.raises(sv.SpecVerifyError):                             # float32 caches
        call(q=c["q"].float(), k=c["k"].float(), v=c["v"].float())
    with pytest.raises(sv.SpecVerifyError):                             # a misaligned pool
        flat = torch.zeros(c["k"].numel() + 8, dtype=torch.bfloat16, device="cuda")
        x = flat[1:1 + c["k"].numel()].view(c["k"].shape)
        call(k=x, v=x)
    with pytest.raises(sv.SpecVerifyError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("N,hq,hkv,D", [(9, 8, 2, 128), (9, 8, 2, 64), (64, 8, 2, 128), (64, 16, 2, 64),
                                        (5, 80, 80, 128), (5, 80, 80, 40)])
def test_same_bits_beside_other_work(N, hq, hkv, D):
    """Many tiles in every division of work between the streams, while products on another
    stream take their turns: no tile's weights, scores or values meet those of another."""
    lens = [2500, 900] if hkv > 2 else [20000, 300, 7000]
    c = _case(N + hq + D, lens, N, hq, hkv, D, 64, torch.float16)
    o, l = _check(c)
    a = torch.randn((4096, 4096), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(side):
            b = a @ a
        o2, l2, st = _run(c)
        assert st == 0 and torch.equal(o, o2) and torch.equal(l, l2)
    del b


SPLITS = [(1, 2, 1, [0, 5]),                # the only key; streams that divide the keys
          (4, 4, 2, [300, 0, 90]),
          (3, 8, 2, [60000]),               # parts of many CTAs
          (64, 8, 2, [500, 130]),           # streams that divide the rows
          (64, 8, 1, [9000]),
          (5, 160, 80, [200, 3]),           # a key head each
          (2, 64, 64, [2900, 2500, 3000])]  # and cut


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,lens", SPLITS)
def test_rows_of_infinitely_low_scores_are_nan(N, hq, hkv, lens, dtype):
    """Where all the scores a row sees are -inf there is no softmax: NaN, as for
    a NaN score, and not the 0 of a row that does not exist."""
    c = _case(N + hq, lens, N, hq, hkv, 64, 16, dtype)
    c["k"][..., 3] = 1.0
    cnt = torch.tensor([N] + [max(1, N // 2)] * (len(lens) - 1), dtype=torch.int32, device="cuda")
    ref_o, ref_l, _ = _run(c, node_count=cnt)
    q = c["q"].clone()
    rows = {(b, n, h) for b in range(len(lens)) for n, h in ((0, 0), (int(cnt[b]) - 1, hq - 1), (N - 1, hq // 2))}
    for r in rows:
        q[r][3] = -math.inf
    o, l, st = _run(dict(c, q=q), node_count=cnt)
    assert st == 0
    for b, n, h in rows:
        if n < int(cnt[b]):
            assert o[b, n, h].isnan().all() and l[b, n, h].isnan()
            o[b, n, h], l[b, n, h] = ref_o[b, n, h], ref_l[b, n, h]
    assert torch.equal(o, ref_o) and torch.equal(l, ref_l)  # rows past the counts among them: 0 and -inf


@pytest.mark.parametrize("N,hq,hkv,lens", SPLITS)
def test_one_infinitely_low_score_has_no_weight(N, hq, hkv, lens):
    """A score below float32's range counts as one that is merely far below the others."""
    c = _case(N + hq, lens, N, hq, hkv, 64, 16, torch.bfloat16)
    c["k"][..., 3] = 0.0
    for b, n0 in enumerate(lens):
        if n0:
            p = int(c["table"][b, (n0 - 1) // 16])
            c["k"][p, (n0 - 1) % 16, :, 3] = 2.0 ** 20
    got = []
    for low in (-1.0, -2.0 ** 120):
        q = c["q"].clone()
        q[..., 3] = low
        o, l, st = _run(dict(c, q=q))
        assert st == 0 and torch.isfinite(o).all() and torch.isfinite(l).all()
        got.append((o, l))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def _some_see(c, window, sinks):
    """Per request the positions that some of its nodes see and others do not."""
    out = []
    for b, n0 in enumerate(c["len"].tolist()):
        par = None if c["parent"] is None else c["parent"][b].tolist()
        sets = [set(ch.seen_positions(n0, p, window, sinks)) for p in ch.paths(par, c["q"].shape[1])]
        out.append(sorted(set().union(*sets) - set.intersection(*sets)))
    return out


def _check_with_non_finite(c, got, **kw):
    """As ch.check_attention where the definition is finite; elsewhere the same infinity, or NaN."""
    (o, l), ref = got, ch.ref_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], **kw)
    want, oc = ref[0], o.cpu().double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(oc), torch.isnan(want))
    assert torch.equal(torch.isfinite(oc), ~odd)
    inf = torch.isinf(want)
    assert torch.equal(oc[inf], want[inf])
    clean = [x.masked_fill(odd, 0.0) for x in (oc, want, ref[2])]
    ch.check_attention(clean[0], l, (clean[1], ref[1], clean[2], ref[3]), o.dtype, o.shape[-1])
    return odd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D,page,lens,window,sinks", [
    (2, 2, 1, 64, 16, [0, 5, 127], 0, 0),
    (9, 8, 2, 128, 16, [0, 119, 124, 700], 0, 0),          # nodes in one tile and across two
    (9, 8, 2, 72, 8, [40000], 0, 0),                        # parts of many CTAs
    (12, 8, 2, 64, 16, [300, 3, 1000, 65], 40, 3),          # the low end of a window
    (12, 8, 2, 128, 64, [300, 130, 1000], 5, 130),          # nodes that leave their own window
    (64, 8, 2, 128, 32, [200, 100, 0], 0, 0),               # rows divided between the streams
    (64, 8, 1, 64, 16, [900, 64], 100, 2),                  # several row tiles
    (7, 160, 80, 64, 16, [250, 30], 0, 0),                  # a key head each
    (7, 80, 80, 128, 16, [1000, 300], 128, 1),
])
def test_values_that_are_not_finite_stay_in_their_branch(N, hq, hkv, D, page, lens, window, sinks, dtype):
    c = _case(N * 7 + D, lens, N, hq, hkv, D, page, dtype, qscale=0.3)
    before = _run(c, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(N)
    odd = [float("inf"), float("-inf"), float("nan")]
    hit = 0
    for b, spots in enumerate(_some_see(c, window, sinks)):
        for j in spots[::3]:
            at = (int(c["table"][b, j // page]), j % page)
            for _ in range(2):
                h, d, x = (int(torch.randint(n, (1,), generator=g)) for n in (hkv, D, 3))
                c["v"][at][h, d] = odd[x]
                hit += 1
    assert hit > 0
    o, l, st = _run(c, window=window, sinks=sinks)
    assert st == 0
    odd = _check_with_non_finite(c, (o, l), window=window, sinks=sinks)
    assert odd.any() and not odd.all()
    assert torch.equal(o[~odd.cuda()], before[0][~odd.cuda()]) and torch.equal(l, before[1])


@pytest.mark.parametrize("N,hq,hkv,lens", [(9, 8, 2, [119, 700]), (64, 8, 2, [200, 0]), (7, 160, 80, [250])])
def test_keys_that_are_not_finite_stay_in_their_branch(N, hq, hkv, lens):
    c = _case(N, lens, N, hq, hkv, 64, 16, torch.bfloat16, qscale=0.3)
    ref_o, ref_l, _ = _run(c)
    par = c["parent"].tolist()
    for b, n0 in enumerate(lens):
        c["k"][int(c["table"][b, (n0 + 1) // 16]), (n0 + 1) % 16] = float("nan")
    o, l, st = _run(c)
    assert st == 0
    for b in range(len(lens)):
        for n, path in enumerate(ch.paths(par[b], N)):
            if 1 in path:
                assert o[b, n].isnan().all() and l[b, n].isnan().all()
            else:
                assert torch.equal(o[b, n], ref_o[b, n]) and torch.equal(l[b, n], ref_l[b, n])


def test_a_flag_without_a_truth_value_is_refused():
    c = _case(1, [20, 30], 4, 4, 2, 64, 16, torch.bfloat16)
    with pytest.raises(RuntimeError, match="ambiguous"):
        _sv().tree_attention(c["q"], c["k"], c["v"], c["table"], c["len"], c["parent"], return_lse=torch.ones(2))
