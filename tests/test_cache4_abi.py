"""Refusals of the entry points of the 4-bit cache and of attention over selected pages, on the host before any CUDA
call."""
import ctypes
import struct

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_69_gb300 as sv
    return sv.load_library()


def _pool(**kw):
    """16 tokens of 64 channels: 1088 bytes per page and head."""
    d = dict(data=0x10000, layers=1, num_pages=10, page_size=16, heads=2, head_dim=64, layer_stride=10 * 2176,
             page_stride=2176, head_stride=1088)
    d.update(kw)
    return struct.pack("Piiiiiqqq", *[d[n] or 0 for n in ("data", "layers", "num_pages", "page_size", "heads", "head_dim",
                                                          "layer_stride", "page_stride", "head_stride")])


def _pages(**kw):
    d = dict(k=0x10000, v=0x10000, dtype=1, layers=1, num_pages=10, page_size=16, heads=2, head_dim=64,
             layer_stride=10 * 16 * 128, page_stride=16 * 128, token_stride=128, head_stride=64)
    d.update(kw)
    return struct.pack("PPiiiiiiqqqq", *d.values())


BAD_POOLS = [dict(data=None), dict(data=0x10008), dict(layers=0), dict(num_pages=0), dict(num_pages=2 ** 31 - 1),
             dict(page_size=4), dict(page_size=24), dict(page_size=1 << 21), dict(heads=0), dict(heads=1025),
             dict(head_dim=4), dict(head_dim=60), dict(head_dim=136), dict(head_stride=1072), dict(head_stride=1096),
             dict(page_stride=2160), dict(page_stride=-2176), dict(head_stride=0), dict(page_stride=1088),
             dict(layers=2, layer_stride=2176)]


def test_page_bytes(lib):
    size = lib.spec_cache4_page_bytes
    assert size(8, 32) == 272 and size(16, 128) == 2176 and size(16, 100) == 0 and size(16, 104) == 2176
    assert size(8, 8) == 272 and size(256, 64) == 256 * 68 and size(1 << 20, 128) == (1 << 20) * 136
    for bad in ((4, 32), (12, 32), (0, 32), (-8, 32), (1 << 21, 32), (8, 0), (8, 4), (8, 136), (8, -8)):
        assert size(*bad) == 0


def test_pools_are_checked(lib):
    calls = [
        lambda p: lib.spec_cache4_append(p, FAKE, FAKE, FAKE, FAKE, 1, 1024, 128, 64, None, 2, 4, 8, None, None),
        lambda p: lib.spec_cache4_read(p, FAKE, FAKE, None, FAKE, FAKE, 1, 2, 4, 8, None, None),
        lambda p: lib.spec_cache4_commit(p, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, None, None),
        lambda p: lib.spec_cache4_copy(p, FAKE, FAKE, 2, None, None),
        lambda p: lib.spec_cache4_fork(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, FAKE, 4096, None, None),
        lambda p: lib.spec_cache4_bounds(p, FAKE, None, FAKE, FAKE, 1, 2, 8, None, None),
        lambda p: lib.spec_tree_attention4(FAKE, 1, 1024, 256, 64, p, FAKE, 0, FAKE, None, None, 2, 4, 4, 8, 0.1, 0, 0,
                                           FAKE, None, FAKE, 1 << 40, None, None),
    ]
    for call in calls:
        for bad in BAD_POOLS:
            assert call(_pool(**bad)) == 1, bad
        assert call(None) == 1


def test_pools_in_any_order_are_taken(lib):
    def fork(p):
        return lib.spec_cache4_fork(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, None, 0, None, None)
    assert fork(_pool()) == 4                                          # the missing workspace is found last
    assert fork(_pool(head_stride=10 * 1088, page_stride=1088, layer_stride=0)) == 4
    assert fork(_pool(layers=3, layer_stride=1088, page_stride=2 * 3264, head_stride=3264)) == 4
    assert fork(_pool(heads=1, head_stride=0, page_stride=1088)) == 4
    assert lib.spec_cache4_fork(_pool(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, ODD, 4096, None, None) == 4
    for bad in (dict(F=0), dict(F=8193), dict(S=0), dict(S=8193), dict(P=0), dict(t=None), dict(src=None)):
        a = dict(dict(F=2, S=4, P=8, t=FAKE, src=FAKE), **bad)
        assert lib.spec_cache4_fork(_pool(), a["t"], FAKE, FAKE, FAKE, a["src"], FAKE, a["F"], a["S"], a["P"], FAKE,
                                    1 << 20, None, None) == 1, bad


def test_append_read_commit_copy(lib):
    base = dict(p=_pool(), t=FAKE, l=FAKE, k=FAKE, v=FAKE, dt=1, sb=1024, sn=128, sh=64, B=2, N=4, P=8)

    def app(**kw):
        a = dict(base, **kw)
        return lib.spec_cache4_append(a["p"], a["t"], a["l"], a["k"], a["v"], a["dt"], a["sb"], a["sn"], a["sh"], None,
                                      a["B"], a["N"], a["P"], None, None)
    for bad in (dict(t=None), dict(l=None), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD), dict(sb=4), dict(sn=-128),
                dict(sh=63), dict(B=0), dict(B=1 << 16), dict(N=0), dict(P=0), dict(p=_pool(layers=2))):
        assert app(**bad) == 1, bad
    assert app(dt=0) == 2 and app(dt=3) == 2

    def read(**kw):
        a = dict(base, **kw)
        return lib.spec_cache4_read(a["p"], a["t"], a["l"], None, a["k"], a["v"], a["dt"], a["B"], a["N"], a["P"], None,
                                    None)
    for bad in (dict(t=None), dict(l=None), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD), dict(B=0), dict(B=1 << 16),
                dict(N=0), dict(P=0)):
        assert read(**bad) == 1, bad
    assert read(dt=0) == 2

    def com(t=FAKE, l=FAKE, a=FAKE, new=FAKE, B=2, N=4, P=8, p=_pool()):
        return lib.spec_cache4_commit(p, t, l, FAKE, a, new, B, N, P, None, None)
    for bad in (dict(t=None), dict(l=None), dict(a=None), dict(new=None), dict(B=0), dict(B=1 << 16), dict(N=0), dict(N=65),
                dict(P=0)):
        assert com(**bad) == 1, bad
    assert lib.spec_cache4_copy(_pool(), None, FAKE, 2, None, None) == 1
    assert lib.spec_cache4_copy(_pool(), FAKE, None, 2, None, None) == 1
    assert lib.spec_cache4_copy(_pool(), FAKE, FAKE, 0, None, None) == 1


def test_attention(lib):
    size = lib.spec_tree_attention4_workspace_bytes
    assert size(2, 4, 4, 2, 64) > 0
    for bad in ((0, 4, 4, 2, 64), (1 << 16, 4, 4, 2, 64), (2, 0, 4, 2, 64), (2, 65, 4, 2, 64), (2, 4, 3, 2, 64),
                (2, 4, 1, 2, 64), (2, 4, 130, 2, 64), (2, 4, 4, 2, 136), (2, 4, 4, 2, 12), (2, 4, 4, 0, 64)):
        assert size(*bad) == 0, bad
    base = dict(q=FAKE, dt=1, sb=1024, sn=256, sh=64, p=_pool(), t=FAKE, per=0, l=FAKE, B=2, N=4, Hq=4, P=8, scale=0.1, w=0,
                s=0, o=FAKE, ws=FAKE, n=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return lib.spec_tree_attention4(a["q"], a["dt"], a["sb"], a["sn"], a["sh"], a["p"], a["t"], a["per"], a["l"], None,
                                        None, a["B"], a["N"], a["Hq"], a["P"], a["scale"], a["w"], a["s"], a["o"], None,
                                        a["ws"], a["n"], None, None)
    for bad in (dict(q=None), dict(t=None), dict(l=None), dict(o=None), dict(q=ODD), dict(o=ODD), dict(sb=4), dict(sn=-8),
                dict(sh=60), dict(B=0), dict(N=65), dict(Hq=3), dict(P=0), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(w=-1), dict(s=-1), dict(per=2), dict(p=_pool(layers=2))):
        assert call(**bad) == 1, bad
    assert call(dt=0) == 2
    assert call(ws=None) == 4 and call(n=0) == 4 and call(ws=ctypes.c_void_p(0x10010)) == 4
    # lists for 16-bit caches: the checks of spec_tree_attention
    assert lib.spec_sparse_attention(None, 1024, 256, 64, _pages(), FAKE, FAKE, None, None, 2, 4, 4, 8, 0.1, 0, 0, FAKE,
                                     None, FAKE, 1 << 40, None, None) == 1
    assert lib.spec_sparse_attention(FAKE, 1024, 256, 64, _pages(dtype=0), FAKE, FAKE, None, None, 2, 4, 4, 8, 0.1, 0, 0,
                                     FAKE, None, FAKE, 1 << 40, None, None) == 2
    assert lib.spec_sparse_attention(FAKE, 1024, 256, 64, _pages(), FAKE, FAKE, None, None, 2, 4, 4, 8, 0.1, 0, 0, FAKE,
                                     None, None, 0, None, None) == 4


def test_bounds_scores_select(lib):
    def bounds(p=_pages(), t=FAKE, l=FAKE, b=FAKE, B=2, P=8):
        return lib.spec_cache_bounds(p, t, None, l, b, B, P, None, None)
    for bad in (dict(p=None), dict(t=None), dict(l=None), dict(b=None), dict(b=ODD), dict(B=0), dict(B=1 << 16), dict(P=0),
                dict(p=_pages(layers=2)), dict(p=_pages(k=0x10008))):
        assert bounds(**bad) == 1, bad
    assert bounds(p=_pages(dtype=0)) == 2
    assert lib.spec_cache4_bounds(_pool(), FAKE, None, FAKE, FAKE, 0, 2, 8, None, None) == 2
    assert lib.spec_cache4_bounds(_pool(), FAKE, None, FAKE, ODD, 1, 2, 8, None, None) == 1
    base = dict(q=FAKE, dt=1, sb=1024, sn=256, sh=64, b=FAKE, t=FAKE, l=FAKE, o=FAKE, B=2, N=4, Hq=4, H=2, D=64, P=8, n=10,
                page=16)

    def scores(**kw):
        a = dict(base, **kw)
        return lib.spec_page_scores(a["q"], a["dt"], a["sb"], a["sn"], a["sh"], a["b"], a["t"], a["l"], None, a["o"], a["B"],
                                    a["N"], a["Hq"], a["H"], a["D"], a["P"], a["n"], a["page"], None, None)
    for bad in (dict(q=None), dict(b=None), dict(t=None), dict(l=None), dict(o=None), dict(q=ODD), dict(b=ODD), dict(sb=4),
                dict(sn=8), dict(sh=60), dict(B=0), dict(B=1 << 16), dict(N=0), dict(N=65), dict(Hq=3), dict(Hq=130),
                dict(H=0), dict(H=1025, Hq=1025), dict(D=12), dict(D=136), dict(P=0), dict(n=0), dict(page=4), dict(page=24)):
        assert scores(**bad) == 1, bad
    assert scores(dt=0) == 2
    base2 = dict(s=FAKE, t=FAKE, l=FAKE, ot=FAKE, ol=FAKE, B=2, H=2, P=8, page=16, keep=4, first=1, recent=1, extra=0)

    def select(**kw):
        a = dict(base2, **kw)
        return lib.spec_page_select(a["s"], a["t"], a["l"], a["ot"], a["ol"], a["B"], a["H"], a["P"], a["page"], a["keep"],
                                    a["first"], a["recent"], a["extra"], None, None)
    for bad in (dict(s=None), dict(t=None), dict(l=None), dict(ot=None), dict(ol=None), dict(B=0), dict(B=1 << 16), dict(H=0),
                dict(H=1025), dict(P=0), dict(P=131073), dict(page=4), dict(page=24), dict(keep=0), dict(keep=131073),
                dict(first=-1), dict(recent=0), dict(first=4), dict(recent=4), dict(recent=2 ** 31 - 1),
                dict(first=2 ** 31 - 1), dict(extra=-1), dict(extra=(1 << 20) + 1)):
        assert select(**bad) == 1, bad


def test_what_the_python_side_refuses():
    import speculative_decoding_verification_69_gb300 as sv
    with pytest.raises(ValueError):
        sv.cache4_page_bytes(12, 64)
    with pytest.raises(TypeError):
        sv.cache4_read(None, None, None, 1, 16, 64, dtype=torch.float32)
    with pytest.raises(TypeError):
        sv.PagedCache4(1, 1, 16, 1, 64, 1, 1, dtype=torch.float32)
    pool, x = torch.zeros((4, 2, 1088), dtype=torch.uint8), torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError):                                    # no CUDA tensors
        sv.cache4_append(pool, i, i[0], x, x, 16)
    with pytest.raises(ValueError):
        sv.tree_attention4(x, pool, i, i[0], 16)
    with pytest.raises(TypeError):
        sv.tree_attention4(x.float(), pool, i, i[0], 16)
    with pytest.raises(TypeError):
        sv.page_scores(None, x, i, i[0], 16)
    with pytest.raises(ValueError):
        sv.page_select(torch.zeros((1, 2, 1)), i, i[0], 16, 2)
