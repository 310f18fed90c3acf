"""Refusals of the paged-cache entry points, on the host before any CUDA call."""
import ctypes
import struct

import pytest

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_69_gb300 as sv
    return sv.load_library()


FIELDS = ("k", "v", "dtype", "layers", "num_pages", "page_size", "heads", "head_dim", "layer_stride", "page_stride",
          "token_stride", "head_stride")


def _pages(**kw):
    d = dict(k=0x10000, v=0x10000, dtype=1, layers=1, num_pages=10, page_size=16, heads=2, head_dim=64,
             layer_stride=10 * 16 * 128, page_stride=16 * 128, token_stride=128, head_stride=64)
    d.update(kw)
    return struct.pack("PPiiiiiiqqqq", *[d[n] or 0 for n in FIELDS])


BAD_POOLS = [dict(k=None), dict(v=None), dict(layers=0), dict(num_pages=0), dict(page_size=4), dict(page_size=24),
             dict(heads=0), dict(heads=2000), dict(head_dim=4), dict(head_dim=60), dict(head_stride=0),
             dict(token_stride=100), dict(page_stride=-128), dict(k=0x10008), dict(num_pages=2 ** 31 - 1)]


def test_pools_are_checked(lib):
    ws = ctypes.c_void_p(0x10000)
    calls = [
        lambda p: lib.spec_cache_fork(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, ws, 4096, None, None),
        lambda p: lib.spec_cache_copy(p, FAKE, FAKE, 2, None, None),
        lambda p: lib.spec_cache_append(p, FAKE, FAKE, FAKE, FAKE, 1024, 128, 64, None, 2, 4, 8, None, None),
        lambda p: lib.spec_cache_commit(p, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, None, None),
        lambda p: lib.spec_tree_attention(FAKE, 1024, 256, 64, p, FAKE, FAKE, None, None, 2, 4, 4, 8, 0.1, 0, 0, FAKE,
                                          None, ws, 1 << 30, None, None),
    ]
    for call in calls:
        for bad in BAD_POOLS:
            assert call(_pages(**bad)) == 1, bad
        assert call(_pages(dtype=7)) == 2
        assert call(None) == 1


def test_resize_refusals(lib):
    base = dict(t=FAKE, c=FAKE, r=FAKE, w=FAKE, extra=0, page=16, B=2, P=4, n=10)

    def call(**kw):
        a = dict(base, **kw)
        return lib.spec_cache_resize(a["t"], a["c"], a["r"], a["w"], a["extra"], a["page"], a["B"], a["P"], a["n"],
                                     None, None)
    for bad in (dict(t=None), dict(c=None), dict(r=None), dict(w=None), dict(extra=-1), dict(page=12), dict(page=4),
                dict(B=0), dict(B=8193), dict(P=0), dict(n=0), dict(n=2 ** 31 - 1)):
        assert call(**bad) == 1, bad


def test_fork_refusals(lib):
    assert lib.spec_cache_fork_workspace_bytes(0) == 0 and lib.spec_cache_fork_workspace_bytes(8193) == 0
    assert lib.spec_cache_fork_workspace_bytes(100) >= 1200
    p = _pages()
    base = dict(t=FAKE, c=FAKE, r=FAKE, l=FAKE, s=FAKE, d=FAKE, F=2, S=4, P=8, ws=FAKE, n=4096)

    def call(**kw):
        a = dict(base, **kw)
        return lib.spec_cache_fork(p, a["t"], a["c"], a["r"], a["l"], a["s"], a["d"], a["F"], a["S"],
                                   a["P"], a["ws"], a["n"], None, None)
    for bad in (dict(t=None), dict(c=None), dict(r=None), dict(l=None), dict(s=None), dict(d=None), dict(F=0),
                dict(F=8193), dict(S=0), dict(S=8193), dict(P=0)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 4 and call(n=8) == 4 and call(ws=ctypes.c_void_p(0x10010)) == 4


def test_append_and_commit_refusals(lib):
    base = dict(p=_pages(), t=FAKE, l=FAKE, k=FAKE, v=FAKE, sb=1024, sn=128, sh=64, B=2, N=4, P=8)

    def app(**kw):
        a = dict(base, **kw)
        return lib.spec_cache_append(a["p"], a["t"], a["l"], a["k"], a["v"], a["sb"], a["sn"], a["sh"],
                                     None, a["B"], a["N"], a["P"], None, None)
    for bad in (dict(t=None), dict(l=None), dict(k=None), dict(v=None), dict(k=ctypes.c_void_p(0x10008)), dict(sb=4),
                dict(sn=-128), dict(sh=63), dict(B=0), dict(B=1 << 16), dict(N=0), dict(P=0),
                dict(p=_pages(layers=2))):
        assert app(**bad) == 1, bad

    def com(t=FAKE, l=FAKE, a=FAKE, new=FAKE, B=2, N=4, P=8):
        return lib.spec_cache_commit(_pages(), t, l, FAKE, a, new, B, N, P, None, None)
    for bad in (dict(t=None), dict(l=None), dict(a=None), dict(new=None), dict(B=0), dict(B=1 << 16), dict(N=0),
                dict(N=65), dict(P=0)):
        assert com(**bad) == 1, bad


def test_attention_refusals(lib):
    size = lib.spec_tree_attention_workspace_bytes
    assert size(2, 4, 4, 2, 64) > 0
    for bad in ((0, 4, 4, 2, 64), (1 << 16, 4, 4, 2, 64), (2, 0, 4, 2, 64), (2, 65, 4, 2, 64), (2, 4, 3, 2, 64),
                (2, 4, 1, 2, 64), (2, 4, 130, 2, 64), (2, 4, 4, 2, 136), (2, 4, 4, 2, 12), (2, 4, 4, 0, 64)):
        assert size(*bad) == 0, bad
    base = dict(q=FAKE, sb=1024, sn=256, sh=64, p=_pages(), t=FAKE, l=FAKE, B=2, N=4, Hq=4, P=8, scale=0.1, w=0, s=0,
                o=FAKE, ws=FAKE, n=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return lib.spec_tree_attention(a["q"], a["sb"], a["sn"], a["sh"], a["p"], a["t"], a["l"], None,
                                       None, a["B"], a["N"], a["Hq"], a["P"], a["scale"], a["w"], a["s"], a["o"], None,
                                       a["ws"], a["n"], None, None)
    for bad in (dict(q=None), dict(t=None), dict(l=None), dict(o=None), dict(q=ctypes.c_void_p(0x10008)),
                dict(o=ctypes.c_void_p(0x10008)), dict(sb=4), dict(sn=-8), dict(sh=60), dict(B=0), dict(N=65),
                dict(Hq=3), dict(P=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(w=-1),
                dict(s=-1), dict(p=_pages(layers=2)), dict(p=_pages(head_dim=136, head_stride=136, token_stride=272,
                                                                    page_stride=16 * 272))):
        assert call(**bad) == 1, bad
    assert call(p=_pages(dtype=0)) == 2                            # float32 caches
    assert call(ws=None) == 4 and call(n=0) == 4 and call(ws=ctypes.c_void_p(0x10010)) == 4
