"""Tree attention over a 4-bit cache where scores are so large that their scaled form is coarse: what two keys weigh
beside each other must not depend on where the work is divided between them."""
import pytest
import torch

import cache4_helpers as c4

pytestmark = pytest.mark.gpu

SHAPES = [(1, 16, 128), (3, 16, 128), (1, 16, 64), (3, 16, 64), (2, 32, 64)]  # nodes, query heads of one key head, head_dim


class Keys:
    """Pages of zeros whose scales are 2^(byte / 8 - 19) for the first 32 channels of the keys and 1 for all else."""

    def __init__(self, pages, page, D, byte):
        self.page, self.D = page, D
        self.pool = torch.full((pages, 1, c4.page_bytes(page, D)), 0x88, dtype=torch.uint8)
        self.at = {kind: c4.places(page, D, kind) for kind in "kv"}
        for kind in "kv":
            self.pool[..., self.at[kind][2]] = 152
        self.pool[..., self.at["k"][2][:, 0]] = byte

    def _put(self, kind, j, channels, code):
        at, shift = (x[j % self.page, channels] for x in self.at[kind][:2])
        row = self.pool[j // self.page, 0]
        for n in (0, 4):                                               # two channels may share a byte
            b = at[shift == n]
            row[b] = (row[b] & ~(15 << n) & 255) | (code + 8) << n

    def key(self, j, codes):
        for channel, code in codes.items():
            self._put("k", j, torch.tensor([channel]), code)

    def value(self, j, code):
        self._put("v", j, torch.arange(self.D), code)

    def numbers(self, n):
        return [x.flatten(0, 1)[:n, 0] for x in c4.decode(self.pool, self.page, self.D)]


def _run(q, keys, n0, scale):
    """The same keys for every request."""
    import speculative_decoding_verification_69_gb300 as sv
    B, P = q.shape[0], keys.pool.shape[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    st = torch.zeros(1, **i32)
    o, l = sv.tree_attention4(q.cuda(), keys.pool.repeat(B, 1, 1).cuda(), torch.arange(B * P, **i32).view(B, P),
                              torch.full((B,), n0, **i32), keys.page, scale=scale, return_lse=True, dev_status=st)
    assert int(st) == 0
    return o.double().cpu(), l.double().cpu()


def _requests(kind):
    return 1 if kind == "one" else torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("requests", ["one", "one for every SM"])
@pytest.mark.parametrize("N,hq,D", SHAPES)
@pytest.mark.parametrize("first", [0, 1])
def test_the_larger_of_two_scores_one_step_apart(first, N, hq, D, requests, dtype):
    """Two keys, one in each of two tiles, whose scores are neighbours among the float32 numbers from 1.5 * 2^31 on (1.5 * 2^29,
    of which the kernel has a quarter, for float16), and so 256 apart when scaled: the larger one has all the weight.  One
    request's tiles are two CTAs'; with a request for every SM both are one CTA's, and its two streams take one each.
    The weight, 2^7 but for 2^-21, is held in float16 to half a step and the result is rounded once."""
    B, bf = _requests(requests), dtype == torch.bfloat16
    scale, step = (1.0, 256.0) if bf else (4.0, 64.0)
    keys = Keys(4, 64, D, 248)                                         # 2^12
    q = torch.zeros((B, N, hq, D), dtype=dtype)
    q[..., 0], q[..., 32], q[..., 33] = step * 512, step, step * (torch.arange(hq) % 16)  # 16 pairs of neighbours
    for j, up, x in zip((140, 70) if first else (70, 140), (0, 1), (-3, 5)):
        keys.key(j, {0: 6, 32: up, 33: 1})
        keys.value(j, x)
    o, l = _run(q, keys, 200, scale)
    assert ((o - 5.0).abs() <= 5.0 * (torch.finfo(dtype).eps / 2 + 2.0 ** -11 + 2.0 ** -16)).all()
    score = scale * step * (512.0 * 6 * 2 ** 12 + 1 + torch.arange(hq).double() % 16)
    assert ((l - score).abs() <= score * 2.0 ** -21).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("requests", ["one", "one for every SM"])
@pytest.mark.parametrize("N,hq,D", SHAPES)
@pytest.mark.parametrize("low", [7340100, 11629060, 11629077])
def test_weights_beside_a_reference_that_moves(low, N, hq, D, requests, dtype):
    """127 keys of one score in each of two tiles and one in the third that is larger by 7, so that a single token's
    reference moves: the scaled scores lie near 2^23, where float32 rounds a reference by up to 1/2, or on both
    sides of 2^24, beyond which references are taken off before scaling.  The scores are whole numbers
    that float32 holds; so what the keys weigh beside each other follows from their exact difference, to half a step of float16
    and 2^-15, and the result is rounded once."""
    B, n0 = _requests(requests), 300
    keys = Keys(5, 64, D, 232)                                         # 2^10
    q = torch.zeros((B, N, hq, D), dtype=dtype)
    left = low - 7 * 1024 * 1024
    q[..., 0], q[..., 1], q[..., 2] = 1024, 1024 * (left >> 22), (left & (1 << 22) - 1) >> 12
    q[..., 33], q[..., 34], q[..., 35] = left & 4032, left & 63, torch.arange(hq) % 16
    q[..., 32] = 7
    many = {0: 7, 1: 4, 2: 4, 33: 1, 34: 1, 35: 1}
    for j in list(range(127)) + list(range(128, 255)) + [290]:
        keys.key(j, {**many, 32: int(j == 290)})
        keys.value(j, -7 if j == 290 else 2)
    k, v = keys.numbers(n0 + 1)
    score = q[0, 0].double() @ k.T
    assert score[:, 0].tolist() == [low + i % 16 for i in range(hq)] and (score[:, 290] - score[:, 0] == 7).all()
    o, l = _run(q, keys, n0, 1.0)
    p = torch.softmax(score, 1)
    want, mag = p @ v, p @ v.abs()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + (2.0 ** -11 + 2.0 ** -15) * mag
    err = (o - want).abs()
    assert (err <= tol).all(), "worst %g of its bound" % float((err / tol).max())
    assert ((l - torch.logsumexp(score, 1)).abs() <= low * 2.0 ** -21).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,hq,hkv,D", [(1, 8, 2, 128), (5, 8, 2, 128), (16, 8, 2, 128), (5, 8, 4, 64), (1, 8, 4, 64)])
def test_rows_beside_one_of_large_scores(N, hq, hkv, D, dtype):
    """Every fourth head's scores are 2^14 times as large, or beyond 2^40 (bfloat16): the other rows, which share the
    kernel's tiles with it, are as ever."""
    import cache_helpers as ch
    import speculative_decoding_verification_69_gb300 as sv
    g = torch.Generator(device="cuda").manual_seed(N + D)
    lens, page = [40, 1000, 0, 3000], 16
    P = -(-(max(lens) + N) // page)
    table, _, _, cl = ch.make_table(g, lens, N, page, P, 4 * P)
    pool = c4.make_pool(g, 4 * P, hkv, page, D)
    parent = ch.random_parents(g, 4, N)
    q = torch.randn((4, N, hq, D), generator=g, device="cuda").to(dtype)
    q[:, :, ::4] *= 2.0 ** 14 if dtype == torch.float16 else 2.0 ** 40
    q.clamp_(-6e4 if dtype == torch.float16 else -1e30, 6e4 if dtype == torch.float16 else 1e30)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = sv.tree_attention4(q, pool, table, cl, page, parent, return_lse=True, dev_status=st)
    ref = c4.ref_attention(q, pool, page, table, cl, parent)
    assert int(st) == 0 and torch.isfinite(o).all() and torch.isfinite(l).all()
    rest = [h for h in range(hq) if h % 4]
    ch.check_attention(o[:, :, rest], l[:, :, rest], tuple(x[:, :, rest] for x in ref), dtype, D)
    # of the large ones at least the sum: the largest score, to float32
    big = l[:, :, ::4].double().cpu()
    want, scale = ref[1][:, :, ::4].double().cpu(), ref[3][:, :, ::4].double().cpu()
    assert ((big - want).abs() <= (D + 4) * 2.0 ** -24 * scale + 2.0 ** -18 + 2.0 ** -22 * want.abs()).all()
