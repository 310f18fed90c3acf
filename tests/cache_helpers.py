"""Plain 64-bit implementations of the paged-cache operators for the tests,
request by request from the definitions in include/spec_cache.h."""
import math

import torch


def paths(parent, N):
    """Root-to-node paths of one request; parent None: a chain."""
    out = []
    for n in range(N):
        p, m = [], n
        while m >= 0:
            p.append(m)
            up = (m - 1 if parent is None else int(parent[m])) if m > 0 else -1
            m = up if 0 <= up < m else -1
        out.append(p[::-1])
    return out


def seen_positions(n0, path, window, sinks):
    """Cache positions that the last node of `path` sees."""
    tip = n0 + len(path) - 1

    def ok(place):
        return not window or tip - place < window or place < sinks
    if window:
        ctx = sorted(set(range(0, min(n0, sinks))) | set(range(max(0, tip - window + 1), n0)))
    else:
        ctx = list(range(n0))
    return ctx + [n0 + m for d, m in enumerate(path) if ok(n0 + d)]


def ref_attention(q, k, v, table, lens, parent, node_count=None, scale=None, window=0, sinks=0):
    """out, lse and sum_j p_j |v_j| (the scale of the rounding errors), float64 on the CPU."""
    B, N, Hq, D = q.shape
    page, hkv = k.shape[1], k.shape[2]
    G = Hq // hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    mag = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    smax = torch.zeros((B, N, Hq), dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    qc = q.detach().cpu().double()
    for b in range(B):
        n0 = int(lens[b])
        cnt = N if node_count is None else max(0, min(N, int(node_count[b])))
        if cnt == 0:
            continue
        pl = paths(None if parent is None else parent[b].tolist(), cnt)
        sets = [seen_positions(n0, p, window, sinks) for p in pl]
        every = sorted(set().union(*map(set, sets)))
        at = torch.tensor(every, device=k.device)
        pg = table[b].long()[at // page]
        kk, vv = k[pg, at % page].cpu().double(), v[pg, at % page].cpu().double()
        index = {j: i for i, j in enumerate(every)}
        for n in range(cnt):
            sel = torch.tensor([index[j] for j in sets[n]])
            kn, vn = kk[sel], vv[sel]                               # [L, hkv, D]
            qn = qc[b, n].view(hkv, G, D)
            z = torch.einsum("hgd,lhd->hgl", qn, kn) * scale
            p = torch.softmax(z, -1)
            lse[b, n] = torch.logsumexp(z, -1).view(Hq)
            smax[b, n] = (torch.einsum("hgd,lhd->hgl", qn.abs(), kn.abs()).amax(-1) * scale).view(Hq)
            out[b, n] = torch.einsum("hgl,lhd->hgd", p, vn).reshape(Hq, D)
            mag[b, n] = torch.einsum("hgl,lhd->hgd", p, vn.abs()).reshape(Hq, D)
    return out, lse, mag, smax


def check_attention(out, lse, ref, dtype, D):
    """Bounds from the arithmetic of the definition: the weights and the result
    are each rounded once to the dtype (unit roundoff u), scores and sums are
    float32 (D products; the approximate exponential is good to 2^-21)."""
    o, l, mag, smax = ref
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    score = (D + 4) * 2.0 ** -24 * smax                             # absolute error of a score
    tol = u * o.abs() + (u + 2.0 ** -15 + 2.0 * score.unsqueeze(-1)) * mag + 1e-7
    err = (out.detach().cpu().double() - o).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), "worst %g of its bound" % float((err / tol).max())
    if lse is not None:
        lc = lse.detach().cpu().double()
        empty = torch.isinf(l)
        assert torch.equal(torch.isneginf(lc), empty)
        lt = score + 2.0 ** -18 + 2.0 ** -22 * l.abs()
        d = (lc - l).abs()[~empty]
        assert (d <= lt[~empty]).all(), "lse: worst %g of its bound" % float((d / lt[~empty]).max())


class Pages:
    """Page bookkeeping with Python lists."""

    def __init__(self, table, count, ref, lens=None):
        self.P = table.shape[1]
        self.rows = [r[:c] for r, c in zip(table.tolist(), count.tolist())]
        self.ref = ref.tolist()
        self.len = None if lens is None else lens.tolist()

    def _drop(self, row, keep):
        while len(row) > keep:
            self.ref[row.pop()] -= 1

    def _take(self, grows):
        """Lists of pages for each item, None where the free pages do not reach."""
        free = [p for p, r in enumerate(self.ref) if r == 0]
        got, asked, at = [], 0, 0
        for g in grows:
            asked += g
            if asked <= len(free):
                got.append(free[at:at + g])
                at += g
            else:
                got.append(None if g else [])
        for x in got:
            for p in x or []:
                self.ref[p] = 1
        return got

    def resize(self, want, extra, page):
        need = [len(r) if w < 0 else min(self.P, -(-(w + extra) // page)) for r, w in zip(self.rows, want)]
        for r, n in zip(self.rows, need):
            self._drop(r, n)
        got = self._take([n - len(r) for r, n in zip(self.rows, need)])
        for r, g in zip(self.rows, got):
            r.extend(g or [])
        return any(g is None for g in got)

    def fork(self, src, dst, page):
        """Returns the pages to copy, (from, to, tokens), and whether pages were missing."""
        S = len(self.rows)
        valid = []
        for f, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < S and 0 <= d < S and d not in src and d not in dst[:f]
            valid.append(ok and 0 <= self.len[s] <= len(self.rows[s]) * page)
        for f, d in enumerate(dst):
            if valid[f]:
                self._drop(self.rows[d], 0)
        part = [self.len[s] % page if ok else 0 for s, ok in zip(src, valid)]
        got = self._take([1 if p else 0 for p in part])
        copies = []
        for f, (s, d) in enumerate(zip(src, dst)):
            if not valid[f]:
                continue
            if got[f] is None:
                self.len[d] = 0
                continue
            full = self.len[s] // page
            self.rows[d] = self.rows[s][:full] + got[f]
            for p in self.rows[s][:full]:
                self.ref[p] += 1
            self.len[d] = self.len[s]
            if part[f]:
                copies.append((self.rows[s][full], got[f][0], part[f]))
        return copies, any(g is None for g in got)

    def check(self, table, count, ref, lens=None):
        assert count.tolist() == [len(r) for r in self.rows]
        assert ref.tolist() == self.ref
        for got, r in zip(table.tolist(), self.rows):
            assert got[:len(r)] == r
            assert all(p == -1 for p in got[len(r):])
        if lens is not None:
            assert lens.tolist() == self.len


def make_pool(g, pages, page, heads, D, dtype, layers=None, hnd=False, device="cuda"):
    lead = () if layers is None else (layers,)
    shape = lead + ((pages, heads, page, D) if hnd else (pages, page, heads, D))
    x = torch.randn(shape, generator=g, device=device, dtype=torch.float32).to(dtype)
    return x.transpose(-2, -3) if hnd else x


def make_table(g, lens, extra, page, P, pages, device="cuda"):
    """A table with pages for lens + extra tokens of every slot, drawn in random order."""
    held = [-(-(n + extra) // page) for n in lens]
    perm = torch.randperm(pages, generator=g, device=device).int().tolist()
    assert sum(held) <= pages and max(held) <= P
    rows, at = [], 0
    for h in held:
        rows.append(perm[at:at + h] + [-1] * (P - h))
        at += h
    ref = [0] * pages
    for p in perm[:at]:
        ref[p] = 1
    i32 = dict(dtype=torch.int32, device=device)
    return (torch.tensor(rows, **i32), torch.tensor(held, **i32), torch.tensor(ref, **i32),
            torch.tensor(lens, **i32))


def random_parents(g, B, N, chain=0.5, device="cuda"):
    rows = []
    for _ in range(B):
        r = [-1]
        for n in range(1, N):
            u = torch.rand((2,), generator=g, device=device).tolist()
            r.append(n - 1 if u[0] < chain else int(u[1] * n))
        rows.append(r)
    return torch.tensor(rows, dtype=torch.int32, device=device)
