"""Cases of the paged-cache operators: tree attention over a paged cache (with and
without a sliding window and sink tokens), appending drafted tokens, committing
an accepted path, and forking requests.

Each case has a plain form in elementary torch operations (32-bit arithmetic,
one rounding at the end) and, with `own` set, the calls a user makes of the
package.  `exact` restates each operator in 64 bits from its definition.

  attention  out[b, n, h] = softmax_j(scale * q[b, n, h] . k_j) v_j over the
             positions j that node n of request b sees: the committed positions
             [0, len) and the node's ancestors and itself (node m of the tree
             sits at position len + m of the cache), with a window only those
             less than `window` tokens back along the node's own path, or among
             the first `sinks` tokens.
  append     pages past each request's length returned, pages for the drafted
             tokens taken (lowest free page first), their keys and values
             written.
  commit     the accepted nodes of each tree moved to follow its root, in every
             layer, and the lengths advanced.
  fork       requests continued in other slots: full pages shared, the last
             partial page copied in every layer.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    """Head shapes: 32 query heads on 8 key heads of 128 and 64 on 8 of 64, the
    attention shapes of the model families whose vocabularies the benchmark
    uses; K = 8 drafts (9 rows with the root) as its workloads have."""
    return [
        # one sequence, one token, a short context: the call's latency
        dict(name="token_b1", op="attention", B=1, N=1, hq=32, hkv=8, D=128, page=16, ctx=1000,
             ragged=False, chain=True, window=0, sinks=0, dtype="bf16", hnd=False),
        # a batch verifying 8 linear drafts each
        dict(name="chain_b32", op="attention", B=32, N=9, hq=32, hkv=8, D=128, page=16, ctx=4096,
             ragged=True, chain=True, window=0, sinks=0, dtype="bf16", hnd=False),
        # the largest trees on a full batch: the product as costly as the cache's bytes
        dict(name="tree64_b64", op="attention", B=64, N=64, hq=32, hkv=8, D=128, page=32, ctx=4096,
             ragged=True, chain=False, window=0, sinks=0, dtype="f16", hnd=True),
        # one long sequence with a tree of 16: few rows, the axis of keys split over the GPU
        dict(name="tree16_long", op="attention", B=1, N=16, hq=32, hkv=8, D=128, page=128,
             ctx=131071, ragged=False, chain=False, window=0, sinks=0, dtype="bf16", hnd=False),
        # windowed layers of a large serving batch: short key ranges, many requests
        dict(name="window128_b512", op="attention", B=512, N=9, hq=64, hkv=8, D=64, page=16,
             ctx=4096, ragged=True, chain=True, window=128, sinks=0, dtype="bf16", hnd=False),
        # long streams with a window and four sink tokens, trees of 16
        dict(name="window4k_sinks", op="attention", B=8, N=16, hq=32, hkv=8, D=128, page=64,
             ctx=65536, ragged=True, chain=False, window=4096, sinks=4, dtype="bf16", hnd=False),
        # page traffic of one decoding step of a few requests
        dict(name="append_step", op="append", B=8, N=9, hkv=8, D=128, page=16, ctx=2000,
             dtype="bf16", hnd=False),
        # prompts entering the cache
        dict(name="append_prompt", op="append", B=16, N=2047, hkv=8, D=128, page=64, ctx=500,
             dtype="bf16", hnd=True),
        # accepted paths of a few small trees
        dict(name="commit_b4", op="commit", B=4, N=8, layers=36, hkv=8, D=128, page=16, ctx=100,
             dtype="bf16", hnd=False),
        # accepted paths of a batch of trees of 64
        dict(name="commit_b128", op="commit", B=128, N=64, layers=36, hkv=8, D=128, page=32,
             ctx=60, dtype="bf16", hnd=False),
        # one request continued eight ways
        dict(name="fork_8", op="fork", S=1, F=8, layers=36, hkv=8, D=128, page=16, ctx=777,
             dtype="bf16", hnd=False),
        # a batch of requests continued four ways each
        dict(name="fork_64", op="fork", S=16, F=64, layers=24, hkv=8, D=64, page=64, ctx=900,
             dtype="bf16", hnd=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "attention", "append", "commit", "fork"])
    hkv, group, D = rng.choice([(8, 4, 128), (8, 8, 64), (8, 4, 64), (4, 7, 128), (1, 8, 128), (16, 1, 96),
                                (2, 16, 64), (8, 5, 80)])
    case = dict(op=op, hkv=hkv, D=D, page=rng.choice([8, 16, 32, 64, 128, 256]),
                dtype=rng.choice(["bf16", "bf16", "f16"]), hnd=rng.random() < 0.5)
    if op == "attention":
        N, B = _log(rng, 1, 64), _log(rng, 1, 256)
        # keys and score rows within those of the largest listed cases
        top = min(131072, (64 * 4096 * 8 * 128) // (B * hkv * D), (64 * 4096 * 32 * 64) // (B * hkv * group * N))
        ctx = _log(rng, 1, max(1, top))
        window = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
        case.update(B=B, N=N, hq=hkv * group, ctx=ctx, ragged=rng.random() < 0.7, chain=rng.random() < 0.4,
                    window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0)
    elif op == "append":
        B = _log(rng, 1, 128)
        case.update(B=B, N=_log(rng, 1, max(1, 32768 // B)), ctx=_log(rng, 1, 1000))
    elif op == "commit":
        case.update(B=_log(rng, 1, 128), N=_log(rng, 2, 64), layers=_log(rng, 1, 36), ctx=_log(rng, 1, 100))
    else:
        S = _log(rng, 1, 16)
        case.update(S=S, F=S * rng.randint(1, 4), layers=_log(rng, 1, 24), ctx=_log(rng, 1, 900))
    return case


# ------------------------------------------------------------------ inputs

def _pool(g, shape, hnd, dtype, dev):
    """Keys or values of a pool of pages [..., pages, page, heads, D]; hnd: the
    heads lie outside the tokens of a page in memory."""
    if hnd:
        shape = shape[:-3] + (shape[-2], shape[-3], shape[-1])
    x = torch.empty(shape, dtype=dtype, device=dev)
    x.normal_(generator=g)
    return x.transpose(-2, -3) if hnd else x


def _trees(g, B, N, chain_prob, dev):
    """parent [B, N] int32: node n under node n - 1 with probability chain_prob,
    else under any earlier node (the benchmark's candidate trees)."""
    n = torch.arange(N, device=dev)
    other = (torch.rand((B, N), generator=g, device=dev) * n).long()
    chain = torch.rand((B, N), generator=g, device=dev) < chain_prob
    parent = torch.where(chain, n - 1, torch.minimum(other, (n - 1).clamp(min=0)))
    parent[:, 0] = -1
    return parent.to(torch.int32).contiguous()


def _paths(g, parent, dev):
    """An accepted path in every tree, as tree verification returns it: node
    indices root to leaf (the root left out), -1 after them, and its length."""
    B, N = parent.shape
    leaf = (torch.rand((B,), generator=g, device=dev) * N).long().cpu().tolist()
    par = parent.cpu().tolist()
    nodes, length = torch.full((B, N), -1, dtype=torch.int32), []
    for b in range(B):
        path, n = [], leaf[b]
        while n > 0:
            path.append(n)
            n = par[b][n]
        path.reverse()
        nodes[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        length.append(len(path))
    return nodes.to(dev), torch.tensor(length, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c, op, page, dtype = case, case["op"], case["page"], DTYPES[case["dtype"]]
    hkv, D = c["hkv"], c["D"]
    B = c["S"] if op == "fork" else c["B"]
    extra = c["N"] if op != "fork" else 0
    if op == "attention" and not c["ragged"]:
        lens = torch.full((B,), c["ctx"], dtype=torch.int32, device=dev)
    else:  # contexts of between half and all of ctx
        lo = (c["ctx"] + 1) // 2
        lens = (lo + torch.rand((B,), generator=g, device=dev) * (c["ctx"] - lo + 1)).int().clamp(max=c["ctx"])
    slots = B if op != "fork" else B + c["F"]
    P = (c["ctx"] + extra + page - 1) // page + 1
    total = lens + (extra if op in ("attention", "commit") else 0)
    held = ((total + page - 1) // page).int()
    n_held = int(held.sum())
    spare = {"append": B * ((extra + page - 1) // page + 1) + 8, "fork": c.get("F", 0) + 8}.get(op, 3)
    pages = B * ((c["ctx"] + extra + page - 1) // page) + spare  # a pool for every request at its longest
    perm = torch.randperm(pages, generator=g, device=dev).int()
    mine = torch.arange(P, device=dev) < held.view(-1, 1)
    table = torch.full((slots, P), -1, dtype=torch.int32, device=dev)
    head = table[:B]
    head[mine] = perm[:n_held]
    ref = torch.zeros((pages,), dtype=torch.int32, device=dev)
    ref[perm[:n_held].long()] = 1
    count = torch.zeros((slots,), dtype=torch.int32, device=dev)
    count[:B] = held
    cache_len = torch.zeros((slots,), dtype=torch.int32, device=dev)
    cache_len[:B] = lens
    layers = (c["layers"],) if "layers" in c else ()
    k = _pool(g, layers + (pages, page, hkv, D), c["hnd"], dtype, dev)
    v = _pool(g, layers + (pages, page, hkv, D), c["hnd"], dtype, dev)
    s = dict(case=dict(case), k=k, v=v, table=table, count=count, ref=ref, len=cache_len)
    if op == "attention":
        # the query rows as they leave a fused projection of queries, keys and values
        qkv = torch.empty((B, c["N"], c["hq"] + 2 * hkv, D), dtype=dtype, device=dev).normal_(generator=g)
        s["q"] = qkv[:, :, :c["hq"]].mul_(2.0)
        s["parent"] = _trees(g, B, c["N"], 1.0 if c["chain"] else 0.5, dev)
    elif op == "append":
        kv = torch.empty((B, c["N"], 2 * hkv, D), dtype=dtype, device=dev).normal_(generator=g)
        s["k_new"], s["v_new"] = kv[:, :, :hkv], kv[:, :, hkv:]
        s["want"] = (cache_len + c["N"]).int()
    elif op == "commit":
        s["nodes"], s["accept"] = _paths(g, _trees(g, B, c["N"], 0.5, dev), dev)
        s["new_len"] = torch.empty_like(cache_len)
    else:
        s["src"] = (torch.arange(c["F"], device=dev) % B).int()
        s["dst"] = (B + torch.randperm(c["F"], generator=g, device=dev)).int()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "commit": _own_commit, "fork": _own_fork}[op](s)
    return {"attention": _attention, "append": _append, "commit": _commit, "fork": _fork}[op](s)


def _own_attention(s):
    import speculative_decoding_verification_69_gb300 as sv
    c = s["case"]
    out, lse = sv.tree_attention(s["q"], s["k"], s["v"], s["table"], s["len"], s["parent"], window=c["window"],
                                 sinks=c["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_append(s):
    import speculative_decoding_verification_69_gb300 as sv
    page = s["case"]["page"]
    sv.cache_resize(s["table"], s["count"], s["ref"], s["len"], page)
    sv.cache_resize(s["table"], s["count"], s["ref"], s["want"], page)
    sv.cache_append(s["k"], s["v"], s["table"], s["len"], s["k_new"], s["v_new"])
    return {"k": s["k"], "v": s["v"], "table": s["table"], "count": s["count"], "ref": s["ref"]}


def _own_commit(s):
    import speculative_decoding_verification_69_gb300 as sv
    sv.cache_commit(s["k"], s["v"], s["table"], s["len"], s["nodes"], s["accept"], new_len=s["new_len"])
    return {"k": s["k"], "v": s["v"], "len": s["new_len"]}


def _own_fork(s):
    import speculative_decoding_verification_69_gb300 as sv
    sv.cache_fork(s["k"], s["v"], s["table"], s["count"], s["ref"], s["len"], s["src"], s["dst"])
    return {"k": s["k"], "v": s["v"], "table": s["table"], "count": s["count"], "ref": s["ref"], "len": s["len"]}


def _attention(s):
    c, q, k, v, table, lens, parent = s["case"], s["q"], s["k"], s["v"], s["table"], s["len"].long(), s["parent"].long()
    B, N, hq, D = q.shape
    hkv, page = c["hkv"], c["page"]
    L = c["ctx"] + N
    pos = torch.arange(L, device=q.device)
    held = table[:, :(L + page - 1) // page].long().clamp(min=0)
    kk = k[held].flatten(1, 2)[:, :L].float()
    vv = v[held].flatten(1, 2)[:, :L].float()
    # ancestors of each node, itself among them: powers of (I + parent links)
    node = torch.arange(N, device=q.device)
    link = (parent.unsqueeze(-1) == node).float() + torch.eye(N, device=q.device)
    anc = torch.matrix_power(link, 64) > 0 if N > 1 else link > 0
    depth = anc.sum(-1) - 1
    node_of = pos - lens.view(B, 1)                               # [B, L]
    in_tree = (node_of >= 0) & (node_of < N)
    at = node_of.clamp(0, N - 1)
    own_path = torch.gather(anc, 2, at.unsqueeze(1).expand(B, N, L))
    seen = torch.where(in_tree.unsqueeze(1), own_path, (node_of < 0).unsqueeze(1))
    if c["window"]:
        key_pos = torch.where(in_tree, lens.view(B, 1) + torch.gather(depth, 1, at), pos.expand(B, L))
        row_pos = lens.view(B, 1) + depth
        near = row_pos.unsqueeze(-1) - key_pos.unsqueeze(1) < c["window"]
        seen = seen & (near | (key_pos < c["sinks"]).unsqueeze(1))
    qq = q.float().view(B, N, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D)
    z = torch.matmul(qq, kk.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(B, hkv, N, hq // hkv, L)
    z = z.masked_fill_(~seen.view(B, 1, N, 1, L), -math.inf)
    m = z.amax(-1, keepdim=True)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, hkv, -1, L), vv.permute(0, 2, 1, 3)).view(B, hkv, N, hq // hkv, D) / total
    lse = (m + total.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, N, hq, D).to(q.dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, N, hq)}


def _resize(table, count, ref, want, page):
    P = table.shape[1]
    need = torch.where(want < 0, count, (want + page - 1) // page).clamp(max=P)
    j = torch.arange(P, device=table.device, dtype=torch.int32)
    drop = (j >= need.view(-1, 1)) & (j < count.view(-1, 1))
    gone = table[drop].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table.masked_fill_(drop, -1)
    keep = torch.minimum(count, need)
    grow = need - keep
    free = torch.nonzero(ref == 0).squeeze(1)
    grow = torch.where(grow.cumsum(0) <= free.numel(), grow, torch.zeros_like(grow))
    fresh = (j >= keep.view(-1, 1)) & (j < (keep + grow).view(-1, 1))
    taken = free[:int(grow.sum())]
    table[fresh] = taken.int()
    ref[taken] = 1
    count.copy_(keep + grow)


def _append(s):
    page, table, lens = s["case"]["page"], s["table"], s["len"].long()
    _resize(table, s["count"], s["ref"], s["len"], page)
    _resize(table, s["count"], s["ref"], s["want"], page)
    pos = lens.view(-1, 1) + torch.arange(s["k_new"].shape[1], device=table.device)
    pg = torch.gather(table.long(), 1, pos // page)
    s["k"][pg, pos % page] = s["k_new"]
    s["v"][pg, pos % page] = s["v_new"]
    return {"k": s["k"], "v": s["v"], "table": table, "count": s["count"], "ref": s["ref"]}


def _commit(s):
    page, table, lens, nodes = s["case"]["page"], s["table"].long(), s["len"].long(), s["nodes"].long()
    B, N = nodes.shape
    step = torch.arange(N, device=table.device)
    real = step < s["accept"].long().view(-1, 1)
    src = (lens.view(-1, 1) + nodes)[real]
    dst = (lens.view(-1, 1) + 1 + step)[real]
    b = torch.arange(B, device=table.device).view(-1, 1).expand(B, N)[real]
    for x in (s["k"], s["v"]):
        x[:, table[b, dst // page], dst % page] = x[:, table[b, src // page], src % page]
    s["new_len"].copy_(s["len"] + 1 + s["accept"])
    return {"k": s["k"], "v": s["v"], "len": s["new_len"]}


def _fork(s):
    page, table, count, ref = s["case"]["page"], s["table"], s["count"], s["ref"]
    src, dst = s["src"].long(), s["dst"].long()
    want = torch.full_like(count, -1)
    want[dst] = 0
    _resize(table, count, ref, want, page)
    lens = s["len"].long()[src]
    full, used = lens // page, lens % page
    j = torch.arange(table.shape[1], device=table.device)
    share = j < full.view(-1, 1)
    rows = torch.where(share, table[src], torch.full_like(table[src], -1))
    both = rows[share].long()
    ref.index_add_(0, both, torch.ones_like(both, dtype=torch.int32))
    part = used > 0
    fresh = torch.nonzero(ref == 0).squeeze(1)[:int(part.sum())]
    ref[fresh] = 1
    old = torch.gather(table[src].long(), 1, full.view(-1, 1)).squeeze(1)[part]
    rows[part.nonzero().squeeze(1), full[part]] = fresh.int()
    table[dst] = rows
    count[dst] = (full + part).int()
    s["len"][dst] = lens.int()
    t = torch.arange(page, device=table.device)
    real = t < used[part].view(-1, 1)
    f, t = fresh.view(-1, 1).expand_as(real)[real], t.expand_as(real)[real]
    o = old.view(-1, 1).expand_as(real)[real]
    for x in (s["k"], s["v"]):
        x[:, f, t] = x[:, o, t]
    return {"k": s["k"], "v": s["v"], "table": table, "count": count, "ref": ref, "len": s["len"]}


# ------------------------------------------------------------------ what one pass needs

def work(case):
    """The positions and pages of a case are drawn: their expectations."""
    c, token = case, case["hkv"] * case["D"] * 2 * 2  # bytes of one token's key and value
    mean = c["ctx"] if not c.get("ragged", True) else 0.75 * c["ctx"]
    if c["op"] == "attention":
        keys = mean + c["N"]
        if c["window"]:
            keys = min(keys, c["window"] + c["sinks"] + c["N"])
        rows = c["B"] * c["N"] * c["hq"]
        return {"bytes": c["B"] * keys * token + rows * (c["D"] * 4 + 4) + c["B"] * (keys / c["page"] + c["N"] + 1) * 4,
                "flops": 4.0 * rows * c["D"] * keys}
    if c["op"] == "append":
        return {"bytes": 2.0 * c["B"] * c["N"] * token + 16.0 * c["B"] * (c["N"] / c["page"] + 1), "flops": 0}
    if c["op"] == "commit":  # mean depth of a uniform node of these trees
        d = 0.0
        depth = [0.0]
        for n in range(1, c["N"]):
            depth.append(1.0 + 0.5 * depth[n - 1] + 0.5 * sum(depth) / n)
        d = sum(depth) / c["N"]
        return {"bytes": 2.0 * c["B"] * d * token * c["layers"] + 8.0 * c["B"], "flops": 0}
    return {"bytes": 2.0 * c["F"] * token * c["layers"] * (c["page"] - 1) / 2 + 12.0 * c["F"] * mean / c["page"],
            "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "commit": _exact_commit, "fork": _exact_fork}[
        case["op"]](s)


def _exact_attention(s):
    """Request by request, over the positions that some node of it sees."""
    c, q = s["case"], s["q"]
    B, N, hq, D = q.shape
    hkv, page, G = c["hkv"], c["page"], hq // c["hkv"]
    lens, parent = s["len"].tolist(), s["parent"].tolist()
    out = torch.empty((B, N, hq, D), dtype=torch.float64, device=q.device)
    lse = torch.empty((B, N, hq), dtype=torch.float64, device=q.device)
    for b in range(B):
        n0, chains = lens[b], []
        for n in range(N):
            chain = [n]
            while chain[-1] > 0:
                chain.append(parent[b][chain[-1]])
            chains.append(chain[::-1])
        first = max(0, n0 - c["window"] + 1) if c["window"] else 0
        head = torch.arange(min(c["sinks"], first), device=q.device)
        at = torch.cat([head, torch.arange(first, n0 + N, device=q.device)])
        pg = s["table"][b].long()[at // page]
        kk, vv = s["k"][pg, at % page].double(), s["v"][pg, at % page].double()
        seen = torch.zeros((N, n0 + N), dtype=torch.bool)
        for n, chain in enumerate(chains):
            tip = n0 + len(chain) - 1
            if c["window"]:
                seen[n, max(0, tip - c["window"] + 1):n0] = True
                seen[n, :min(c["sinks"], n0)] = True
            else:
                seen[n, :n0] = True
            for d, m in enumerate(chain):
                if not c["window"] or tip - (n0 + d) < c["window"] or n0 + d < c["sinks"]:
                    seen[n, n0 + m] = True
        seen = seen.to(q.device)[:, at]
        rows = q[b].double().view(N, hkv, G, D)
        z = torch.einsum("nhgd,lhd->nhgl", rows, kk) / math.sqrt(D)
        z = torch.where(seen.view(N, 1, 1, -1), z, torch.full_like(z, -math.inf))
        lse[b] = torch.logsumexp(z, -1).view(N, hq)
        out[b] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(z, -1), vv).reshape(N, hq, D)
    return {"out": out, "lse": lse}


def _exact_pages(table, count, ref, want, page):
    """Page lists as Python lists: frees first, then grants of the lowest free pages in request order."""
    lists = [row[:n] for row, n in zip(table, count)]
    need = [len(x) if w < 0 else min(-(-w // page), len(table[0])) for x, w in zip(lists, want)]
    for x, n in zip(lists, need):
        while len(x) > n:
            ref[x.pop()] -= 1
    free = [p for p, r in enumerate(ref) if r == 0]
    asked, at = 0, 0
    for x, n in zip(lists, need):
        grow = n - len(x)
        asked += grow
        if asked <= len(free):
            for p in free[at:at + grow]:
                ref[p] = 1
                x.append(p)
            at += grow
    return lists


def _exact_append(s):
    page, N = s["case"]["page"], s["k_new"].shape[1]
    ref, table = s["ref"].tolist(), s["table"].tolist()
    lists = _exact_pages(table, s["count"].tolist(), ref, s["len"].tolist(), page)
    padded = [x + [-1] * (len(table[0]) - len(x)) for x in lists]
    lists = _exact_pages(padded, [len(x) for x in lists], ref, s["want"].tolist(), page)
    k, v = s["k"].clone(), s["v"].clone()
    for b, n0 in enumerate(s["len"].tolist()):
        own_pages = torch.tensor(lists[b], device=k.device)
        at = torch.arange(n0, n0 + N, device=k.device)
        k[own_pages[at // page], at % page] = s["k_new"][b]
        v[own_pages[at // page], at % page] = s["v_new"][b]
    return {"k": k, "v": v, "table": None, "count": None, "ref": None}


def _exact_commit(s):
    page = s["case"]["page"]
    k, v = s["k"].clone(), s["v"].clone()
    table, lens, accept = s["table"].tolist(), s["len"].tolist(), s["accept"].tolist()
    frm, to = [], []
    for b, path in enumerate(s["nodes"].tolist()):
        for i, n in enumerate(path[:accept[b]]):
            a, z = lens[b] + n, lens[b] + 1 + i
            frm.append((table[b][a // page], a % page))
            to.append((table[b][z // page], z % page))
    if frm:
        f, t = torch.tensor(frm, device=k.device), torch.tensor(to, device=k.device)
        k[:, t[:, 0], t[:, 1]] = s["k"][:, f[:, 0], f[:, 1]]
        v[:, t[:, 0], t[:, 1]] = s["v"][:, f[:, 0], f[:, 1]]
    return {"k": k, "v": v, "len": None}


def _exact_fork(s):
    page = s["case"]["page"]
    k, v = s["k"].clone(), s["v"].clone()
    ref, table, lens = s["ref"].tolist(), s["table"].tolist(), s["len"].tolist()
    free = [p for p, r in enumerate(ref) if r == 0]
    for a in s["src"].tolist():
        full, used = divmod(lens[a], page)
        if used:
            p = free.pop(0)
            k[:, p, :used] = s["k"][:, table[a][full], :used]
            v[:, p, :used] = s["v"][:, table[a][full], :used]
    return {"k": k, "v": v, "table": None, "count": None, "ref": None, "len": None}
