"""Cases of the operators that make a long cache cheap to read: a paged cache held
in 4 bits with the attention over it, and attention over the pages that a cheap
score selects.

Each case has a plain form in elementary torch operations (32-bit arithmetic,
one rounding at the end) and, with `own` set, the calls a user makes of the
package.  `exact` restates each operator in 64 bits from its definition.

  The 4-bit cache.  32 channels of one token and head share a scale
  s = (1 + m / 8) 2^(e - 19), kept as the byte 8 e + m: a seventh of their largest
  magnitude, to the nearest such number.  A number x is kept as the code
  clamp(rint(x / s), -8, 7) + 8 and stands for (code - 8) s, which bfloat16 and
  float16 hold exactly.  The bytes of one page and head are blocks of
  T = min(page, 128) tokens, one after the other, each
      keys' codes    [T / 8][C / 32][8 tokens][16 bytes]
      values' codes  [T / 8][C][4 bytes: 8 tokens]
      keys' scales   [C / 32][T], values' scales [C / 32][T]
  for C channels (head_dim rounded up to 32).  The codes 0 .. 7 of a 32-bit word
  lie at its bits 0, 16, 4, 20, 8, 24, 12, 28.

  attention4  out[b, n, h] = softmax_j(scale * q[b, n, h] . k_j) v_j over the
              positions j that node n of request b sees (the committed ones, its
              ancestors and itself; with a window only those less than `window`
              tokens back along its path, or the first `sinks`), k and v the
              numbers that the 4-bit cache stands for.
  append4     new keys and values written to the 4-bit cache and read back.
  commit4     accepted paths moved behind their roots in every layer, and the
              positions that the trees took read back.
  sparse      one step of attention over selected pages: the bounds (smallest
              and largest key of each channel) of the pages written since `start`,
              the score of every page for a request and key head, max over the
              rows of sum_d max(q_d lo_d, q_d hi_d), the `keep` pages with
              the highest scores (the first and the last always, ties to the
              earlier one) in their order, and attention over those alone.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BITS = (0, 16, 4, 20, 8, 24, 12, 28)  # of the codes of a word


def listed():
    """Head shapes: 32 query heads on 8 key heads of 128 or of 64, the attention
    shapes of the model families whose vocabularies the benchmark uses; K = 8
    drafts (9 rows with the root) as its workloads have."""
    return [
        # one sequence, one token, a short context: the call's latency
        dict(name="token4_b1", op="attention4", B=1, N=1, hq=32, hkv=8, D=128, page=16, ctx=1000, ragged=False,
             chain=True, window=0, sinks=0, dtype="bf16"),
        # a batch drafting one token each from its 4-bit caches
        dict(name="token4_b64", op="attention4", B=64, N=1, hq=32, hkv=8, D=128, page=16, ctx=8192, ragged=True,
             chain=True, window=0, sinks=0, dtype="bf16"),
        # a batch verifying 8 linear drafts each, small heads
        dict(name="chain4_b32", op="attention4", B=32, N=9, hq=32, hkv=8, D=64, page=32, ctx=4096, ragged=True,
             chain=True, window=0, sinks=0, dtype="f16"),
        # one long sequence with a tree of 16: the axis of keys split over the GPU
        dict(name="tree4_long", op="attention4", B=1, N=16, hq=32, hkv=8, D=128, page=128, ctx=131071, ragged=False,
             chain=False, window=0, sinks=0, dtype="bf16"),
        # one layer's new keys and values of a step of a few requests
        dict(name="append4_step", op="append4", B=8, N=9, layers=1, hkv=8, D=128, page=16, ctx=2000, dtype="bf16"),
        # prompts entering the cache
        dict(name="append4_prompt", op="append4", B=16, N=2047, layers=1, hkv=8, D=128, page=64, ctx=500,
             dtype="bf16"),
        # accepted paths of a few small trees
        dict(name="commit4_b4", op="commit4", B=4, N=8, layers=36, hkv=8, D=128, page=16, ctx=100, dtype="bf16"),
        # accepted paths of a batch of larger trees
        dict(name="commit4_b64", op="commit4", B=64, N=32, layers=36, hkv=8, D=128, page=32, ctx=60, dtype="f16"),
        # the first step after a prompt: all of its pages summarised
        dict(name="sparse_first", op="sparse", B=1, N=1, hq=32, hkv=8, D=128, page=16, ctx=32768, ragged=False,
             whole=True, keep=64, four=False, dtype="bf16"),
        # a few requests with long contexts, 4096 tokens read of each
        dict(name="sparse_long", op="sparse", B=4, N=1, hq=32, hkv=8, D=128, page=32, ctx=131071, ragged=False,
             whole=False, keep=128, four=False, dtype="bf16"),
        # a serving batch, four drafts each
        dict(name="sparse_b64", op="sparse", B=64, N=5, hq=32, hkv=8, D=64, page=16, ctx=8192, ragged=True,
             whole=False, keep=48, four=False, dtype="f16"),
        # selected pages of a 4-bit cache
        dict(name="sparse4_b32", op="sparse", B=32, N=1, hq=32, hkv=8, D=128, page=16, ctx=16384, ragged=True,
             whole=False, keep=64, four=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention4", "attention4", "attention4", "sparse", "sparse", "sparse", "append4", "commit4"])
    hkv, group, D = rng.choice([(8, 4, 128), (8, 8, 64), (8, 4, 64), (4, 7, 128), (1, 8, 128), (16, 1, 96),
                                (2, 16, 64), (8, 5, 80)])
    case = dict(op=op, hkv=hkv, D=D, page=rng.choice([8, 16, 32, 64, 128, 256]),
                dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op == "attention4":
        N, B = _log(rng, 1, 64), _log(rng, 1, 256)
        top = min(131072, (64 * 8192 * 8 * 128) // (B * hkv * D), (16 * 131072 * 32) // (B * hkv * group * N))
        window = _log(rng, 1, 8192) if rng.random() < 0.3 else 0
        case.update(B=B, N=N, hq=hkv * group, ctx=_log(rng, 1, max(1, top)), ragged=rng.random() < 0.7,
                    chain=rng.random() < 0.4, window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0)
    elif op == "sparse":
        N, B = _log(rng, 1, 16), _log(rng, 1, 128)
        ctx = _log(rng, 1, max(1, min(131072, (4 * 131072 * 8 * 128) // (2 * B * hkv * D))))
        case.update(B=B, N=N, hq=hkv * group, ctx=ctx, ragged=rng.random() < 0.7, whole=rng.random() < 0.2,
                    keep=_log(rng, 2, max(2, min(4096 // case["page"], (64 * 1024 * 8 * 64) // (B * hkv * D * case["page"])))),
                    four=rng.random() < 0.4)
    elif op == "append4":
        B = _log(rng, 1, 128)
        case.update(B=B, N=_log(rng, 1, max(1, 32768 // B)), layers=1, ctx=_log(rng, 1, 1000))
    else:
        B = _log(rng, 1, 64)
        case.update(B=B, N=_log(rng, 2, max(2, min(64, 2048 // B))), layers=_log(rng, 1, 36), ctx=_log(rng, 1, 100))
    return case


# ------------------------------------------------------------------ the 4-bit format

def _channels(D):
    return (D + 31) // 32 * 32


def page_bytes(page, D):
    return page * _channels(D) * 17 // 16


def _quantise(x):
    """Codes (0 .. 15) and scale bytes of x [..., C], C a multiple of 32."""
    g = x.float().unflatten(-1, (-1, 32))
    # (a quotient next to the middle between two scales is in the balance: 64 bits)
    bits = (g.abs().amax(-1).double() / 7.0).float().view(torch.int32)
    byte = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (108 << 3)
    byte = byte.clamp(0, 255)
    s = ((byte + (108 << 3)) << 20).view(torch.float32)
    code = torch.round(g / s.unsqueeze(-1)).clamp(-8, 7) + 8
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def _scale(byte):
    return ((byte.int() + (108 << 3)) << 20).view(torch.float32)


def _values(code, byte):
    g = (code.float() - 8.0).unflatten(-1, (-1, 32))
    return (g * _scale(byte).unsqueeze(-1)).flatten(-2)


def _words(code):
    """[..., 8] codes as 4 bytes."""
    return code[..., [0, 4, 1, 5]] | (code[..., [2, 6, 3, 7]] << 4)


def _codes(byte):
    """4 bytes as [..., 8] codes."""
    lo, hi = byte & 15, byte >> 4
    return torch.stack((lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]),
                       -1)


def _pack(kc, ks, vc, vs):
    """Bytes of pages from codes [..., page, C] and scale bytes [..., page, C / 32]."""
    page, C = kc.shape[-2:]
    T = min(page, 128)
    parts = []
    k = kc.unflatten(-2, (page // T, T // 8, 8)).unflatten(-1, (C // 32, 4, 8))   # [.., r, T/8, 8, C/32, 4, 8]
    parts.append(_words(k).transpose(-4, -3).flatten(-5))                          # [.., r, T/8, C/32, 8, 4, 4]
    v = vc.unflatten(-2, (page // T, T // 8, 8)).transpose(-1, -2)                 # [.., r, T/8, C, 8]
    parts.append(_words(v).flatten(-3))
    for s in (ks, vs):
        parts.append(s.unflatten(-2, (page // T, T)).transpose(-1, -2).flatten(-2))
    return torch.cat(parts, -1).flatten(-2)


def _unpack(data, page, C):
    """kc, ks, vc, vs of pages [..., page_bytes]."""
    T = min(page, 128)
    r = data.unflatten(-1, (page // T, -1))
    n = T * C // 2
    k = _codes(r[..., :n].unflatten(-1, (T // 8, C // 32, 8, 4, 4))).transpose(-4, -3).flatten(-3)   # [.., r, T/8, 8, C]
    v = _codes(r[..., n:2 * n].unflatten(-1, (T // 8, C, 4))).transpose(-1, -2)
    ks, vs = (x.unflatten(-1, (C // 32, T)).transpose(-1, -2) for x in r[..., 2 * n:].chunk(2, -1))
    return k.flatten(-4, -2), ks.flatten(-3, -2), v.flatten(-4, -2), vs.flatten(-3, -2)


# ------------------------------------------------------------------ inputs

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
    """An accepted path in every tree, as tree verification returns it."""
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


def _pool4(g, lead, page, D, dtype, dev, grid):
    """A 4-bit pool [*lead, page_bytes] of normal keys and values, quantised in pieces."""
    C = _channels(D)
    out = torch.empty(lead + (page_bytes(page, D),), dtype=torch.uint8, device=dev)
    flat = out.view(-1, out.shape[-1])
    step = max(1, (1 << 25) // (page * C))
    for i in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - i)
        x = torch.zeros((2, n, page, C), dtype=dtype, device=dev)
        x[..., :D].normal_(generator=g)
        if grid:
            x = (x * 16).round() / 16
        flat[i:i + n] = _pack(*_quantise(x[0]), *_quantise(x[1]))
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c, op, page, dtype = case, case["op"], case["page"], DTYPES[case["dtype"]]
    hkv, D, B, N = c["hkv"], c["D"], c["B"], c["N"]
    if op in ("attention4", "sparse") and not c["ragged"]:
        lens = torch.full((B,), c["ctx"], dtype=torch.int32, device=dev)
    else:  # contexts of between half and all of ctx
        lo = (c["ctx"] + 1) // 2
        lens = (lo + torch.rand((B,), generator=g, device=dev) * (c["ctx"] - lo + 1)).int().clamp(max=c["ctx"])
    P = (c["ctx"] + N + page - 1) // page + 1
    held = ((lens + N + page - 1) // page).int()
    n_held = int(held.sum())
    pages = B * ((c["ctx"] + N + page - 1) // page) + 3  # a pool for every request at its longest
    perm = torch.randperm(pages, generator=g, device=dev).int()
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    table[torch.arange(P, device=dev) < held.view(-1, 1)] = perm[:n_held]
    s = dict(case=dict(case), table=table, len=lens)
    if op == "sparse":
        # Keys and queries are multiples of 1 / 16, so that every order of addition gives the
        # same scores, and the choice of pages does not hang on it.
        if c["four"]:
            s["pool"] = _pool4(g, (pages, hkv), page, D, dtype, dev, True)
        else:
            s["k"] = torch.empty((pages, page, hkv, D), dtype=dtype, device=dev).normal_(generator=g)
            s["k"].mul_(16).round_().div_(16)
            s["v"] = torch.empty((pages, page, hkv, D), dtype=dtype, device=dev).normal_(generator=g)
        qkv = torch.empty((B, N, c["hq"] + 2 * hkv, D), dtype=dtype, device=dev).normal_(generator=g)
        s["q"] = qkv[:, :, :c["hq"]].mul_(32.0).round_().div_(16.0)
        s["start"] = torch.zeros_like(lens) if c["whole"] else (lens - N).clamp(min=0).int()
        # the bounds of earlier steps: pages before `start` have theirs
        bounds = torch.zeros((pages, hkv, 2, D), dtype=dtype, device=dev)
        s["bounds"] = bounds
        _bounds(s, torch.zeros_like(lens), s["start"])
    elif op == "attention4":
        s["pool"] = _pool4(g, (pages, hkv), page, D, dtype, dev, False)
        # the query rows as they leave a fused projection of queries, keys and values
        qkv = torch.empty((B, N, c["hq"] + 2 * hkv, D), dtype=dtype, device=dev).normal_(generator=g)
        s["q"] = qkv[:, :, :c["hq"]].mul_(2.0)
        s["parent"] = _trees(g, B, N, 1.0 if c["chain"] else 0.5, dev)
    else:
        s["pool"] = _pool4(g, (c["layers"], pages, hkv), page, D, dtype, dev, False)
        if op == "append4":
            kv = torch.empty((B, N, 2 * hkv, D), dtype=dtype, device=dev).normal_(generator=g)
            s["k_new"], s["v_new"] = kv[:, :, :hkv], kv[:, :, hkv:]
        else:
            s["nodes"], s["accept"] = _paths(g, _trees(g, B, N, 0.5, dev), dev)
            s["new_len"] = torch.empty_like(lens)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention4": _own_attention4, "append4": _own_append4, "commit4": _own_commit4,
                "sparse": _own_sparse}[op](s)
    return {"attention4": _attention4, "append4": _append4, "commit4": _commit4, "sparse": _sparse}[op](s)


def _own_attention4(s):
    import speculative_decoding_verification_69_gb300 as sv
    c = s["case"]
    out, lse = sv.tree_attention4(s["q"], s["pool"], s["table"], s["len"], c["page"], s["parent"], window=c["window"],
                                  sinks=c["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_append4(s):
    import speculative_decoding_verification_69_gb300 as sv
    c, layer = s["case"], s["pool"][0]
    sv.cache4_append(layer, s["table"], s["len"], s["k_new"], s["v_new"], c["page"])
    k, v = sv.cache4_read(layer, s["table"], s["len"], c["N"], c["page"], c["D"], dtype=s["k_new"].dtype)
    return {"k": k, "v": v}


def _own_commit4(s):
    import speculative_decoding_verification_69_gb300 as sv
    c = s["case"]
    sv.cache4_commit(s["pool"], s["table"], s["len"], s["nodes"], s["accept"], c["page"], c["D"], new_len=s["new_len"])
    k, v = sv.cache4_read(s["pool"], s["table"], s["len"], c["N"], c["page"], c["D"], dtype=DTYPES[c["dtype"]])
    return {"k": k, "v": v, "len": s["new_len"]}


def _own_sparse(s):
    import speculative_decoding_verification_69_gb300 as sv
    c, page = s["case"], s["case"]["page"]
    if c["four"]:
        sv.cache4_bounds(s["pool"], s["bounds"], s["table"], s["len"], page, start=s["start"])
    else:
        sv.cache_bounds(s["k"], s["bounds"], s["table"], s["len"], start=s["start"])
    scores = sv.page_scores(s["q"], s["bounds"], s["table"], s["len"], page)
    table, kept = sv.page_select(scores, s["table"], s["len"], page, c["keep"], extra=c["N"])
    if c["four"]:
        out, lse = sv.tree_attention4(s["q"], s["pool"], table, kept, page, return_lse=True)
    else:
        out, lse = sv.tree_attention(s["q"], s["k"], s["v"], table, kept, return_lse=True)
    return {"bounds": s["bounds"], "scores": scores, "table": table, "kept": kept, "out": out, "lse": lse}


def _softmax_values(z, v):
    """Softmax over the last axis of z [..., rows, L] times v [..., L, D], and the log of its sum."""
    m = z.amax(-1, keepdim=True)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / total, (m + total.log()).squeeze(-1)


def _attention4(s):
    c, q, table, lens, parent = s["case"], s["q"], s["table"], s["len"].long(), s["parent"].long()
    B, N, hq, D = q.shape
    hkv, page, C = c["hkv"], c["page"], _channels(D)
    L = c["ctx"] + N
    pos = torch.arange(L, device=q.device)
    held = table[:, :(L + page - 1) // page].long().clamp(min=0)
    kc, ks, vc, vs = _unpack(s["pool"][held], page, C)                     # [B, pages, hkv, page, C]
    kk = _values(kc, ks).transpose(1, 2).flatten(2, 3)[:, :, :L, :D]       # [B, hkv, L, D]
    vv = _values(vc, vs).transpose(1, 2).flatten(2, 3)[:, :, :L, :D]
    del kc, ks, vc, vs
    # ancestors of each node, itself among them: powers of (I + parent links)
    node = torch.arange(N, device=q.device)
    link = (parent.unsqueeze(-1) == node).float() + torch.eye(N, device=q.device)
    anc = torch.matrix_power(link, 64) > 0 if N > 1 else link > 0
    depth = anc.sum(-1) - 1
    node_of = pos - lens.view(B, 1)                                        # [B, L]
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
    z = torch.matmul(qq, kk.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, hkv, N, hq // hkv, L)
    z = z.masked_fill_(~seen.view(B, 1, N, 1, L), -math.inf).flatten(2, 3)
    o, lse = _softmax_values(z, vv)
    return {"out": o.view(B, hkv, N, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D).to(q.dtype),
            "lse": lse.view(B, hkv, N, hq // hkv).permute(0, 2, 1, 3).reshape(B, N, hq)}


def _region(s, N):
    """The pages and places inside them of the positions [len, len + N)."""
    page = s["case"]["page"]
    pos = s["len"].long().view(-1, 1) + torch.arange(N, device=s["len"].device)
    return torch.gather(s["table"].long(), 1, pos // page), pos % page


def _read4(s, pool, pg, at):
    """Keys and values [..., B, N, hkv, D] at these places, one layer after the other."""
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    C, D = _channels(c["D"]), c["D"]
    k, v = [], []
    some, where = torch.unique(pg, return_inverse=True)
    for layer in pool:
        kc, ks, vc, vs = _unpack(layer[some], c["page"], C)
        k.append(_values(kc[where, :, at], ks[where, :, at])[..., :D].to(dtype))
        v.append(_values(vc[where, :, at], vs[where, :, at])[..., :D].to(dtype))
    return torch.stack(k), torch.stack(v)


def _append4(s):
    c, pool, N = s["case"], s["pool"][0], s["case"]["N"]
    C, D = _channels(c["D"]), c["D"]
    pg, at = _region(s, N)
    some, where = torch.unique(pg, return_inverse=True)
    kc, ks, vc, vs = (x.contiguous() for x in _unpack(pool[some], c["page"], C))
    for new, code, scale in ((s["k_new"], kc, ks), (s["v_new"], vc, vs)):
        x = torch.zeros(new.shape[:-1] + (C,), dtype=new.dtype, device=new.device)
        x[..., :D] = new
        code[where, :, at], scale[where, :, at] = _quantise(x)
    pool[some] = _pack(kc, ks, vc, vs)
    k, v = _read4(s, s["pool"], pg, at)
    return {"k": k[0], "v": v[0]}


def _commit4(s):
    c, N = s["case"], s["case"]["N"]
    C = _channels(c["D"])
    pg, at = _region(s, N)
    some, where = torch.unique(pg, return_inverse=True)
    step = torch.arange(N, device=pg.device)
    real = step < s["accept"].long().view(-1, 1)
    b = torch.arange(pg.shape[0], device=pg.device).view(-1, 1).expand_as(pg)[real]
    frm, to = s["nodes"].long()[real], (1 + step).expand_as(pg)[real]
    for layer in s["pool"]:
        parts = [x.contiguous() for x in _unpack(layer[some], c["page"], C)]
        for x in parts:
            x[where[b, to], :, at[b, to]] = x[where[b, frm], :, at[b, frm]]
        layer[some] = _pack(*parts)
    s["new_len"].copy_(s["len"] + 1 + s["accept"])
    k, v = _read4(s, s["pool"], pg, at)
    return {"k": k, "v": v, "len": s["new_len"]}


def _keys(s, pg):
    """Keys [..., page, hkv, D] of these pages in 32 bits."""
    if not s["case"]["four"]:
        return s["k"][pg].float()
    kc, ks, _, _ = _unpack(s["pool"][pg], s["case"]["page"], _channels(s["case"]["D"]))
    return _values(kc, ks)[..., :s["case"]["D"]].transpose(-2, -3)


def _bounds(s, start, end):
    """Bounds of the pages that hold positions [start, end), over their positions before `end`."""
    page, table = s["case"]["page"], s["table"]
    place = torch.arange(table.shape[1], device=table.device)
    some = (place >= (start // page).view(-1, 1)) & (place * page < end.view(-1, 1)) & (start < end).view(-1, 1)
    b, at = some.nonzero(as_tuple=True)
    used = (end.long()[b] - at * page).clamp(max=page)
    pg = table[b, at].long()
    step = max(1, (1 << 26) // (page * s["bounds"][0, :, 0].numel()))
    t = torch.arange(page, device=table.device)
    for i in range(0, pg.numel(), step):
        k = _keys(s, pg[i:i + step])
        real = (t < used[i:i + step].view(-1, 1)).view(-1, page, 1, 1)
        lo = k.masked_fill(~real, math.inf).amin(1)
        hi = k.masked_fill(~real, -math.inf).amax(1)
        s["bounds"][pg[i:i + step]] = torch.stack((lo, hi), 2).to(s["bounds"].dtype)


def _select(scores, s, keep):
    """The `keep` pages of each request and key head with the highest scores, in order, the pages of
    the drafted tokens behind them, and the tokens that the former hold."""
    page, table, lens, N = s["case"]["page"], s["table"], s["len"].long(), s["case"]["N"]
    B, H, P = scores.shape
    n = (lens + page - 1) // page
    place = torch.arange(P, device=scores.device)
    last = (place == (n - 1).view(B, 1)) | (place == 0)
    rank = scores.masked_fill(last.view(B, 1, P), math.inf)
    rank = torch.where((place < n.view(B, 1)).view(B, 1, P), rank, torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :keep]
    kept = n.clamp(max=keep)
    i = torch.arange(min(keep, P), device=scores.device)
    order = torch.where(i < kept.view(B, 1, 1), order, torch.full_like(order, P)).sort(-1)[0]
    tail = (N + page - 1) // page
    out = torch.full((B, H, keep + tail), -1, dtype=torch.int32, device=scores.device)
    full = torch.cat([table, torch.full((B, tail + 1), -1, dtype=torch.int32, device=table.device)], 1)
    chosen = torch.gather(full.unsqueeze(1).expand(B, H, -1), 2, order)
    out[..., :order.shape[-1]] = torch.where(order < P, chosen, torch.full_like(chosen, -1))
    for t in range(tail):
        nxt = torch.gather(full, 1, (n + t).clamp(max=P).view(B, 1))
        out.scatter_(2, (kept + t).view(B, 1, 1).expand(B, H, 1), nxt.view(B, 1, 1).expand(B, H, 1))
    return out, torch.where(n > keep, (keep - n) * page + lens, lens).int()


def _sparse(s):
    c, q, lens = s["case"], s["q"], s["len"].long()
    B, N, hq, D = q.shape
    hkv, page, G, P = c["hkv"], c["page"], hq // c["hkv"], s["table"].shape[1]
    _bounds(s, s["start"], s["len"])
    n = (lens + page - 1) // page
    rows = q.float().view(B, N, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, D)
    scores = torch.full((B, hkv, P), -math.inf, dtype=torch.float32, device=q.device)
    for b in range(B):
        nb = int(n[b])
        bd = s["bounds"][s["table"][b, :nb].long()].float()                # [pages, hkv, 2, D]
        best = torch.matmul(rows[b].clamp(min=0), bd[:, :, 1].permute(1, 2, 0))
        best += torch.matmul(rows[b].clamp(max=0), bd[:, :, 0].permute(1, 2, 0))
        scores[b, :, :nb] = best.amax(1)
    table, kept = _select(scores, s, c["keep"])
    L = table.shape[2] * page
    pg = table.long().clamp(min=0)
    h = torch.arange(hkv, device=q.device).view(1, hkv, 1)
    if c["four"]:
        kc, ks, vc, vs = _unpack(s["pool"][pg, h], page, _channels(D))
        kk, vv = (_values(*x)[..., :D].flatten(2, 3) for x in ((kc, ks), (vc, vs)))
    else:
        kk, vv = (x.transpose(1, 2)[pg, h].float().flatten(2, 3) for x in (s["k"], s["v"]))
    z = torch.matmul(rows, kk.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, hkv, N, G, L)
    pos = torch.arange(L, device=q.device)
    seen = pos <= (kept.view(B, 1) + torch.arange(N, device=q.device)).unsqueeze(-1)
    z = z.masked_fill_(~seen.view(B, 1, N, 1, L), -math.inf).flatten(2, 3)
    o, lse = _softmax_values(z, vv)
    return {"bounds": s["bounds"], "scores": scores, "table": table, "kept": kept,
            "out": o.view(B, hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D).to(q.dtype),
            "lse": lse.view(B, hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, hq)}


# ------------------------------------------------------------------ what one pass needs

def work(case):
    """The positions and pages of a case are drawn: their expectations."""
    c, D = case, case["D"]
    token4, token = c["hkv"] * _channels(D) * 17 / 16, c["hkv"] * D * 2 * 2  # bytes of one token's key and value
    mean = c["ctx"] if not c.get("ragged", True) else 0.75 * c["ctx"]
    rows = c["B"] * c["N"] * c.get("hq", 0)
    if c["op"] == "attention4":
        keys = mean + c["N"]
        if c["window"]:
            keys = min(keys, c["window"] + c["sinks"] + c["N"])
        return {"bytes": c["B"] * keys * token4 + rows * (D * 4 + 4) + c["B"] * (keys / c["page"] + c["N"] + 1) * 4,
                "flops": 4.0 * rows * D * keys}
    if c["op"] == "append4":  # written and read back
        return {"bytes": 2.0 * c["B"] * c["N"] * (token + token4), "flops": 0}
    if c["op"] == "commit4":  # mean depth of a uniform node of these trees
        depth = [0.0]
        for n in range(1, c["N"]):
            depth.append(1.0 + 0.5 * depth[n - 1] + 0.5 * sum(depth) / n)
        d = sum(depth) / c["N"]
        return {"bytes": c["B"] * c["layers"] * (2.0 * d * token4 + c["N"] * (token + token4)) + 8.0 * c["B"],
                "flops": 0}
    pages = -(-mean // c["page"])
    fresh = mean if c["whole"] else min(mean, c["N"] + c["page"] / 2)
    kept = min(c["keep"], pages)
    one = token4 if c["four"] else token
    return {"bytes": c["B"] * (fresh * one / 2 + fresh / c["page"] * token + pages * (token + 4 * c["hkv"] + 4)
                               + (kept * c["page"] + c["N"]) * one + kept * 4 * c["hkv"]) + rows * (D * 4 + 4),
            "flops": rows * D * (4.0 * pages + 4.0 * (kept * c["page"] + c["N"]))}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention4": _exact_attention4, "append4": _exact_append4, "commit4": _exact_commit4,
            "sparse": _exact_sparse}[case["op"]](s)


def _power(e):
    """2^e for whole e, in 64 bits, exact on every device."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stored(pool, page, D, pg, at, values):
    """The numbers that a 4-bit pool [pages, hkv, bytes] holds at places (pg, at) [L], as [L, hkv, D] in 64 bits,
    each fetched by the position of its byte."""
    C, T = _channels(D), min(page, 128)
    size, base, t = T * C * 17 // 16, at // T, at % T
    d = torch.arange(D, device=pool.device)
    t, base = t.view(-1, 1), (base * size).view(-1, 1)
    if values:
        code = T * C // 2 + (t // 8 * C + d) * 4
        i = t % 8
        scale = T * C + T * (C // 32) + d // 32 * T + t
    else:
        code = ((t // 8 * (C // 32) + d // 32) * 8 + t % 8) * 16 + d % 32 // 8 * 4
        i = d % 8 + 0 * t
        scale = T * C + d // 32 * T + t
    bit = torch.tensor(BITS, device=pool.device)[i]
    head = torch.arange(pool.shape[1], device=pool.device).view(1, -1, 1)

    def take(index):
        return pool[pg.view(-1, 1, 1), head, index.unsqueeze(1)].long()
    c = (take(base + code + bit // 8) >> (bit % 8).unsqueeze(1)) & 15
    b = take(base + scale)
    return (c - 8).double() * ((1.0 + (b % 8).double() / 8.0) * _power(b // 8 - 19))


def _exact_rows(q, kk, vv, seen):
    """Attention of rows [N, hkv, G, D] over keys [L, hkv, D] in 64 bits."""
    z = torch.einsum("nhgd,lhd->nhgl", q, kk) / math.sqrt(q.shape[-1])
    z = torch.where(seen.view(seen.shape[0], 1, 1, -1), z, torch.full_like(z, -math.inf))
    return torch.einsum("nhgl,lhd->nhgd", torch.softmax(z, -1), vv), torch.logsumexp(z, -1)


def _exact_attention4(s):
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
        kk, vv = (_stored(s["pool"], page, D, pg, at % page, v) for v in (False, True))
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
        o, l = _exact_rows(q[b].double().view(N, hkv, G, D), kk, vv, seen.to(q.device)[:, at])
        out[b], lse[b] = o.reshape(N, hq, D), l.view(N, hq)
    return {"out": out, "lse": lse}


def _exact_kept(x):
    """What the 4-bit cache keeps of x [..., D], in 64 bits."""
    D, C = x.shape[-1], _channels(x.shape[-1])
    g = torch.nn.functional.pad(x.double(), (0, C - D)).unflatten(-1, (-1, 32))
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True) / 7.0)             # m in [1/2, 1)
    s = torch.round(m * 16.0) / 16.0 * _power(e)
    s = s.clamp(2.0 ** -19, 1.875 * 2.0 ** 12)
    return (torch.round(g / s).clamp(-8, 7) * s).flatten(-2)[..., :D]


def _exact_append4(s):
    return {"k": _exact_kept(s["k_new"]), "v": _exact_kept(s["v_new"])}


def _exact_commit4(s):
    c, page, N, D = s["case"], s["case"]["page"], s["case"]["N"], s["case"]["D"]
    table, lens, accept = s["table"].tolist(), s["len"].tolist(), s["accept"].tolist()
    pg, at = [], []
    for b, path in enumerate(s["nodes"].tolist()):
        places = list(range(N))
        places[1:1 + accept[b]] = path[:accept[b]]
        pg += [table[b][(lens[b] + p) // page] for p in places]
        at += [(lens[b] + p) % page for p in places]
    pg, at = (torch.tensor(x, device=s["pool"].device) for x in (pg, at))
    k, v = (torch.stack([_stored(layer, page, D, pg, at, vals).view(len(lens), N, -1, D) for layer in s["pool"]])
            for vals in (False, True))
    return {"k": k, "v": v, "len": None}


def _exact_sparse(s):
    """Request by request and head by head."""
    c, q, table = s["case"], s["q"], s["table"]
    B, N, hq, D = q.shape
    hkv, page, G, P = c["hkv"], c["page"], hq // c["hkv"], table.shape[1]
    tail = -(-N // page)
    scores = torch.full((B, hkv, P), -math.inf, dtype=torch.float64, device=q.device)
    out = torch.empty((B, N, hq, D), dtype=torch.float64, device=q.device)
    lse = torch.empty((B, N, hq), dtype=torch.float64, device=q.device)
    picked, kept, bounds = [], [], s["bounds"].double()
    for b, n0 in enumerate(s["len"].tolist()):
        n = -(-n0 // page)
        row, first = table[b].tolist(), int(s["start"][b]) // page
        for i in range(first, n if int(s["start"][b]) < n0 else 0, 1024):
            places = torch.arange(i, min(n, i + 1024), device=q.device)
            pg = table[b].long()[places]
            t = torch.arange(page, device=q.device)
            if c["four"]:
                k = _stored(s["pool"], page, D, pg.repeat_interleave(page), t.repeat(len(pg)), False)
                k = k.view(len(pg), page, hkv, D)
            else:
                k = s["k"][pg].double()
            gone = (places.view(-1, 1) * page + t >= n0).view(-1, page, 1, 1)
            bounds[pg, :, 0] = torch.where(gone, torch.full_like(k, math.inf), k).amin(1)
            bounds[pg, :, 1] = torch.where(gone, torch.full_like(k, -math.inf), k).amax(1)
        rows = q[b].double().view(N, hkv, G, D)
        picks = []
        for h in range(hkv):
            r = rows[:, h].reshape(-1, D)
            for i in range(0, n, 256):
                bd = bounds[table[b, i:min(n, i + 256)].long(), h]
                top = torch.maximum(r.unsqueeze(1) * bd[:, 0], r.unsqueeze(1) * bd[:, 1]).sum(-1)
                scores[b, h, i:i + 256][:bd.shape[0]] = top.amax(0)
            value = scores[b, h, :n].tolist()
            must = {0, n - 1} if n else set()
            rest = sorted((p for p in range(n) if p not in must), key=lambda p: (-value[p], p))
            chosen = sorted((sorted(must) + rest)[:c["keep"]])
            picks.append(chosen)
        m = len(picks[0])
        kept.append(n0 if n <= c["keep"] else n0 - (n - m) * page)
        behind = [row[n + i] if n + i < P else -1 for i in range(tail)]
        picked.append([[row[p] for p in ch] + behind + [-1] * (c["keep"] - m) for ch in picks])
        at = torch.arange(kept[b] + N, device=q.device)
        seen = at <= (kept[b] + torch.arange(N, device=q.device)).view(-1, 1)
        for h in range(hkv):
            pg = torch.tensor(picked[b][h], device=q.device)[at // page]
            if c["four"]:
                kk, vv = (_stored(s["pool"][:, h:h + 1], page, D, pg, at % page, v) for v in (False, True))
            else:
                kk, vv = (x[pg, at % page, h:h + 1].double() for x in (s["k"], s["v"]))
            o, l = _exact_rows(rows[:, h:h + 1], kk, vv, seen)
            out[b, :, h * G:(h + 1) * G], lse[b, :, h * G:(h + 1) * G] = o[:, 0], l[:, 0]
    i32 = dict(dtype=torch.int32, device=q.device)
    return {"bounds": bounds, "scores": scores, "table": torch.tensor(picked, **i32), "kept": torch.tensor(kept, **i32),
            "out": out, "lse": lse}
