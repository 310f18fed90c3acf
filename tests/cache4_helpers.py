"""The 4-bit cache of include/spec_cache.h in plain 64-bit steps, byte by byte from its layout, for the tests."""
import math

import torch

import cache_helpers as ch

BITS = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28])


def channels(D):
    return -(-D // 32) * 32


def page_bytes(page, D):
    return page * channels(D) * 17 // 16


def kept(x):
    """Codes and scale bytes of x [..., D]: int64 [..., C] and [..., C / 32]."""
    D, C = x.shape[-1], channels(x.shape[-1])
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=math.inf, neginf=-math.inf)
    g = torch.nn.functional.pad(x, (0, C - D)).unflatten(-1, (-1, 32))
    top = g.abs().amax(-1) / 7.0
    m, e = torch.frexp(torch.nan_to_num(top, posinf=2.0 ** 40))     # top = m 2^e, m in [1/2, 1)
    r = torch.round(m * 16.0).long()                                # 8 .. 16
    e = e.long() + (r == 16)
    r = torch.where(r == 16, torch.full_like(r, 8), r)
    byte = (8 * (e - 1 + 19) + (r - 8)).clamp(0, 255)
    byte = torch.where(top == 0, torch.zeros_like(byte), byte)
    s = scale(byte).unsqueeze(-1)
    code = torch.round((g / s).clamp(-100.0, 100.0)).clamp(-8, 7).long() + 8
    return code.flatten(-2), byte


def scale(byte):
    power = ((byte // 8 - 19 + 1023) << 52).view(torch.float64)      # 2^(e - 19)
    return (1.0 + (byte % 8).double() / 8.0) * power


def values(x):
    """What the cache keeps of x, float64."""
    code, byte = kept(x)
    return ((code - 8).double().unflatten(-1, (-1, 32)) * scale(byte).unsqueeze(-1)).flatten(-2)[..., :x.shape[-1]]


def places(page, D, kind):
    """Byte offsets and shifts of the codes [page, D] and offsets of the scales [page, C / 32] in a page and head."""
    C, T = channels(D), min(page, 128)
    tok, d, g = torch.arange(page).view(-1, 1), torch.arange(D), torch.arange(C // 32)
    base, t = tok // T * (T * C * 17 // 16), tok % T
    if kind == "k":
        word, i = base + ((t // 8 * (C // 32) + d // 32) * 8 + t % 8) * 16 + d % 32 // 8 * 4, (d % 8).expand(page, D)
        sc = base + T * C + g * T + t
    else:
        word, i = base + T * C // 2 + (t // 8 * C + d) * 4, (t % 8).expand(page, D)
        sc = base + T * C + T * (C // 32) + g * T + t
    bit = BITS[i]
    return word + bit // 8, bit % 8, sc


def decode(pool, page, D):
    """The numbers of a pool [..., num_pages, heads, bytes]: k and v [..., num_pages, page, heads, D] float64 on its
    device."""
    out = []
    for kind in "kv":
        at, shift, sc = (x.to(pool.device) for x in places(page, D, kind))
        code = (pool[..., at].long() >> shift) & 15                  # [..., heads, page, D]
        s = scale(pool[..., sc].long())                              # [..., heads, page, C / 32]
        g = torch.arange(D, device=pool.device) // 32
        out.append(((code - 8).double() * s[..., g]).transpose(-2, -3))
    return out


def make_pool(g, pages, heads, page, D, layers=None, device="cuda"):
    """Random bytes, with scales from 2^-4 to 2^1 (byte 120 to 160)."""
    lead = () if layers is None else (layers,)
    x = torch.randint(0, 256, lead + (pages, heads, page_bytes(page, D)), generator=g, device=device, dtype=torch.uint8)
    for kind in "kv":
        sc = places(page, D, kind)[2].to(device)
        x[..., sc] = torch.randint(120, 160, x.shape[:-1] + tuple(sc.shape), generator=g, device=device,
                                   dtype=torch.uint8)
    return x


def ref_attention(q, pool, page, table, lens, parent, **kw):
    """ch.ref_attention over a 4-bit pool; table [B, P] or [B, heads, P]."""
    k, v = decode(pool, page, q.shape[-1])
    return ref_lists(q, k, v, table, lens, parent, **kw)


def ref_lists(q, k, v, table, lens, parent, **kw):
    if table.dim() == 2:
        return ch.ref_attention(q, k, v, table, lens, parent, **kw)
    hkv, G = k.shape[2], q.shape[2] // k.shape[2]
    each = [ch.ref_attention(q[:, :, h * G:(h + 1) * G], k[:, :, h:h + 1], v[:, :, h:h + 1], table[:, h], lens, parent,
                             **dict(kw, scale=kw.get("scale") or 1.0 / math.sqrt(q.shape[-1]))) for h in range(hkv)]
    return tuple(torch.cat(x, 2) for x in zip(*each))
