"""Speculative decoding of drafted trees on a paged cache, end to end.

A small transformer with random weights is the target, its embedding and head
alone (no attention) the drafter.  One prompt is read into slot 0 in chunks of
up to 64 tokens, forked to the other slots, and every slot continues it, even
slots greedily, odd ones sampled.  A step drafts a tree of nodes per slot, runs
the target on all nodes at once (cache_append, tree_attention in every layer),
verifies the tree (verify_tree) and keeps the accepted path (cache_commit).

    python examples/tree_decode.py [--slots 4] [--steps 24] [--prompt 150]

Prints the tokens emitted per step, and the largest difference between the
logits the steps verified and the ones of the plain model on the finished
sequences.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_69_gb300 as sv  # noqa: E402

PARENT = (-1, 0, 0, 0, 1, 1, 2, 4, 4, 7)  # parent of every node: the root, three guesses, and what follows them


class Model:
    """Attention layers between an embedding and a head; q, k and v are rounded
    to `dtype`, as the cache stores them, all else is float32."""

    def __init__(self, layers=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, vocab=1000, max_len=1024,
                 dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g).cuda()
        self.q_heads, self.kv_heads, self.head_dim, self.dtype = q_heads, kv_heads, head_dim, dtype
        self.layers, self.vocab = layers, vocab
        self.embed, self.place = rand(vocab, hidden), rand(max_len, hidden) * 0.1
        self.head = rand(hidden, vocab) * (4.0 / hidden ** 0.5)
        cols = (q_heads + 2 * kv_heads) * head_dim
        self.w_qkv = [rand(hidden, cols) / hidden ** 0.5 for _ in range(layers)]
        self.w_out = [rand(q_heads * head_dim, hidden) / (q_heads * head_dim) ** 0.5 for _ in range(layers)]

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def forward(self, tokens, places, attend):
        """Logits [B, N, vocab]; attend(layer, q, k, v) -> [B, N, q_heads, head_dim]."""
        x = self.embed[tokens.long()] + self.place[places.long()]
        for layer in range(self.layers):
            qkv = (self.norm(x) @ self.w_qkv[layer]).to(self.dtype).unflatten(-1, (-1, self.head_dim))
            q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), dim=2)
            x = x + attend(layer, q, k, v).float().flatten(2) @ self.w_out[layer]
        return self.norm(x) @ self.head

    def draft(self, tokens):
        return self.norm(self.embed[tokens.long()]) @ self.head

    def plain(self, tokens):
        """The logits of a whole sequence [1, n], with plain causal attention."""
        n = tokens.shape[1]
        mask = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()

        def attend(layer, q, k, v):
            G = self.q_heads // self.kv_heads
            k, v = (t.double().repeat_interleave(G, 2) for t in (k, v))
            s = torch.einsum("bnhd,bmhd->bhnm", q.double(), k) / self.head_dim ** 0.5
            return torch.einsum("bhnm,bmhd->bnhd", s.masked_fill(~mask, -torch.inf).softmax(-1), v)
        return self.forward(tokens, torch.arange(n, device="cuda")[None], attend)


def prefill(model, cache, prompt, chunk=64):
    """The prompt into slot 0.  The chunks are chains: every token sees those before it."""
    want = torch.zeros_like(cache.cache_len)
    want[0] = prompt.numel()
    sv.cache_resize(cache.page_table, cache.page_count, cache.page_ref, want, cache.page_size,
                    dev_status=cache.status)
    table, length = cache.page_table[:1], cache.cache_len[:1]
    for at in range(0, prompt.numel(), chunk):
        part = prompt[None, at:at + chunk]
        n = part.shape[1]

        def attend(layer, q, k, v):
            sv.cache_append(cache.k[layer], cache.v[layer], table, length, k, v, dev_status=cache.status)
            return sv.tree_attention(q, cache.k[layer], cache.v[layer], table, length, dev_status=cache.status)
        model.forward(part, torch.arange(at, at + n, device="cuda")[None], attend)
        # a chain whose every token is kept: the root and n - 1 nodes after it
        sv.cache_commit(cache.k, cache.v, table, length, None, torch.full_like(length, n - 1), nodes=n,
                        dev_status=cache.status)


def draft_tree(model, root, temperature, g):
    """Tokens [B, N] of the tree's nodes, and the drafter's logits after nodes
    0 .. N - 2.  Greedy slots try a node's likeliest successors, sampled ones
    draw each child independently from the node's distribution."""
    B, N = root.numel(), len(PARENT)
    tokens, logits = [root], [model.draft(root)]
    for n in range(1, N):
        z = logits[PARENT[n]]
        best = z.topk(3).indices[:, PARENT[1:n].count(PARENT[n])]
        p = (z / temperature.clamp_min(1e-3)[:, None]).softmax(-1)
        drawn = torch.multinomial(p, 1, generator=g)[:, 0]
        tokens.append(torch.where(temperature > 0, drawn, best).int())
        logits.append(model.draft(tokens[-1]))
    return torch.stack(tokens, 1), torch.stack(logits[:-1], 1)


def run(slots=4, steps=24, prompt_len=150, page_size=16, seed=0, model=None):
    """Decodes, and returns (sequences, tokens emitted per step and slot, the
    largest difference from the plain model's logits)."""
    model = model or Model(seed=seed)
    N = len(PARENT)
    pages = -(-(prompt_len + steps * N + N) // page_size) + 1
    cache = sv.PagedCache(model.layers, slots * pages, page_size, model.kv_heads, model.head_dim, slots, pages,
                          dtype=model.dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    prompt = torch.randint(model.vocab, (prompt_len,), generator=g, device="cuda", dtype=torch.int32)
    prefill(model, cache, prompt[:-1])  # the last token is the first root
    i32 = dict(dtype=torch.int32, device="cuda")
    if slots > 1:
        cache.fork(torch.zeros(slots - 1, **i32), torch.arange(1, slots, **i32))

    parent = torch.tensor(PARENT, **i32).repeat(slots, 1)
    depth = [0] * N
    for n in range(1, N):
        depth[n] = depth[PARENT[n]] + 1
    depth = torch.tensor(depth, device="cuda")
    temperature = torch.where(torch.arange(slots, device="cuda") % 2 == 0, 0.0, 0.8)
    root = prompt[-1:].repeat(slots)
    sequences = [prompt.tolist() for _ in range(slots)]
    verified = [[] for _ in range(slots)]  # the target's logits along each sequence
    for step in range(steps):
        tokens, draft = draft_tree(model, root, temperature, g)
        cache.reserve(N)

        def attend(layer, q, k, v):
            cache.append(layer, k, v)
            return cache.attention(layer, q, parent)
        target = model.forward(tokens, cache.cache_len[:, None] + depth, attend)
        out, nodes, accepted = sv.verify_tree(target, draft.contiguous(), parent, tokens, temperature, seed + step)
        cache.commit(nodes, accepted)
        cache.trim()
        last = accepted.long()[:, None]
        root = out.gather(1, last)[:, 0]
        for b, (n, emitted, path) in enumerate(zip(accepted.tolist(), out.tolist(), nodes.tolist())):
            verified[b] += [target[b, i] for i in [0] + path[:n]]
            sequences[b] += emitted[:n + 1]
    if int(cache.status):
        raise sv.SpecVerifyError("device status %d" % int(cache.status))
    worst = 0.0
    for b in range(slots):
        assert int(cache.cache_len[b]) == len(sequences[b]) - 1  # the last token is the next root
        plain = model.plain(torch.tensor(sequences[b], **i32)[None])[0, prompt_len - 1:-1]
        worst = max(worst, float((plain - torch.stack(verified[b])).abs().max()))
    emitted = sum(len(s) - prompt_len for s in sequences) / (steps * slots)
    return sequences, emitted, worst


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--slots", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--prompt", type=int, default=150)
    a = ap.parse_args()
    _, emitted, worst = run(a.slots, a.steps, a.prompt)
    print("%d slots, %d steps: %.2f tokens a step; logits within %.4f of the plain model's"
          % (a.slots, a.steps, emitted, worst))


if __name__ == "__main__":
    main()
