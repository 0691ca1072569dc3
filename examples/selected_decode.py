"""Decoding with attention over selected tokens of a 4-bit paged cache.

    python examples/selected_decode.py

A small random two-layer decoder without vocabulary shows how the operators go
together in a serving loop:

  prompt    pages_reserve gives the sequences their pages, kv4_append fills them
  step      pages_reserve, kv4_append of the new token, index scores of every
            cached token, topk of the scores, kv4_attention over the chosen tokens
  drafts    several tokens at once, attention over everything, causal among them
  branch    pages_fork: children share the parent's full pages
  end       pages_free, then pages_compact puts the live pages first

The page table is shared by the layers: one pool [layers, pages, heads, page
size, record bytes], and the page functions move all layers of a page.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import top_selection_deepselect_gb300 as ds


class Cache:
    """A pool of pages, who holds which, and the index keys that selection goes by."""

    def __init__(self, layers, n_pages, page_size, kv_heads, head_dim, max_seqs, max_pages, index_dim,
                 device):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size, self.head_dim = page_size, head_dim
        self.pool = torch.empty((layers, n_pages, kv_heads, page_size, ds.kv4_record_bytes(head_dim)),
                                dtype=torch.uint8, device=device)
        self.table = torch.full((max_seqs, max_pages), -1, **i32)
        self.lengths = torch.zeros(max_seqs, **i32)
        self.refs = torch.zeros(n_pages, **i32)
        # index keys by position; a program with long contexts would page these too
        self.index = torch.zeros((layers, max_seqs, max_pages * page_size, index_dim),
                                 dtype=torch.bfloat16, device=device)

    def reserve(self, seqs, tokens):
        status = ds.pages_reserve(self.table, self.lengths, self.refs, seqs, tokens, self.page_size)
        short = int(status[0])          # a serving loop would read this a step later
        if short:
            raise RuntimeError("%d pages short" % short)

    def fork(self, src, dst):
        status = ds.pages_fork(self.pool, self.table, self.lengths, self.refs, src, dst)
        if int(status[0]):
            raise RuntimeError("%d pages short" % int(status[0]))
        self.index[:, dst.long()] = self.index[:, src.long()]

    def free(self, seqs):
        ds.pages_free(self.table, self.lengths, self.refs, seqs, self.page_size)

    def compact(self):
        return ds.pages_compact(self.pool, self.table, self.refs)


class Decoder:
    """Random weights: fused q, k, v and index projections and an output projection a layer."""

    def __init__(self, layers, heads, kv_heads, head_dim, index_dim, seed, device):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.layers, self.heads, self.kv_heads, self.head_dim = layers, heads, kv_heads, head_dim
        self.index_dim, self.width = index_dim, heads * head_dim
        out = (heads + 2 * kv_heads) * head_dim + 2 * index_dim

        def weight(a, b):
            return (torch.randn((a, b), device=device, generator=g) * a ** -0.5).bfloat16()

        self.w_in = [weight(self.width, out) for _ in range(layers)]
        self.w_out = [weight(self.width, self.width) for _ in range(layers)]

    def step(self, x, cache, seqs, k):
        """x: [batch, queries, width], the newest tokens of seqs (int32), whose places are reserved.

        Attends the k tokens of the highest index scores (one query), or every
        token (k = 0).  Returns the hidden states, like x."""
        batch, queries, _ = x.shape
        at = cache.lengths[seqs.long()]
        pos = at[:, None] - queries + torch.arange(queries, dtype=torch.int32, device=x.device)
        flat_seq, flat_pos = seqs.repeat_interleave(queries), pos.flatten().to(torch.int32)
        h, hk, d, di = self.heads, self.kv_heads, self.head_dim, self.index_dim
        for layer in range(self.layers):
            norm = torch.nn.functional.rms_norm(x, (self.width,))
            q, key, value, qi, ki = (norm @ self.w_in[layer]).split([h * d, hk * d, hk * d, di, di], -1)
            pool = cache.pool[layer]
            ds.kv4_append(pool, cache.table, flat_seq, flat_pos, key.reshape(-1, hk, d),
                          value.reshape(-1, hk, d))
            cache.index[layer, flat_seq.long(), flat_pos.long()] = ki.reshape(-1, di)
            indices = None
            if k:
                scores = torch.bmm(cache.index[layer, seqs.long()], qi.reshape(batch, di, 1))[..., 0]
                indices = ds.topk(scores.contiguous(), k, 128, 128, row_len=at)[0].view(batch, 1, k)
            out, _ = ds.kv4_attention(q.reshape(batch, queries, h, d), pool, cache.table, cache.lengths,
                                      indices=indices, seqs=seqs)
            x = x + out.reshape(batch, queries, -1) @ self.w_out[layer]
        return x


def run(prompts=(70, 33, 5, 128), steps=4, k=64, layers=2, heads=8, kv_heads=2, head_dim=128,
        page_size=16, seed=0, device="cuda:0"):
    """Prompts of these lengths, a few selected steps, drafts, a fork, an end; returns what happened."""
    device = torch.device(device)
    g = torch.Generator(device=device)
    g.manual_seed(seed + 1)
    n = len(prompts)
    cache = Cache(layers, 96, page_size, kv_heads, head_dim, 2 * n, 16, 32, device)
    model = Decoder(layers, heads, kv_heads, head_dim, 32, seed, device)
    i32 = dict(dtype=torch.int32, device=device)
    seqs = torch.arange(n, **i32)

    def tokens(queries):
        return torch.randn((n, queries, model.width), device=device, generator=g).bfloat16()

    # prompts, one sequence at a time, in one step over all of its tokens
    for s, length in enumerate(prompts):
        one = seqs[s:s + 1]
        cache.reserve(one, torch.tensor([length], **i32))
        model.step(tokens(length)[:1], cache, one, 0)

    one_each = torch.ones(n, **i32)
    for _ in range(steps):
        cache.reserve(seqs, one_each)
        hidden = model.step(tokens(1), cache, seqs, k)

    # three drafted tokens a sequence, checked at once
    cache.reserve(seqs, 3 * one_each)
    drafts = model.step(tokens(3), cache, seqs, 0)

    # two children of the longest sequence; the same token keeps all three alike
    best = int(torch.argmax(cache.lengths))
    family = torch.tensor([best, n, n + 1], **i32)
    cache.fork(family[:1].repeat(2), family[1:])
    x = tokens(1)[:1].repeat(3, 1, 1)
    cache.reserve(family, torch.ones(3, **i32))
    branched = model.step(x, cache, family, k)

    # everything but the children ends; their pages move to the front
    before = ds.kv4_attention(x.view(3, 1, heads, head_dim), cache.pool[0], cache.table,
                              cache.lengths, seqs=family)[0]
    cache.free(seqs)
    _, status = cache.compact()
    after = ds.kv4_attention(x.view(3, 1, heads, head_dim)[1:], cache.pool[0], cache.table,
                             cache.lengths, seqs=family[1:])[0]
    live, moved = status.tolist()
    return dict(hidden=hidden, drafts=drafts, branched=branched, before=before, after=after, live=live,
                moved=moved, lengths=cache.lengths.tolist(), refs=cache.refs.tolist(),
                table=cache.table.tolist(), family=family.tolist())


def main():
    r = run()
    print("selected steps: hidden states", tuple(r["hidden"].shape), "drafts", tuple(r["drafts"].shape))
    print("children of sequence %d alike: %s" % (r["family"][0], bool((r["branched"][1:] == r["branched"][0]).all())))
    print("after the end: %d live pages, %d moved to the front, attention unchanged: %s"
          % (r["live"], r["moved"], bool((r["before"][1:] == r["after"]).all())))


if __name__ == "__main__":
    main()
