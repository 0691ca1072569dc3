"""Scoring given texts against a 4-bit paged cache, and learning from the scores.

    python examples/score_text.py

A small random two-layer decoder shows how the operators go together:

  chunks    each text is read a chunk at a time, as many tokens of each as it has left:
            pages_reserve, kv4_append of the chunk's keys and values, and
            kv4_chunk_attention over all that its sequence holds by then
  scores    token_logprobs of the chunk's logits: the log probability of each next
            token, the entropy, the likeliest alternatives
  gradient  of a loss on log probabilities and entropies, by the output embedding:
            through token_logprobs as through any torch function
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import top_selection_deepselect_gb300 as ds


class Model:
    """Random weights: an embedding, fused q, k, v and an output projection a layer."""

    def __init__(self, vocab, layers, heads, kv_heads, head_dim, seed, device):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.vocab, self.layers, self.heads, self.kv_heads, self.head_dim = vocab, layers, heads, kv_heads, head_dim
        self.width = heads * head_dim

        def weight(a, b, size=1.0):
            return (torch.randn((a, b), device=device, generator=g) * size * a ** -0.5).bfloat16()

        self.embed = weight(vocab, self.width, vocab ** 0.5)
        self.w_in = [weight(self.width, (heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.w_out = [weight(self.width, self.width) for _ in range(layers)]
        self.head = weight(self.width, vocab)

    def read(self, pool, table, lengths, tokens, seqs, starts):
        """Hidden states of tokens [rows] (int32): rows starts[b] to starts[b + 1] are the newest of sequence seqs[b],
        whose places are reserved."""
        count = (starts[1:] - starts[:-1]).long()
        seq = torch.repeat_interleave(seqs, count).to(torch.int32)
        first = torch.repeat_interleave(lengths[seqs.long()] - starts[1:], count)
        pos = (first + torch.arange(len(tokens), device=tokens.device)).to(torch.int32)
        h, hk, d = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens.long()]
        for layer in range(self.layers):
            norm = torch.nn.functional.rms_norm(x, (self.width,))
            q, k, v = (norm @ self.w_in[layer]).split([h * d, hk * d, hk * d], -1)
            ds.kv4_append(pool[layer], table, seq, pos, k.unflatten(-1, (hk, d)), v.unflatten(-1, (hk, d)))
            out, _ = ds.kv4_chunk_attention(q.unflatten(-1, (h, d)), pool[layer], table, lengths, starts, seqs=seqs)
            x = x + out.flatten(1) @ self.w_out[layer]
        return torch.nn.functional.rms_norm(x, (self.width,))


def score(model, texts, chunk, k=4, scale=1.0, page_size=16):
    """Reads the texts (lists of tokens) in chunks of at most `chunk` tokens each.

    Returns, for the tokens of all texts one after another: hidden states, the token that comes next (-1 after the
    last of a text), and token_logprobs of it: (logprob, entropy, lse, idx, top)."""
    device = model.head.device
    i32 = dict(dtype=torch.int32, device=device)
    n, longest = len(texts), max(len(t) for t in texts)
    wide = -(-longest // page_size)
    pages = sum(-(-len(t) // page_size) for t in texts)
    pool = torch.empty((model.layers, pages, model.kv_heads, page_size, ds.kv4_record_bytes(model.head_dim)),
                       dtype=torch.uint8, device=device)
    table, lengths, refs = torch.full((n, wide), -1, **i32), torch.zeros(n, **i32), torch.zeros(pages, **i32)
    parts = [[] for _ in texts]
    for at in range(0, longest, chunk):
        now = [b for b in range(n) if len(texts[b]) > at]
        new = [texts[b][at:at + chunk] for b in now]
        seqs = torch.tensor(now, **i32)
        starts = torch.tensor([sum(len(t) for t in new[:i]) for i in range(len(new) + 1)], **i32)
        ds.pages_reserve(table, lengths, refs, seqs, starts[1:] - starts[:-1], page_size)
        hidden = model.read(pool, table, lengths, torch.tensor(sum(new, []), **i32), seqs, starts)
        following = torch.tensor([t for b in now for t in (texts[b] + [-1])[at + 1:at + 1 + chunk]], **i32)
        got = (hidden, following) + ds.token_logprobs(hidden @ model.head, following, k, scale)
        sizes = [len(t) for t in new]
        for b, *rows in zip(now, *(x.split(sizes) for x in got)):
            parts[b].append(rows)
    return [torch.cat([rows[i] for part in parts for rows in part]) for i in range(7)]


def gradient(model, hidden, following, advantage, entropy_weight, scale=1.0):
    """Gradient by the output embedding of -mean(advantage logprob + entropy_weight entropy) over the scored tokens."""
    head = model.head.detach().requires_grad_()
    logprob, entropy, _, _, _ = ds.token_logprobs(hidden @ head, following, scale=scale)
    scored = following >= 0
    loss = -(advantage * logprob + entropy_weight * entropy * scored).sum() / scored.sum()
    return torch.autograd.grad(loss, head)[0], loss.detach()


def run(sizes=(70, 1, 33, 150), chunk=48, vocab=3001, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda:0"):
    device = torch.device(device)
    model = Model(vocab, 2, heads, kv_heads, head_dim, seed, device)
    g = torch.Generator()
    g.manual_seed(seed + 1)
    texts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in sizes]
    hidden, following, logprob, entropy, lse, idx, top = score(model, texts, chunk)
    advantage = torch.randn(len(logprob), generator=g).to(device)
    grad, loss = gradient(model, hidden, following, advantage, 0.01)
    return dict(model=model, texts=texts, hidden=hidden, following=following, logprob=logprob, entropy=entropy, lse=lse,
                idx=idx, top=top, advantage=advantage, grad=grad, loss=loss)


def main():
    r = run()
    at = 0
    for text in r["texts"]:
        rows = slice(at, at + len(text))
        at += len(text)
        print("%4d tokens: log probability %9.2f, mean entropy %.3f"
              % (len(text), r["logprob"][rows].sum(), r["entropy"][rows].mean()))
    print("likeliest after the first token:", r["idx"][0].tolist(), [round(x, 2) for x in r["top"][0].tolist()])
    print("gradient by the output embedding: norm %.4f" % r["grad"].float().norm())


if __name__ == "__main__":
    main()
