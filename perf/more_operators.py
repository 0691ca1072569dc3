"""Cases for reading and scoring given text: attention of chunks of new tokens over the paged 4-bit cache, and log
probabilities of given tokens with entropy and the likeliest alternatives, with their gradient.

Cache records (see include/ds_kv4.h): the key's codes, the value's codes (two codes a byte), the key's scales and the
value's scales (fp16, one for each 32 channels), filled up to a multiple of 16 bytes.  A code u of 4 bits stands for
(u - 8) * scale.  Within a stretch of up to 128 channels the key's 32-bit words, eight channels each, are stored with
word 4 i + t of the stretch at place n t + i (n: groups of the stretch), and the value's 16-bit pieces, four channels
each, with piece 8 i + g at place n g + i.  The pool is [pages, heads, page size, record].
"""
import math

import torch

own = False

DEV = "cuda:0"
GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAIR_CAP = 2.2e12     # operations of one attention case
SCORE_CAP = 1.75e10   # bytes of its scores in 32 bits
LOGIT_CAP = 5.3e8     # bytes of one case's logits


def ds():
    import top_selection_deepselect_gb300 as package
    return package


def listed():
    return [
        # the first chunk of one short prompt, nothing cached before it: latency
        dict(name="chunk one short prompt", op="chunk", batch=1, new=33, before=0, ragged=False, heads=4, kv_heads=1,
             dim=64, page=16, dtype="bf16"),
        # prompts of odd and unequal lengths read together, each after what its sequence holds already
        dict(name="chunk ragged prompts", op="chunk", batch=9, new=701, before=3001, ragged=True, heads=24, kv_heads=8,
             dim=64, page=48, dtype="fp16"),
        # the last chunk of a long prompt, at the long context of the index-score workload (32768)
        dict(name="chunk 2048 of 32768", op="chunk", batch=1, new=2048, before=30720, ragged=False, heads=64,
             kv_heads=8, dim=128, page=64, dtype="bf16"),
        # short questions about two long cached documents: few rows, a long axis
        dict(name="chunk 129 after 130943", op="chunk", batch=2, new=129, before=130943, ragged=False, heads=64,
             kv_heads=8, dim=128, page=64, dtype="bf16"),
        # wide heads
        dict(name="chunk wide heads", op="chunk", batch=5, new=513, before=4000, ragged=True, heads=16, kv_heads=2,
             dim=256, page=32, dtype="fp16"),
        # one decoded token of one sequence with a small vocabulary (the 1 x 4096 workload): latency
        dict(name="score one row", op="score", rows=1, vocab=4096, k=5, scale=1.0, dtype="fp32"),
        # a sampled batch over the vocabulary of the sampling workload (256 x 128000), alternatives as servers give them
        dict(name="score 256x128000", op="score", rows=256, vocab=128000, k=20, scale=1.0, dtype="bf16"),
        # the logits of a prompt's chunk, at a temperature
        dict(name="score 2048x128000", op="score", rows=2048, vocab=128000, k=1, scale=1.25, dtype="bf16"),
        # an odd vocabulary, rows that start anywhere, no alternatives
        dict(name="score odd", op="score", rows=513, vocab=50257, k=0, scale=1.0, dtype="fp16"),
        # a few rows of a policy-gradient step
        dict(name="gradient small", op="gradient", rows=4, vocab=32001, k=0, scale=1.0, dtype="bf16"),
        # a policy-gradient step with an entropy term
        dict(name="gradient 1024x128000", op="gradient", rows=1024, vocab=128000, k=0, scale=1.0, dtype="bf16"),
        # distillation on a teacher's likeliest tokens, logits in 32 bits, an odd vocabulary
        dict(name="gradient of alternatives", op="gradient", rows=257, vocab=50257, k=16, scale=0.8, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "score", "gradient"])
    if op == "chunk":
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        heads = kv_heads * group
        new = _log(rng, 2, 4096)
        # no more pairs, and no larger scores, than the largest listed case
        most = min(PAIR_CAP / (4.0 * heads * dim), SCORE_CAP / (4.0 * heads)) / new
        before = _log(rng, 1, max(1, int(min(131072, most)) - new)) if rng.random() < 0.85 else 0
        batch = _log(rng, 1, max(1, min(64, int(most / (before + new)))))
        return dict(op=op, batch=batch, new=new, before=before, ragged=rng.random() < 0.7, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 48, 64, 128]),
                    dtype=rng.choice(["bf16", "fp16"]))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    size = 4 if dtype == "fp32" else 2
    vocab = _log(rng, 1000, 262144)
    rows = _log(rng, 1, min(4096, int(LOGIT_CAP / size / vocab / (1 if op == "score" else 2))))
    return dict(op=op, rows=rows, vocab=vocab, k=rng.choice([0, 1, 5, 8, 20, 32]),
                scale=rng.choice([1.0, 1.0, 0.8, 1.25]), dtype=dtype)


# ---- sizes that follow from a case ----------------------------------------------------------------------------
def _data(dim):
    return dim + 2 * (dim // GROUP) * 2


def _record(dim):
    return (_data(dim) + 15) // 16 * 16


def _spread_sizes(n, top, ragged, least, turn):
    """Sizes of n sequences: all `top`, or spread over (top / 16, top] by the golden section, the last one `top`."""
    if not ragged:
        return [top] * n
    got = [max(least, int(top * (1 / 16 + 15 / 16 * ((b + turn) * 0.6180339887498949 % 1.0)))) for b in range(n)]
    got[-1] = top
    return got


def _sizes(case):
    """(new tokens, tokens cached before them) of every sequence."""
    new = _spread_sizes(case["batch"], case["new"], case["ragged"], 1, 1)
    return new, _spread_sizes(case["batch"], case["before"], case["ragged"], 0, 4)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "chunk":
        rows = tokens = pairs = 0
        for n, b in zip(*_sizes(case)):
            rows += n
            tokens += n + b
            pairs += n * b + n * (n + 1) // 2
        return {"bytes": tokens * case["kv_heads"] * _data(case["dim"])
                + rows * case["heads"] * (case["dim"] * 2 * size + 4),
                "flops": 4.0 * pairs * case["heads"] * case["dim"]}
    rows, cells = case["rows"], case["rows"] * case["vocab"]
    if case["op"] == "score":
        return {"bytes": cells * size + rows * (4 + 12 + 8 * case["k"]), "flops": 6.0 * cells}
    return {"bytes": 2 * cells * size + rows * (4 + 8 + 8 + 8 * case["k"]), "flops": 8.0 * cells}


# ---- what a program has in hand --------------------------------------------------------------------------------
def _rand_pool(shape, dim, g):
    """Records as quantised channels give them: codes of rounded normal values, scales around a quarter."""
    pool = torch.zeros(shape, dtype=torch.uint8, device=DEV)
    flat = pool.view(-1, shape[-1])
    for part in flat.split(1 << 21):
        u = torch.randn((part.shape[0], dim, 2), device=DEV, dtype=torch.float16, generator=g)
        u = u.mul_(2.5).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        part[:, :dim] = u[..., 0] | (u[..., 1] << 4)
        s = torch.rand((part.shape[0], 2 * dim // GROUP), device=DEV, generator=g).mul_(0.2).add_(0.15)
        part[:, dim:_data(dim)] = s.half().view(torch.uint8).view(part.shape[0], -1)
    return pool


def _spread(lengths, page, g, spare=3):
    """A table whose sequences' pages lie at random places of the pool, and the number of pages of that pool."""
    used = [-(-n // page) for n in lengths]
    total = sum(used) + spare
    wide = max(1, max(used))
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    have = torch.tensor(used, device=DEV)
    start = torch.cumsum(have, 0) - have
    col = torch.arange(wide, device=DEV)
    at = (start[:, None] + col).clamp_(max=total - 1)
    table = torch.where(col < have[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
    return table.contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 31) + 54321)
    s = dict(case=case)
    if case["op"] == "chunk":
        new, before = _sizes(case)
        lengths = [n + b for n, b in zip(new, before)]
        s["table"], pages = _spread(lengths, case["page"], g)
        s["pool"] = _rand_pool((pages, case["kv_heads"], case["page"], _record(case["dim"])), case["dim"], g)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        s["starts"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=DEV)
        s["longest"] = max(new)
        s["q"] = torch.randn((sum(new), case["heads"], case["dim"]), device=DEV, generator=g).to(DTYPES[case["dtype"]])
        return s
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    # logits of a trained model: a broad bulk and, in each row, some tokens that stand out
    x = torch.randn((rows, vocab), device=DEV, generator=g).mul_(2.0)
    lead = torch.randint(0, vocab, (rows, 12), device=DEV, generator=g)
    x.scatter_add_(1, lead, torch.rand((rows, 12), device=DEV, generator=g).mul_(14.0))
    s["logits"] = x.to(DTYPES[case["dtype"]])
    pick = torch.randint(0, 12, (rows, 1), device=DEV, generator=g)
    stray = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    often = torch.rand(rows, device=DEV, generator=g) < 0.8
    s["tokens"] = torch.where(often, lead.gather(1, pick)[:, 0], stray).to(torch.int32)
    if case["op"] == "gradient":
        # what the forward pass left, and the gradients of what a loss took from it
        _, s["entropy"], s["lse"], s["idx"], _ = plain_score(s["logits"], s["tokens"], k, case["scale"])
        s["grad_logprob"] = torch.randn(rows, device=DEV, generator=g)
        s["grad_entropy"] = torch.randn(rows, device=DEV, generator=g).mul_(0.01)
        s["grad_top"] = torch.rand((rows, k), device=DEV, generator=g).neg_()
    return s


# ---- one pass --------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["op"] == "chunk":
        if own:
            out, lse = ds().kv4_chunk_attention(s["q"], s["pool"], s["table"], s["lengths"], s["starts"])
        else:
            out, lse = plain_chunk(s["q"], s["pool"], s["table"], s["lengths"], s["starts"], s["longest"])
        return {"out": out, "lse": lse}
    if case["op"] == "score":
        if own:
            got = ds().token_logprobs(s["logits"], s["tokens"], case["k"], scale=case["scale"])
        else:
            got = plain_score(s["logits"], s["tokens"], case["k"], case["scale"])
        return dict(zip(("logprob", "entropy", "lse", "idx", "top"), got))
    if own:
        grad = ds().token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"],
                                            grad_logprob=s["grad_logprob"], grad_entropy=s["grad_entropy"],
                                            idx=s["idx"], grad_top=s["grad_top"], scale=case["scale"])
    else:
        grad = plain_gradient(s["logits"], s["tokens"], s["lse"], s["entropy"], s["grad_logprob"], s["grad_entropy"],
                              s["idx"], s["grad_top"], case["scale"])
    return {"grad": grad}


# ---- the plain forms -------------------------------------------------------------------------------------------
def _nibbles(codes):
    """Codes of [..., bytes] as whole numbers [..., 2 * bytes], low half first."""
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _decode(records, dim):
    """Keys and values [..., dim] in 32 bits of records [..., record bytes]."""
    lead, half = records.shape[:-1], dim // 2
    wide = min(dim, 128)
    parts, groups = dim // wide, wide // GROUP
    kc = _nibbles(records[..., :half]).view(*lead, parts, 4, groups, 8).transpose(-3, -2)
    vc = _nibbles(records[..., half:dim]).view(*lead, parts, 8, groups, 4).transpose(-3, -2)
    scales = records[..., dim:_data(dim)].contiguous().view(torch.float16).float()
    ks, vs = scales.chunk(2, -1)
    k = (kc.reshape(*lead, dim // GROUP, GROUP).float() - 8) * ks[..., None]
    v = (vc.reshape(*lead, dim // GROUP, GROUP).float() - 8) * vs[..., None]
    return k.flatten(-2), v.flatten(-2)


def plain_chunk(q, pool, table, lengths, starts, longest):
    """Rows starts[b] to starts[b + 1] of q are the newest tokens of sequence b, `longest` of them at most."""
    _, heads, dim = q.shape
    hk, page = pool.shape[1:3]
    batch, n = table.shape[0], table.shape[1] * page
    count = (starts[1:] - starts[:-1]).long()
    j = torch.arange(longest, device=q.device)
    here = j < count[:, None]                                                          # [batch, longest]
    row = torch.where(here, starts[:-1].long()[:, None] + j, torch.zeros_like(j))
    limit = torch.where(here, (lengths.long() - count)[:, None] + 1 + j, torch.zeros_like(j)).clamp(min=0)
    x = q[row].float().view(batch, longest, hk, heads // hk, dim).permute(0, 2, 1, 3, 4)
    k, v = _decode(pool[table.long().clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(batch, hk, n, -1), dim)
    score = torch.matmul(x.reshape(batch, hk, -1, dim) / math.sqrt(dim), k.transpose(-1, -2))
    score = score.view(batch, hk, longest, heads // hk, n)
    hide = torch.arange(n, device=q.device) >= limit[..., None]                        # [batch, longest, tokens]
    score.masked_fill_(hide[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(batch, hk, -1, n), v).view(batch, hk, longest, heads // hk, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3)
    out = torch.empty_like(q)
    out[row[here]] = o[here].reshape(-1, heads, dim).to(q.dtype)
    out_lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    out_lse[row[here]] = lse[here].reshape(-1, heads)
    return out, out_lse


def plain_score(logits, tokens, k, scale):
    """(log probability of the given token, entropy, log of the sum, the k likeliest tokens, their log probabilities)"""
    z = logits.float() * scale
    top = z.amax(-1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    total = e.sum(-1)
    entropy = torch.log(total) - (e * d).sum(-1) / total
    lse = top[:, 0] + torch.log(total)
    logprob = z.gather(1, tokens.long()[:, None])[:, 0] - lse
    del d, e
    # the order by (value descending, index ascending) as one whole number; adding 0 makes -0 and 0 the same
    bits = (logits.float() + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * (1 << 32) - torch.arange(logits.shape[1], device=logits.device)
    idx = torch.topk(key, k, dim=-1)[1]
    return logprob, entropy, lse, idx.to(torch.int32), z.gather(1, idx) - lse[:, None]


def plain_gradient(logits, tokens, lse, entropy, grad_logprob, grad_entropy, idx, grad_top, scale):
    """Gradient of sum(grad_logprob logprob + grad_entropy entropy + grad_top top) by the logits."""
    logp = logits.float() * scale - lse[:, None]
    g = -(grad_logprob + grad_top.sum(-1))[:, None] - grad_entropy[:, None] * (logp + entropy[:, None])
    g = g * torch.exp(logp)
    g.scatter_add_(1, tokens.long()[:, None], grad_logprob[:, None])
    g.scatter_add_(1, idx.long(), grad_top)
    return (g * scale).to(logits.dtype)


# ---- the definition in 64 bits ---------------------------------------------------------------------------------
def _channels64(records, dim):
    """Keys and values in 64 bits, each channel looked up at its own place in the record."""
    wide = min(dim, 128)
    groups = wide // GROUP
    d = torch.arange(dim, device=records.device)
    base, c = d // wide * wide, d % wide
    i, r = c // GROUP, c % GROUP
    at = {"k": base + ((r // 8) * groups + i) * 8 + r % 8, "v": base + ((r // 4) * groups + i) * 4 + r % 4}
    scales = records[..., dim:_data(dim)].contiguous().view(torch.float16).double()
    got = []
    for name, first, lo in (("k", 0, 0), ("v", dim // 2, dim // GROUP)):
        byte = records[..., first + at[name] // 2].to(torch.int32)
        u = torch.where(at[name] % 2 == 1, byte >> 4, byte & 15)
        got.append((u - 8).double() * scales[..., lo + d // GROUP])
    return got


def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "chunk":
        heads, hk, page, dim = case["heads"], case["kv_heads"], case["page"], case["dim"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
        first = 0
        for b, (n, before) in enumerate(zip(*_sizes(case))):
            t = torch.arange(before + n, device=DEV)
            k, v = _channels64(s["pool"][s["table"][b].long()[t // page], :, t % page], dim)  # [tokens, hk, dim]
            unseen = t[None] > (before + torch.arange(n, device=DEV))[:, None]
            for h in range(heads):
                x = s["q"][first:first + n, h].double()
                score = (x @ k[:, h * hk // heads].T) / math.sqrt(dim)
                score.masked_fill_(unseen, -math.inf)
                lse[first:first + n, h] = torch.logsumexp(score, -1)
                out[first:first + n, h] = torch.softmax(score, -1) @ v[:, h * hk // heads]
            first += n
        return {"out": out, "lse": lse}
    at = torch.arange(case["rows"], device=DEV)
    logp = torch.log_softmax(s["logits"].double() * case["scale"], -1)
    if case["op"] == "score":
        z = s["logits"].double() * case["scale"]
        idx = plain_score(s["logits"], s["tokens"], case["k"], case["scale"])[3].long()
        return {"logprob": logp[at, s["tokens"].long()], "entropy": torch.special.entr(logp.exp()).sum(-1),
                "lse": torch.logsumexp(z, -1), "idx": None, "top": logp.gather(1, idx)}
    p = logp.exp()
    gp, ge, gt = (s["grad_" + name].double() for name in ("logprob", "entropy", "top"))
    # by the chain through log p: the gradient of sum(w log p) + ge entropy, w the weights of the given tokens
    w = torch.zeros_like(p)
    w[at, s["tokens"].long()] = gp
    w.scatter_add_(1, s["idx"].long(), gt)
    entropy = -(p * logp).sum(-1, keepdim=True)
    g = w - p * w.sum(-1, keepdim=True) - ge[:, None] * p * (logp + entropy)
    return {"grad": g * case["scale"]}
