"""Plain 64-bit model of the 4-bit paged cache (include/ds_kv4.h): records,
attention and the pages' bookkeeping, in numpy and plain Python.  Test
infrastructure only; it shares no code with the library."""
import numpy as np

GROUP = 32


def data_bytes(dim):
    return dim + 4 * (dim // GROUP)


def record_bytes(dim):
    return -(-data_bytes(dim) // 16) * 16


def channel_places(dim):
    """For each channel, the place of its code (in codes) within the key's and the value's part."""
    key, value = [], []
    wide = min(dim, 128)
    n = wide // GROUP
    for c in range(dim):
        base, local = c // wide * wide, c % wide
        word = local // 8                      # 4 i + t -> n t + i
        i, t = divmod(word, 4)
        key.append(base + (n * t + i) * 8 + local % 8)
        piece = local // 4                     # 8 i + g -> n g + i
        i, g = divmod(piece, 8)
        value.append(base + (n * g + i) * 4 + local % 4)
    return np.array(key), np.array(value)


def quantise(x):
    """(codes 0..15 [..., D], scales fp16 [..., D/32]) of float32 values x."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    with np.errstate(all="ignore"):
        top = np.where(bad, np.float32(0), np.abs(g).max(-1).astype(np.float32))
        scale = (top * (np.float32(1) / np.float32(7))).astype(np.float16)
        scale = np.where(np.isinf(scale), np.float16(65504), scale)
        step = scale.astype(np.float32)[..., None]
        code = np.where((step > 0) & ~bad[..., None], np.rint(g / step), 0)
        code = np.clip(code, -7, 7)
    scale = scale.astype(np.float16).view(np.uint16)
    scale = np.where(bad, np.uint16(0x7FFF), scale).view(np.float16)
    return (code.astype(np.int64) + 8).reshape(x.shape), scale


def encode(k, v):
    """Records uint8 [..., record bytes] of float32 keys and values [..., D]."""
    dim = k.shape[-1]
    places = channel_places(dim)
    rec = np.zeros((*k.shape[:-1], record_bytes(dim)), dtype=np.uint8)
    for which, x in enumerate((k, v)):
        code, scale = quantise(x)
        part = np.zeros((*k.shape[:-1], dim), dtype=np.int64)
        part[..., places[which]] = code
        first = which * dim // 2
        rec[..., first:first + dim // 2] = part[..., 0::2] | part[..., 1::2] << 4
        n = dim // GROUP * 2
        rec[..., dim + which * n:dim + (which + 1) * n] = np.ascontiguousarray(scale).view(np.uint8)
    return rec


def decode(rec, dim):
    """Keys and values in 64 bits of records."""
    out = []
    places = channel_places(dim)
    for which in range(2):
        b = rec[..., which * dim // 2:(which + 1) * dim // 2].astype(np.int64)
        code = np.stack((b & 15, b >> 4), -1).reshape(*rec.shape[:-1], dim)[..., places[which]]
        n = dim // GROUP * 2
        s = np.ascontiguousarray(rec[..., dim + which * n:dim + (which + 1) * n]).view(np.float16)
        out.append((code - 8) * np.repeat(s.astype(np.float64), GROUP, -1))
    return out


def slots(table, n_pages, page, seq, positions):
    """(page, offset) of the positions that are there, and which those are."""
    p = np.asarray(positions, dtype=np.int64)
    there = (p >= 0) & (p < table.shape[1] * page) & (0 <= seq < table.shape[0])
    col = np.where(there, p // page, 0)
    home = table[seq if 0 <= seq < table.shape[0] else 0, col].astype(np.int64)
    there &= (home >= 0) & (home < n_pages)
    return home, p % page, there


def attention(q, pool, table, lengths, scale, indices=None, seqs=None):
    """(out, lse, spread, reach) in 64 bits of float64 q [B, Tq, H, D].

    spread: sum of p |v| over the sum of p, per output; reach: the largest
    scale * sum |q| |code| * key scale, per (b, j, h) -- what the rounding
    errors of probabilities and scores are multiples of."""
    batch, queries, heads, dim = q.shape
    n_pages, hk, page, _ = pool.shape
    out = np.zeros(q.shape)
    spread = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    reach = np.zeros(q.shape[:3])
    for b in range(batch):
        seq = b if seqs is None else int(seqs[b])
        length = int(lengths[seq]) if 0 <= seq < table.shape[0] else 0
        length = max(0, min(length, table.shape[1] * page))
        for j in range(queries):
            limit = max(0, length - queries + 1 + j)
            t = np.arange(limit) if indices is None else np.asarray(indices[b, j], dtype=np.int64)
            t = t[(t >= 0) & (t < limit)]
            home, off, there = slots(table, n_pages, page, seq, t)
            home, off = home[there], off[there]
            if not home.size:
                continue
            k, v = decode(pool[home, :, off], dim)             # [tokens, hk, D]
            for h in range(heads):
                g = h // (heads // hk)
                with np.errstate(all="ignore"):
                    s = scale * (k[:, g] @ q[b, j, h])
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    out[b, j, h] = p @ v[:, g] / total
                    spread[b, j, h] = p @ np.abs(v[:, g]) / total
                    lse[b, j, h] = m + np.log(total)
                    reach[b, j, h] = (abs(scale) * (np.abs(k[:, g]) + 8 * np.repeat(
                        np.abs(k[:, g]).reshape(len(k), -1, GROUP).max(-1) / 7, GROUP, -1))
                        @ np.abs(q[b, j, h])).max()
    return out, lse, spread, reach


def rising(starts, tokens):
    """Starts of chunks as they are read: within [0, tokens], and never falling."""
    return np.maximum.accumulate(np.clip(np.asarray(starts, dtype=np.int64), 0, tokens))


def chunk_attention(q, pool, table, lengths, starts, scale, seqs=None):
    """(out, lse, spread, reach) in 64 bits of float64 q [tokens, H, D]: rows starts[b] to
    starts[b + 1] are the newest tokens of entry b's sequence.  Rows of no entry are NaN.

    spread and reach as in attention(), reach without the codes' offset."""
    tokens, heads, dim = q.shape
    n_pages, hk, page, _ = pool.shape
    group = heads // hk
    out, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, reach = np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    starts = rising(starts, tokens)
    for b in range(len(starts) - 1):
        seq = b if seqs is None else int(seqs[b])
        length = int(lengths[seq]) if 0 <= seq < table.shape[0] else 0
        length = max(0, min(length, table.shape[1] * page))
        home, off, there = slots(table, n_pages, page, seq, np.arange(length))
        k, v = decode(pool[np.where(there, home, 0), :, off], dim)       # [length, hk, D]
        first, n = starts[b], starts[b + 1] - starts[b]
        for j in range(n):
            seen = there[:max(0, length - n + 1 + j)]
            row = first + j
            out[row], spread[row], lse[row], reach[row] = 0, 0, -np.inf, 0
            if not seen.any():
                continue
            for g in range(hk):
                x, kk, vv = q[row, g * group:(g + 1) * group], k[:len(seen), g][seen], v[:len(seen), g][seen]
                with np.errstate(all="ignore"):
                    s = scale * (x @ kk.T)
                    m = s.max(-1, keepdims=True)
                    p = np.exp(s - m)
                    total = p.sum(-1, keepdims=True)
                    at = slice(g * group, (g + 1) * group)
                    out[row, at] = p @ vv / total
                    spread[row, at] = p @ np.abs(vv) / total
                    lse[row, at] = (m + np.log(total))[:, 0]
                    reach[row, at] = abs(scale) * (np.abs(x) @ np.abs(kk).T).max(-1)
    return out, lse, spread, reach


class Book:
    """The pages' bookkeeping, one step at a time."""

    def __init__(self, table, lengths, refs, page):
        self.table, self.lengths, self.refs = table.copy(), lengths.copy(), refs.copy()
        self.page = page

    def used(self, s):
        return -(-int(self.lengths[s]) // self.page)

    def free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0]

    def reserve(self, seqs, tokens):
        need, seen = [], set()
        short = 0
        for s, t in zip(seqs, tokens):
            s, t = int(s), int(t)
            if not 0 <= s < len(self.lengths) or t < 1 or s in seen:
                continue
            seen.add(s)
            want = -(-(int(self.lengths[s]) + t) // self.page)
            short += max(0, want - self.table.shape[1])
            need.append((s, t, self.used(s), min(want, self.table.shape[1])))
        free = self.free_pages()
        total = sum(want - have for _, _, have, want in need)
        short += max(0, total - len(free))
        if short:
            return short, 0
        for s, t, have, want in need:
            for j in range(have, want):
                p = free.pop(0)
                self.table[s, j] = p
                self.refs[p] = 1
            self.lengths[s] += t
        return 0, total

    def fork(self, pool, src, dst):
        pairs, seen = [], set()
        before = self.lengths.copy()
        for s, d in zip(src, dst):
            s, d = int(s), int(d)
            n = len(before)
            if not (0 <= s < n and 0 <= d < n) or s == d or before[d] != 0 or d in seen:
                continue
            seen.add(d)
            pairs.append((s, d, int(before[s])))
        free = self.free_pages()
        total = sum(n % self.page != 0 for _, _, n in pairs)
        if total > len(free):
            return total - len(free), 0
        for s, d, n in pairs:
            full = n // self.page
            self.table[d] = -1
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if n % self.page:
                p = free.pop(0)
                self.table[d, full] = p
                self.refs[p] = 1
                pool[:, p] = pool[:, self.table[s, full]]
            self.lengths[d] = n
        return 0, total

    def free(self, seqs):
        for s in dict.fromkeys(int(s) for s in seqs):
            if 0 <= s < len(self.lengths):
                for p in self.table[s, :self.used(s)]:
                    self.refs[p] -= 1
                self.table[s] = -1
                self.lengths[s] = 0

    def compact(self, pool):
        n = int((self.refs > 0).sum())
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        remap = np.array([p if self.refs[p] > 0 else -1 for p in range(len(self.refs))], dtype=np.int32)
        for h, m in zip(holes, movers):
            remap[m] = h
            pool[:, h] = pool[:, m]
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.table = np.where(self.table >= 0, remap[np.maximum(self.table, 0)], self.table)
        return remap, (n, len(movers))
