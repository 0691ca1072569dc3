"""Plain 64-bit model of include/ds_logprob.h in numpy: log probabilities of given
tokens, entropy, the likeliest alternatives, and their gradient.  Test
infrastructure only; it shares no code with the library."""
import numpy as np


def order(x):
    """Indices of a row by (value descending, index ascending), NaN above +inf, -0 equal to +0."""
    x = np.asarray(x, dtype=np.float64) + 0.0
    nan = np.isnan(x)
    return np.lexsort((np.arange(len(x)), -np.where(nan, 0.0, x), ~nan))


def log_probs(z):
    """(log probabilities, log of the sum, entropy) of one row; differences from the maximum are taken
    first, so that rows of any magnitude keep them."""
    live = z[~np.isneginf(z)]
    if np.isnan(live).any() or np.isposinf(live).any():
        return np.full(len(z), np.nan), np.nan, np.nan
    if not live.size:
        return np.full(len(z), -np.inf), -np.inf, 0.0
    m = live.max()
    e = np.exp(live - m)
    bits = np.log(e.sum())
    return (z - m) - bits, m + bits, bits - (e * (live - m)).sum() / e.sum()


def forward(x, tokens, k, scale):
    """(logprob, entropy, lse [rows], idx, top [rows, k]) of float64 logits x."""
    rows, vocab = x.shape
    logprob, entropy, lse = np.zeros(rows), np.zeros(rows), np.full(rows, -np.inf)
    idx, top = np.zeros((rows, k), dtype=np.int64), np.zeros((rows, k))
    for r in range(rows):
        lp, lse[r], entropy[r] = log_probs(x[r] * scale)
        idx[r] = order(x[r])[:k]
        top[r] = lp[idx[r]]
        if 0 <= tokens[r] < vocab:
            logprob[r] = lp[tokens[r]]
    return logprob, entropy, lse, idx, top


def backward(x, tokens, idx, scale, g_logprob, g_entropy, g_lse, g_top):
    """Gradient by x of sum(g_logprob logprob + g_entropy entropy + g_lse lse + g_top top), from the
    definition: the vocab weights w of log probabilities, then the chain through the softmax."""
    rows, vocab = x.shape
    out = np.zeros_like(x)
    for r in range(rows):
        lp, lse, entropy = log_probs(x[r] * scale)
        if np.isneginf(lse):
            continue
        w = np.zeros(vocab)
        if 0 <= tokens[r] < vocab:
            w[tokens[r]] += g_logprob[r]
        for i, g in zip(idx[r], g_top[r]):
            if 0 <= i < vocab:
                w[i] += g
        with np.errstate(invalid="ignore"):
            p = np.exp(lp)
            surprise = np.where(p == 0, 0.0, p * (np.where(p == 0, 0.0, lp) + entropy))
        out[r] = scale * (w + p * (g_lse[r] - w.sum()) - g_entropy[r] * surprise)
    return out
