"""Attention over the 4-bit cache for values of every size that its scales can hold, and for
probabilities that one token dwarfs, against the 64-bit model."""
import numpy as np
import pytest

import oracle.kv4 as model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as _ds
    _ds.build()
    _ds.load_library()
    return _ds


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def largest_scales(pool, table, lengths, dim):
    """Largest value scale of each sequence's tokens, [sequence, head, channel]."""
    page = pool.shape[2]
    n = dim // 32 * 2
    got = np.zeros((len(lengths), pool.shape[1], dim))
    for b, length in enumerate(lengths):
        t = np.arange(length)
        rec = pool[table[b, t // page], :, t % page]
        s = np.ascontiguousarray(rec[..., dim + n:dim + 2 * n]).view(np.float16).astype(np.float64)
        if length:
            got[b] = np.repeat(s.max(0), 32, -1)
    return got


def check(ds, q, dtype, k, v, lengths, page, indices=None):
    """Attention over records of k and v [tokens, heads, dim], whose tokens are the sequences' one
    after another.

    Bounds.  A weight, probability times value scale, is rounded to fp16's 11 significant bits:
    2^-11 relative.  What is below 2^-28 of the largest probability times the group's largest
    scale may be off by 2^-39 of that instead, a code is at most 8 and the sum of probabilities at
    least 1: 8 n 2^-39 of the largest scale for n tokens.  Scores are sums in 32 bits, 2^-18 of
    the sum of their terms' sizes (32 roundings of 2^-23), which moves a probability by as much in
    the numerator and in the sum; exp and the sums: 2^-18.  Nothing else is allowed, so that the
    bound shrinks with the values."""
    batch, queries, heads, dim = q.shape
    hk = k.shape[1]
    wide = -(-max(max(lengths), 1) // page)
    order = np.random.default_rng(0).permutation(batch * wide + 1).astype(np.int32)
    table = order[:batch * wide].reshape(batch, wide)
    pool = np.zeros((len(order), hk, page, model.record_bytes(dim)), dtype=np.uint8)
    rec, at = model.encode(k.astype(np.float32), v.astype(np.float32)), 0
    for b, n in enumerate(lengths):
        t = np.arange(n)
        pool[table[b, t // page], :, t % page] = rec[at:at + n]
        at += n
    lengths = np.array(lengths, dtype=np.int32)
    qt = dev(q.astype(np.float32)).to(DTYPES[dtype])
    out, lse = ds.kv4_attention(qt, dev(pool), dev(table), dev(lengths),
                                indices=None if indices is None else dev(indices))
    ref, rlse, spread, reach = model.attention(qt.double().cpu().numpy(), pool, table, lengths, dim ** -0.5,
                                               indices)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = int(lengths.max()) if indices is None else indices.shape[2]
    most = np.repeat(largest_scales(pool, table, lengths, dim), heads // hk, 1)[:, None]
    move = 2.0 ** -18 * (1 + reach)
    t = (2.0 ** -11 + 2 * move[..., None]) * spread + 8 * n * 2.0 ** -39 * most
    lo, hi = (torch.from_numpy(x).to(qt.dtype).double().numpy() for x in (ref - t, ref + t))
    assert np.isfinite(got).all()
    off = ~((lo <= got) & (got <= hi))
    assert not off.any(), (off.mean(), np.max(np.abs(got - ref) / np.maximum(t, 1e-300)))
    seen = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(glse), ~seen)
    assert (np.abs(glse[seen] - rlse[seen]) <= move[seen] + 2.0 ** -21 * (1 + np.abs(rlse[seen]))).all()
    return ref


SHAPES = [(64, 2, 3), (128, 2, 4), (256, 1, 5), (64, 1, 12), (128, 1, 16), (256, 1, 11)]


def data(seed, lengths, hk, group, dim, queries=1, sharp=1.0):
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((2, sum(lengths), hk, dim))
    q = rng.standard_normal((len(lengths), queries, hk * group, dim)) * sharp
    return rng, q, k, v


@pytest.mark.parametrize("dim,hk,group", SHAPES)
@pytest.mark.parametrize("size", [1e-7, 1e-6, 1e-5, 1e-4, 1e-2, 1e6])
def test_size_of_the_values(ds, dim, hk, group, size):
    """From scales that are fp16's smallest number to scales that are its largest."""
    lengths = [1, 0, 45, 700, 2600]
    _, q, k, v = data(dim + group, lengths, hk, group, dim)
    ref = check(ds, q, "bf16", k, v * size, lengths, 16)
    assert np.abs(ref[3:]).max() > 0


@pytest.mark.parametrize("dim,hk,group", SHAPES)
@pytest.mark.parametrize("size", [1e-5, 1e-3])
def test_one_token_dwarfs_the_others(ds, dim, hk, group, size):
    """One score lies 12 above the others; its value is small, so that theirs still count."""
    lengths = [900, 2500]
    rng, q, k, v = data(7 * dim + group, lengths, hk, group, dim)
    base = rng.standard_normal(dim)
    q = base * (1 + 0.02 * rng.standard_normal((2, 1, hk * group, 1)))
    for at in (3, 900 + 1234):
        k[at] = base * 12 / (base @ base * dim ** -0.5)
        v[at] *= 1e-4
    check(ds, q, "bf16", k, v * size, lengths, 48)


@pytest.mark.parametrize("dim,hk,group", SHAPES)
@pytest.mark.parametrize("rising", [True, False])
def test_values_of_unequal_size(ds, dim, hk, group, rising):
    """Groups of channels from 1e-6 to 1e4, and tokens whose values grow or shrink a hundredfold."""
    lengths = [333, 1800]
    _, q, k, v = data(3 * dim + group, lengths, hk, group, dim)
    v *= np.repeat(10.0 ** np.linspace(-6, 4, dim // 32), 32)
    at = np.concatenate([np.arange(n) / n for n in lengths])
    v *= (10.0 ** (2 * (at if rising else 1 - at) - 1))[:, None, None]
    check(ds, q, "bf16", k, v, lengths, 7)


@pytest.mark.parametrize("dim,hk,group", SHAPES)
@pytest.mark.parametrize("dtype,queries", [("fp16", 1), ("bf16", 3)])
def test_listed_tokens_with_small_values(ds, dim, hk, group, dtype, queries):
    lengths = [60, 3000]
    rng, q, k, v = data(5 * dim + group, lengths, hk, group, dim, queries)
    idx = rng.integers(-40, 3000, (2, queries, 1300)).astype(np.int32)
    check(ds, q, dtype, k, v * (1e-3 if dtype == "fp16" else 3e-6), lengths, 16, idx)


@pytest.mark.parametrize("dim,hk,group", SHAPES)
def test_values_that_no_query_sees(ds, dim, hk, group):
    """The newest tokens' huge values, which earlier queries do not see, cost those no accuracy, and
    neither do other tokens' records in the same tile that a list leaves out."""
    lengths = [37, 410]
    rng, q, k, v = data(11 * dim + group, lengths, hk, group, dim)
    v *= 1e-5
    huge = v.copy()
    huge[[36, 36 + 410]] = 1e5
    idx = np.full((2, 1, 20), -1, dtype=np.int32)
    idx[0, 0, 3:18], idx[1, 0] = np.arange(15) * 2, np.arange(20) * 20
    check(ds, q, "bf16", k, huge, lengths, 16, idx)
