"""The 4-bit paged cache on the GPU against the 64-bit model: records bit for
bit, attention within bounds derived from its roundings."""
import numpy as np
import pytest

import oracle.kv4 as model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as _ds
    _ds.build()
    _ds.load_library()
    return _ds


def make_table(rng, lengths, page, wide, spare=2):
    """Pages at random places; returns (table, number of pages)."""
    used = [-(-max(0, n) // page) for n in lengths]
    order = rng.permutation(sum(used) + spare).astype(np.int32)
    table = np.full((len(lengths), wide), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


def random_pool(rng, n_pages, hk, page, dim, spread=1.0):
    """Records of normal keys and values, with noise where no token is."""
    k, v = (rng.standard_normal((2, n_pages, hk, page, dim)) * spread).astype(np.float32)
    return model.encode(k, v)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def check_attention(ds, q, dtype, pool, table, lengths, scale=None, indices=None, seqs=None, **kw):
    """Runs attention and compares with the model.

    Bounds.  The result before its rounding to q's type is within t of the
    model's, so the output lies between the roundings of the model's value
    minus t and plus t (rounding keeps order).  A probability times a value
    scale may be rounded to fp16: 2^-11 relative, and 2^-25 absolute where it
    is below fp16's normal range; a code is at most 8, so n tokens give
    8 n 2^-25 over a sum that is at least 1.  Scores are sums in 32 bits of up
    to 256 products of total magnitude `reach` (offset codes: |u| <= 15):
    2^-18 reach covers 32 roundings of 2^-23; it moves a probability by as
    much, both in the numerator and in the sum.  exp and the sums: 2^-18."""
    dim = q.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    qt = q if isinstance(q, torch.Tensor) else dev(q).to(DTYPES[dtype])
    out, lse = ds.kv4_attention(
        qt, dev(pool) if isinstance(pool, np.ndarray) else pool, dev(table), dev(lengths),
        scale=scale, indices=None if indices is None else dev(indices),
        seqs=None if seqs is None else dev(seqs), **kw)
    torch.cuda.synchronize()
    host = pool if isinstance(pool, np.ndarray) else pool.cpu().numpy()
    ref, rlse, spread, reach = model.attention(qt.double().cpu().numpy(), host, table, lengths, scale,
                                               indices, seqs)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = table.shape[1] * host.shape[2] if indices is None else indices.shape[2]
    move = 2.0 ** -18 * (1 + reach)
    t = (2.0 ** -11 + 2 * move[..., None]) * spread + 8 * n * 2.0 ** -25
    lo, hi = (torch.from_numpy(x).to(qt.dtype).double().numpy() for x in (ref - t, ref + t))
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert ((lo <= got) & (got <= hi))[fine].all(), np.nanmax(np.abs(got - ref) / t)
    assert np.array_equal(np.isneginf(glse), np.isneginf(rlse))
    f = np.isfinite(rlse)
    assert (np.abs(glse[f] - rlse[f]) <= (move + 2.0 ** -21 * (1 + np.abs(rlse)))[f]).all()
    return out, lse


# ---- append and read -----------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("page,hk", [(16, 2), (1, 1), (7, 3)])
def test_append_and_read(ds, dim, dtype, page, hk):
    rng = np.random.default_rng(dim * page + hk)
    lengths = [0, 1, 23, page, 40]
    table, n_pages = make_table(rng, lengths, page, wide=45)
    seq = np.repeat(np.arange(5), lengths).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
    order = rng.permutation(len(seq))
    seq, pos = seq[order], pos[order]
    x = (rng.standard_normal((2, len(seq), hk, dim)) * np.exp(rng.normal(size=(2, len(seq), 1, 1)))
         ).astype(np.float32)
    k, v = (dev(t).to(DTYPES[dtype]) for t in x)
    before = rng.integers(0, 256, (n_pages, hk, page, model.record_bytes(dim)), dtype=np.uint8)
    pool = dev(before)
    ds.kv4_append(pool, dev(table), dev(seq), dev(pos), k, v)
    want = before.copy()
    rec = model.encode(k.float().cpu().numpy(), v.float().cpu().numpy())
    want[table[seq, pos // page], :, pos % page] = rec
    assert np.array_equal(pool.cpu().numpy(), want)
    gk, gv = ds.kv4_read(pool, dev(table), dev(seq), dev(pos), dim, DTYPES[dtype])
    for got, ref in zip((gk, gv), model.decode(rec, dim)):
        ref = torch.from_numpy(ref.astype(np.float32)).to(DTYPES[dtype])
        assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_append_of_strided_keys_and_values(ds, dtype, offset):
    """Slices of a fused projection, at starts that are and are not 16-byte aligned."""
    rng = np.random.default_rng(offset)
    hk, dim, tokens = 2, 64, 9
    wide = dev(rng.standard_normal((tokens, 3 * hk * dim + 13)).astype(np.float32)).to(DTYPES[dtype])
    k = wide.as_strided((tokens, hk, dim), (wide.stride(0), dim, 1), offset)
    v = wide.as_strided((tokens, hk, dim), (wide.stride(0), dim + 3, 1), offset + hk * dim)
    pool = torch.zeros((2, hk, 16, 80), dtype=torch.uint8, device=DEV)
    table = np.array([[1, 0]], dtype=np.int32)
    seq, pos = np.zeros(tokens, dtype=np.int32), np.arange(12, 12 + tokens, dtype=np.int32)
    ds.kv4_append(pool, dev(table), dev(seq), dev(pos), k, v)
    want = np.zeros((2, hk, 16, 80), dtype=np.uint8)
    want[table[seq, pos // 16], :, pos % 16] = model.encode(k.float().cpu().numpy(),
                                                           v.float().cpu().numpy())
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_of_special_values(ds):
    """Zero groups, NaN and infinite groups, values beyond fp16 scales and below them."""
    x = np.zeros((9, 1, 128), dtype=np.float32)
    x[1] = 1e30
    x[2, 0, 5] = np.nan
    x[3, 0, 70] = np.inf
    x[4, 0, 70] = -np.inf
    x[5] = 1e-8
    x[6] = -3e-7
    x[7] = np.linspace(-3.5, 3.5, 128)
    x[8] = -0.0
    pool = torch.zeros((1, 1, 9, 144), dtype=torch.uint8, device=DEV)
    table, seq, pos = (dev(np.zeros((1, 1), np.int32)), dev(np.zeros(9, np.int32)),
                       dev(np.arange(9, dtype=np.int32)))
    ds.kv4_append(pool, table, seq, pos, dev(x), dev(x[::-1]))
    want = model.encode(x, x[::-1].copy())
    assert np.array_equal(pool.cpu().numpy()[0, 0], want[:, 0])
    k, v = ds.kv4_read(pool, table, seq, pos, 128, torch.float32)
    rk, rv = model.decode(want, 128)
    assert np.array_equal(k.cpu().numpy(), rk.astype(np.float32), equal_nan=True)
    assert np.array_equal(v.cpu().numpy(), rv.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_ties_and_their_neighbours(ds, dtype):
    """Channels at and next to (n + 1/2) * scale, for every significand of a scale and exponents
    from subnormal scales to the largest; values beyond all scales."""
    step = (np.arange(1024, 2048)[:, None] * 2.0 ** np.array([-34, -25, -12, 0, 3])).reshape(-1)
    ties = np.concatenate([np.arange(-7, 7) + 0.5, [7.0, -7.0]])
    x = (step[:, None] * ties).astype(np.float32)
    t = torch.from_numpy(x).to(DTYPES[dtype])
    up, down = (torch.nextafter(t, torch.full_like(t, side)) for side in (np.inf, -np.inf))
    t = torch.stack([t, t, up, down, t, up], 1).reshape(-1, 3, 32)
    t[:, 1:, 30] = t[:, :1, 30]            # groups of one scale, where the neighbours' is not larger
    big = torch.finfo(DTYPES[dtype]).max
    t = torch.cat([t.reshape(-1, 32), torch.linspace(-1, 1, 32)[None].to(t.dtype) * big,
                   torch.full((1, 32), -big, dtype=t.dtype)])
    x = t[:len(t) // 4 * 4].reshape(-1, 1, 128).to(DEV)
    tail = t[-4:].reshape(1, 1, 128).to(DEV)
    k = torch.cat([x, tail])
    v = k.flip(0)
    tokens = len(k)
    pool = torch.zeros((-(-tokens // 64), 1, 64, 144), dtype=torch.uint8, device=DEV)
    table = dev(np.arange(len(pool), dtype=np.int32)[None])
    seq, pos = dev(np.zeros(tokens, np.int32)), dev(np.arange(tokens, dtype=np.int32))
    ds.kv4_append(pool, table, seq, pos, k, v)
    want = model.encode(k.float().cpu().numpy(), v.float().cpu().numpy())
    assert np.array_equal(pool.cpu().numpy().reshape(-1, 144)[:tokens], want[:, 0])


def test_tokens_that_are_not_there(ds):
    """Out-of-range sequences, positions and pages: nothing is written, zeros are read."""
    table = np.array([[0, -1, 5], [2, 1, -7]], dtype=np.int32)   # 3 pages in the pool
    seq = np.array([-1, 2, 0, 0, 0, 0, 1, 1, 2 ** 31 - 1], dtype=np.int32)
    pos = np.array([0, 0, -1, 4, 8, 12, 11, 2 ** 31 - 1, 0], dtype=np.int32)
    before = np.random.default_rng(0).integers(0, 256, (3, 1, 4, 80), dtype=np.uint8)
    pool = dev(before)
    x = torch.ones((9, 1, 64), device=DEV)
    ds.kv4_append(pool, dev(table), dev(seq), dev(pos), x, x)
    assert np.array_equal(pool.cpu().numpy(), before)
    k, v = ds.kv4_read(pool, dev(table), dev(seq), dev(pos), 64, torch.float32)
    assert (k == 0).all() and (v == 0).all()
    none = torch.zeros((0, 1, 64), device=DEV)
    ds.kv4_append(pool, dev(table), dev(seq[:0]), dev(pos[:0]), none, none)
    assert np.array_equal(pool.cpu().numpy(), before)


# ---- attention ------------------------------------------------------------------
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("hk,group", [(1, 1), (2, 3), (1, 8), (1, 16), (2, 40)])
@pytest.mark.parametrize("page,queries", [(16, 1), (7, 3), (48, 5), (64, 2)])
def test_attention(ds, dim, dtype, hk, group, page, queries):
    rng = np.random.default_rng(dim + 7 * hk + group + 1000 * page)
    lengths = np.array([0, 1, 2, 31, 32, 33, 130, 517], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, page, wide=-(-520 // page))
    pool = random_pool(rng, n_pages, hk, page, dim)
    q = rng.standard_normal((len(lengths), queries, hk * group, dim)).astype(np.float32)
    check_attention(ds, q, dtype, pool, table, lengths)


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16")])
@pytest.mark.parametrize("hk,group,k", [(1, 1, 1), (2, 8, 33), (1, 12, 200), (3, 4, 64)])
@pytest.mark.parametrize("page,queries", [(16, 1), (5, 3), (64, 2)])
def test_selected_attention(ds, dim, dtype, hk, group, k, page, queries):
    """Lists with -1, positions that are not seen, and positions listed twice."""
    rng = np.random.default_rng(dim + 7 * hk + group + 1000 * page)
    lengths = np.array([0, 1, 5, 40, 133, 260], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, page, wide=-(-260 // page))
    pool = random_pool(rng, n_pages, hk, page, dim)
    idx = rng.integers(-3, 300, (6, queries, k)).astype(np.int32)
    idx[4, 0] = -1
    idx[5, 0] = rng.permutation(260)[:k] if k <= 260 else idx[5, 0]
    q = rng.standard_normal((6, queries, hk * group, dim)).astype(np.float32)
    check_attention(ds, q, dtype, pool, table, lengths, indices=idx)


@pytest.mark.parametrize("dim,hk,group,k,batch", [
    (128, 2, 4, 1500, 3), (64, 1, 16, 2048, 2), (256, 1, 3, 1025, 2), (128, 1, 32, 700, 1), (64, 3, 2, 4096, 1),
    (128, 1, 8, 20000, 2), (256, 1, 16, 555, 2), (64, 8, 4, 600, 40), (128, 1, 40, 513, 2)])
def test_long_lists(ds, dim, hk, group, k, batch):
    """Lists that are one CTA's, that a cluster shares, and that a launch joins; parts without any token."""
    rng = np.random.default_rng(dim + k)
    page = 16
    lengths = np.array([3000] * batch, dtype=np.int32)
    lengths[0] = 40
    table, n_pages = make_table(rng, lengths, page, wide=-(-3000 // page))
    pool = random_pool(rng, n_pages, hk, page, dim)
    idx = rng.integers(0, 3000, (batch, 1, k)).astype(np.int32)
    idx[-1, 0, k // 5:k // 2] = -1
    idx[-1, 0, -(k // 4):] = -1
    q = rng.standard_normal((batch, 1, hk * group, dim)).astype(np.float32)
    out, lse = check_attention(ds, q, "fp16", pool, table, lengths, indices=idx)
    again = ds.kv4_attention(dev(q).half(), dev(pool), dev(table), dev(lengths), indices=dev(idx))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("lengths,hk,group,dim", [
    ([20011], 1, 4, 128), ([9000, 3, 0, 5000, 1], 2, 8, 64), ([4099] * 3, 1, 20, 256)])
def test_long_sequences(ds, lengths, hk, group, dim):
    """Sequences that are shared by many CTAs, and their join."""
    rng = np.random.default_rng(len(lengths))
    lengths = np.array(lengths, dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 64, wide=-(-lengths.max() // 64))
    pool = random_pool(rng, n_pages, hk, 64, dim)
    q = rng.standard_normal((len(lengths), 1, hk * group, dim)).astype(np.float32)
    out, lse = check_attention(ds, q, "bf16", pool, table, lengths)
    again = ds.kv4_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])   # a fixed order of sums


@pytest.mark.parametrize("size", [1e-6, 30.0, 3e4])
@pytest.mark.parametrize("scale", [0.01, 1.0, -0.5])
def test_size_of_the_queries(ds, size, scale):
    """Tiny, sharp and enormous scores."""
    rng = np.random.default_rng(3)
    lengths = np.array([70, 300], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=20)
    pool = random_pool(rng, n_pages, 1, 16, 128)
    q = (rng.standard_normal((2, 1, 8, 128)) * size).astype(np.float32)
    q[0, 0, 3] = 0
    q[0, 0, 4, 1:] *= 1e-5          # one large channel beside small ones
    if size * abs(scale) > 100:     # there one token takes everything: compare the choice
        out, _ = ds.kv4_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths), scale=scale)
        ref = model.attention(dev(q).bfloat16().double().cpu().numpy(), pool, table, lengths, scale)[0]
        assert torch.isfinite(out).all()
        near = np.abs(out.double().cpu().numpy() - ref) <= 0.02 * (1 + np.abs(ref))
        assert near.mean() > 0.9    # scores of 1e6 carry errors of about one
        return
    check_attention(ds, q, "bf16", pool, table, lengths, scale=scale)


def test_a_scale_of_zero_is_the_mean(ds):
    rng = np.random.default_rng(4)
    lengths = np.array([45, 7], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=3)
    pool = random_pool(rng, n_pages, 1, 16, 64)
    q = rng.standard_normal((2, 2, 4, 64)).astype(np.float32)
    check_attention(ds, q, "bf16", pool, table, lengths, scale=0.0)


def test_what_is_masked_is_not_read_into_the_result(ds):
    """NaN records past the ends, in free pages and at unlisted positions leave no trace."""
    rng = np.random.default_rng(5)
    lengths = np.array([37, 16, 1, 0], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=4)
    clean = random_pool(rng, n_pages, 2, 16, 128)
    dirty = np.full_like(clean, 0xFF)
    for b, n in enumerate(lengths):
        t = np.arange(n)
        dirty[table[b, t // 16], :, t % 16] = clean[table[b, t // 16], :, t % 16]
    q = rng.standard_normal((4, 1, 4, 128)).astype(np.float32)
    a, b = (check_attention(ds, q, "bf16", p, table, lengths) for p in (clean, dirty))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    idx = np.full((4, 1, 40), -1, dtype=np.int32)
    idx[0, 0, :3], idx[1, 0, 5:8], idx[2, 0, 39] = [36, 37, 0], [15, 16, 3], 0
    a, b = (check_attention(ds, q, "bf16", p, table, lengths, indices=idx) for p in (clean, dirty))
    assert torch.equal(a[0], b[0])


def test_nan_reaches_the_rows_that_see_it_and_no_other(ds):
    rng = np.random.default_rng(6)
    lengths = np.array([40, 40, 40], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=3)
    pool = random_pool(rng, n_pages, 2, 16, 64)
    q = rng.standard_normal((3, 2, 4, 64)).astype(np.float32)
    q[0, 1, 2, 7] = np.nan
    pool[table[1, 0], 1, 3, 64:66] = 0xFF       # a key scale of head 1
    pool[table[2, 2], 0, 7, 68:70] = 0xFF       # a value scale of the newest token, head 0
    out, _ = check_attention(ds, q, "bf16", pool, table, lengths)
    bad = torch.isnan(out).any(-1).cpu().numpy()
    want = np.zeros((3, 2, 4), dtype=bool)
    want[0, 1, 2] = want[1, :, 2:] = want[2, 1, :2] = True
    assert np.array_equal(bad, want)


def test_lengths_sequences_and_pages_out_of_range(ds):
    rng = np.random.default_rng(7)
    table = np.array([[0, 1], [2, -1], [3, 9], [4, 5]], dtype=np.int32)     # 6 pages
    pool = random_pool(rng, 6, 1, 16, 64)
    lengths = np.array([2 ** 31 - 1, 30, 32, -5], dtype=np.int32)
    q = rng.standard_normal((6, 1, 2, 64)).astype(np.float32)
    check_attention(ds, q, "bf16", pool, table, lengths,
                    seqs=np.array([3, 0, 2, 1, -1, 4], dtype=np.int32))


def test_strided_queries_tables_and_pools(ds):
    rng = np.random.default_rng(8)
    lengths = np.array([50, 3], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=4)
    wide_table = dev(np.concatenate((table, np.full((2, 5), 99, np.int32)), 1))[:, :4]
    pool = random_pool(rng, n_pages, 2, 16, 128)
    layers = torch.zeros((n_pages, 3, *pool.shape[1:]), dtype=torch.uint8, device=DEV)
    layers[:, 1] = dev(pool)
    fused = dev(rng.standard_normal((2, 2, 3, 4, 130)).astype(np.float32)).bfloat16()
    for q in (fused[:, :, 1, :, :128], fused[:, :, 1, :, 1:129]):
        plain = ds.kv4_attention(q.contiguous(), dev(pool), dev(table), dev(lengths))
        got = ds.kv4_attention(q, layers[:, 1], wide_table, dev(lengths))
        assert torch.equal(plain[0], got[0]) and torch.equal(plain[1], got[1])


def test_attention_over_the_choice_of_topk(ds):
    """The indices of a top-k call go in as they come out; all of them equals no list."""
    rng = np.random.default_rng(9)
    lengths = np.array([300, 40, 0], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 32, wide=10)
    pool = random_pool(rng, n_pages, 1, 32, 128)
    q = rng.standard_normal((3, 1, 8, 128)).astype(np.float32)
    scores = dev(rng.standard_normal((3, 320)).astype(np.float32))
    idx, _ = ds.topk(scores, 64, 128, 128, row_len=dev(lengths))
    assert (idx[1, 40:] == -1).all() and (idx[2] == -1).all()
    check_attention(ds, q, "bf16", pool, table, lengths, indices=idx.view(3, 1, 64).cpu().numpy())
    idx, _ = ds.topk(scores, 320, 128, 128, row_len=dev(lengths))
    some = ds.kv4_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths),
                            indices=idx.view(3, 1, 320))
    every = ds.kv4_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths))
    assert (some[0].float() - every[0].float()).abs().max() < 2e-2
    none = ds.kv4_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths),
                            indices=idx.view(3, 1, 320)[..., :0].contiguous())
    assert (none[0] == 0).all() and torch.isneginf(none[1]).all()


def test_places_beyond_32_bits(ds):
    """A pool of over 4 GiB whose used pages lie at its end."""
    dim, page, hk = 128, 64, 8
    rec = model.record_bytes(dim)
    n_pages = (5 << 30) // (hk * page * rec)
    pool = torch.zeros((n_pages, hk, page, rec), dtype=torch.uint8, device=DEV)
    table = np.array([[n_pages - 1, n_pages - 3, 1]], dtype=np.int32)
    rng = np.random.default_rng(10)
    k, v = (dev(rng.standard_normal((150, hk, dim)).astype(np.float32)) for _ in range(2))
    seq, pos = dev(np.zeros(150, np.int32)), dev(np.arange(150, dtype=np.int32))
    ds.kv4_append(pool, dev(table), seq, pos, k, v)
    q = rng.standard_normal((1, 1, 8, dim)).astype(np.float32)
    small = pool[torch.from_numpy(table[0].astype(np.int64)).to(DEV)].clone()
    a = ds.kv4_attention(dev(q).half(), pool, dev(table), dev(np.array([150], np.int32)))
    b, _ = check_attention(ds, q, "fp16", small, np.array([[0, 1, 2]], np.int32),
                           np.array([150], np.int32))
    assert torch.equal(a[0], b)
    assert pool[1, 0, :22].any() and not pool[1, 0, 22:].any()


def test_another_stream_and_a_graph(ds):
    rng = np.random.default_rng(11)
    lengths = np.array([700, 90], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, 16, wide=50)
    pool, t, n = dev(random_pool(rng, n_pages, 2, 16, 64)), dev(table), dev(lengths)
    q = dev(rng.standard_normal((2, 1, 8, 64)).astype(np.float32)).bfloat16()
    want = ds.kv4_attention(q, pool, t, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = q * 1
        got = ds.kv4_attention(late, pool, t, n)
    given = ds.kv4_attention(q, pool, t, n, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[0], given[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ds.kv4_attention(q, pool, t, n)
    n.copy_(dev(np.array([3, 800], np.int32)))       # lengths are read when the graph runs
    graph.replay()
    now = ds.kv4_attention(q, pool, t, n)
    torch.cuda.synchronize()
    assert torch.equal(out, now[0]) and torch.equal(lse, now[1])


def test_steps_without_a_wait_between_them(ds):
    """A decode loop enqueued at once equals one that waits after every call: each kernel sees
    what the one before it left (lengths, table, records), though it may start before that ends."""
    def loop(wait):
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        n, hk, dim, page = 5, 2, 64, 16
        i32 = dict(dtype=torch.int32, device=DEV)
        pool = torch.zeros((60, hk, page, 80), dtype=torch.uint8, device=DEV)
        table, lengths = torch.full((n, 12), -1, **i32), torch.zeros(n, **i32)
        refs, seqs = torch.zeros(60, **i32), torch.arange(n, **i32)
        grow = torch.tensor([1, 3, 2, 1, 4], **i32)
        flat = seqs.repeat_interleave(grow.long())
        within = torch.cat([torch.arange(x, **i32) for x in grow.tolist()])
        results = []
        kv = torch.randn((40, len(flat), 2, hk, dim), device=DEV, generator=g).bfloat16()
        q = torch.randn((40, n, 1, 4, dim), device=DEV, generator=g).bfloat16()
        torch.cuda.synchronize()
        done = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(40):
            before = lengths.clone()
            done()
            ds.pages_reserve(table, lengths, refs, seqs, grow, page)
            done()
            ds.kv4_append(pool, table, flat, before[flat.long()] + within, kv[i, :, 0], kv[i, :, 1])
            done()
            results.append(ds.kv4_attention(q[i], pool, table, lengths)[0])
            done()
            if i % 10 == 9:
                ds.pages_free(table, lengths, refs, seqs[i // 10:i // 10 + 1], page)
                done()
                ds.pages_compact(pool[None], table, refs)
                done()
        return torch.stack(results), lengths, pool
    a, b = loop(True), loop(False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_streams_and_threads_do_not_share_a_workspace_at_a_time(ds):
    """Calls without a workspace, from several streams and from several host threads on one."""
    import threading
    rng = np.random.default_rng(12)
    jobs = []
    for i, n in enumerate([9000, 4000, 7000, 12000]):
        lengths = np.array([n], dtype=np.int32)
        table, n_pages = make_table(rng, lengths, 16, wide=-(-n // 16))
        pool, t, size = dev(random_pool(rng, n_pages, 1, 16, 64)), dev(table), dev(lengths)
        q = dev(rng.standard_normal((1, 1, 8, 64)).astype(np.float32)).bfloat16()
        space = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
        jobs.append(((q, pool, t, size), ds.kv4_attention(q, pool, t, size, workspace=space)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]

    def work(job, stream, got):
        with torch.cuda.stream(stream):
            got += [ds.kv4_attention(*job[0]) for _ in range(40)]

    for one in (False, True):
        got = [[] for _ in jobs]
        threads = [threading.Thread(target=work, args=(j, streams[0] if one else s, g))
                   for j, s, g in zip(jobs, streams, got)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for (_, want), results in zip(jobs, got):
            assert len(results) == 40
            assert all(torch.equal(want[0], r[0]) and torch.equal(want[1], r[1]) for r in results)


def test_refusals(ds):
    pool = torch.zeros((4, 2, 16, 144), dtype=torch.uint8, device=DEV)
    table = torch.zeros((3, 4), dtype=torch.int32, device=DEV)
    lengths = torch.zeros(3, dtype=torch.int32, device=DEV)
    q = torch.zeros((3, 1, 4, 128), dtype=torch.bfloat16, device=DEV)
    ok = dict(q=q, pool=pool, table=table, lengths=lengths)
    ds.kv4_attention(**ok)
    for bad in [dict(q=q[0]), dict(q=q.double()), dict(q=q.cpu()), dict(q=q.transpose(2, 3)),
                dict(q=q[..., :64]), dict(pool=pool.view(torch.int8)), dict(pool=pool[..., :128]),
                dict(pool=pool.transpose(1, 2)), dict(table=table.long()), dict(table=table.t()),
                dict(lengths=lengths[:2]), dict(lengths=lengths.cpu()),
                dict(indices=torch.zeros((3, 4), dtype=torch.int32, device=DEV)),
                dict(indices=torch.zeros((3, 1, 4), dtype=torch.int64, device=DEV)),
                dict(out=torch.zeros((3, 1, 4, 128), device=DEV)), dict(lse=q[..., 0]),
                dict(table=table[:1].expand(3, -1)), dict(pool=pool[:1].expand(4, -1, -1, -1)),
                dict(seqs=lengths[:1]), dict(q=torch.cat((q, q)))]:
        with pytest.raises((ValueError, TypeError)):
            ds.kv4_attention(**{**ok, **bad})
    for bad, status in [(dict(q=q.float()), ds.DS_EUNSUPPORTED), (dict(q=q[:, :, :3]), ds.DS_EINVAL)]:
        with pytest.raises(ds.DSError) as e:
            ds.kv4_attention(**{**ok, **bad})
        assert e.value.status == status
    x = torch.zeros((5, 2, 128), device=DEV)
    at = torch.zeros(5, dtype=torch.int32, device=DEV)
    for bad in [dict(k=x[:, :1], v=x[:, :1]), dict(k=x[:4]), dict(v=x.half()), dict(seq=at[:4]),
                dict(pos=at.long()), dict(k=x.cpu(), v=x.cpu()), dict(k=x.double(), v=x.double())]:
        with pytest.raises((ValueError, TypeError)):
            ds.kv4_append(**{**dict(pool=pool, table=table, seq=at, pos=at, k=x, v=x), **bad})
    with pytest.raises(ds.DSError):
        ds.kv4_read(pool, table, at, at, 96, torch.float32)
