"""Attention of chunks over the 4-bit paged cache on the GPU against the 64-bit model, within bounds
derived from its roundings."""
import numpy as np
import pytest

import oracle.kv4 as model
from test_gpu_kv4 import DEV, DTYPES, dev, make_table, random_pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as _ds
    _ds.build()
    _ds.load_library()
    return _ds


def check(ds, q, dtype, pool, table, lengths, starts, scale=None, seqs=None, **kw):
    """Runs the chunks and compares with the model.

    Bounds.  The result before its last rounding is within t of the model's, so the output lies
    between the roundings of the model's value minus t and plus t.  A value and a probability are
    rounded to fp16 before they are multiplied: 2^-11 relative each, and absolute 2^-24 of the largest
    value, and for each of n tokens 2^-32 of the largest probability (their sum is at least 1) times
    that value.  Products are exact; a product instruction adds 16 of them to a
    32-bit sum, which may cut each addend off at 2^-22 of the largest: 2 D / 16 <= 32 instructions
    move a score by 2^-17 reach, a probability as much relative, numerator and sum alike; n / 16 move
    the output by n 2^-26 spread.  exp and the sums: 2^-18."""
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    qt = q if isinstance(q, torch.Tensor) else dev(q).to(DTYPES[dtype])
    pool_t = pool if isinstance(pool, torch.Tensor) else dev(pool)
    out, lse = ds.kv4_chunk_attention(qt, pool_t, dev(table), dev(lengths), dev(starts), scale=scale,
                                      seqs=None if seqs is None else dev(seqs), **kw)
    torch.cuda.synchronize()
    host = pool_t.cpu().numpy()
    ref, rlse, spread, reach = model.chunk_attention(qt.double().cpu().numpy(), host, table, lengths, starts,
                                                     float(np.float32(scale)), seqs)
    starts = model.rising(starts, len(qt))
    rows = slice(starts[0], starts[-1])
    got, glse = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    ref, rlse, spread, reach = ref[rows], rlse[rows], spread[rows], reach[rows]
    n = table.shape[1] * host.shape[2]
    u = 2.0 ** -11
    move = 2.0 ** -17 * (1 + reach)
    with np.errstate(invalid="ignore"):
        big = np.abs(model.decode(host, dim)[1])
        big = np.max(np.where(np.isfinite(big), big, 0))
        t = (2 * u + u * u + 2 * move[..., None] + n * 2.0 ** -26) * spread + (n * 2.0 ** -32 + 2.0 ** -24) * big
        lo, hi = (torch.from_numpy(x).to(qt.dtype).double().numpy() for x in (ref - t, ref + t))
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert ((lo <= got) & (got <= hi))[fine].all(), np.nanmax(np.abs(got - ref) / t)
    assert np.array_equal(np.isnan(glse), np.isnan(rlse))
    assert np.array_equal(np.isneginf(glse), np.isneginf(rlse))
    f = np.isfinite(rlse)
    assert (np.abs(glse[f] - rlse[f]) <= (move + 2.0 ** -21 * (1 + np.abs(rlse)))[f]).all()
    return out, lse


def chunk(rng, new, before, heads, hk, dim, page, spread=1.0, wide=0):
    """(q, pool, table, lengths, starts) of sequences with these new tokens after these others."""
    lengths = np.array([n + b for n, b in zip(new, before)], dtype=np.int32)
    table, n_pages = make_table(rng, lengths, page, wide=max(1, max(-(-int(n) // page) for n in lengths)) + wide)
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = rng.standard_normal((int(starts[-1]), heads, dim)).astype(np.float32)
    return q, random_pool(rng, n_pages, hk, page, dim, spread), table, lengths, starts


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,hk,page,new,before", [
    (1, 1, 16, [1], [0]), (4, 1, 16, [33], [0]), (2, 2, 64, [64, 65], [0, 63]), (6, 2, 48, [50, 1, 97], [3, 200, 31]),
    (7, 1, 7, [45], [90]), (8, 1, 1, [16], [130]), (16, 1, 128, [40], [500]), (3, 3, 24, [130, 300], [0, 70])])
def test_chunks(ds, dim, dtype, heads, hk, page, new, before):
    rng = np.random.default_rng(dim + heads * 10 + page)
    check(ds, *chunk_args(rng, new, before, heads, hk, dim, page, dtype))


def chunk_args(rng, new, before, heads, hk, dim, page, dtype, **kw):
    q, pool, table, lengths, starts = chunk(rng, new, before, heads, hk, dim, page, **kw)
    return q, dtype, pool, table, lengths, starts


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_axis_few_rows(ds, dim):
    """One unit over many CTAs, and its parts joined."""
    rng = np.random.default_rng(dim)
    check(ds, *chunk_args(rng, [5, 40], [6001, 2500], 8, 1, dim, 32, "bf16"))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,hk", [(4, 2), (5, 1)])
def test_many_short_sequences(ds, dim, heads, hk):
    """More units than CTAs, several a CTA, one row tile and two in turn, some without a new token,
    some without any."""
    rng = np.random.default_rng(dim + heads)
    new = [0, 1, 60, 2, 0, 130, 7, 64, 0, 3] * 12
    before = [0, 0, 5, 70, 9, 0, 128, 1, 3, 64] * 12
    args = list(chunk_args(rng, new, before, heads, hk, dim, 16, "bf16"))
    args[4] = args[4].copy()
    args[4][3] = 1      # a sequence shorter than its chunk: rows that see nothing
    args[4][6] = 0
    args[4][16] = -5
    check(ds, *args)


def test_more_entries_than_planning_threads(ds):
    """2500 entries, most of them without a new token, over a few sequences."""
    rng = np.random.default_rng(15)
    q, pool, table, lengths, _ = chunk(rng, [40, 50, 60], [30, 90, 0], 2, 1, 64, 16)
    new = np.zeros(2500, dtype=np.int64)
    new[rng.choice(2500, 90, replace=False)] = 1
    new[[3, 1023, 1024, 2047, 2048, 2499]] = 10
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    seqs = rng.integers(0, 3, 2500).astype(np.int32)
    check(ds, q[:starts[-1]] if starts[-1] <= len(q) else np.resize(q, (starts[-1], 2, 64)), "bf16", pool, table,
          lengths, starts, seqs=seqs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_entries_of_any_sequence(ds, dtype):
    """seqs in any order, the same sequence twice, sequences that are none, lengths beyond the table."""
    rng = np.random.default_rng(4)
    q, pool, table, lengths, starts = chunk(rng, [20, 30, 5, 9, 40], [10, 0, 300, 70, 2], 4, 2, 64, 16)
    seqs = np.array([2, 0, 7, -1, 2], dtype=np.int32)
    lengths[0] = 1 << 30
    check(ds, q, dtype, pool, table, lengths, starts, seqs=seqs)


def test_starts_that_fall_and_rows_of_no_entry(ds):
    rng = np.random.default_rng(5)
    q, pool, table, lengths, _ = chunk(rng, [30, 30, 30, 30], [5, 5, 5, 5], 4, 2, 64, 16)
    starts = np.array([7, 30, 12, 50, 1000], dtype=np.int32)
    out = torch.full((120, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((120, 4), 3.0, device=DEV)
    check(ds, q, "bf16", pool, table, lengths, starts, out=out, lse=lse)
    assert (out[:7] == 3).all() and (lse[:7] == 3).all()
    starts = np.array([-9, 10, 20, 30, 90], dtype=np.int32)
    out.fill_(3.0), lse.fill_(3.0)
    check(ds, q, "bf16", pool, table, lengths, starts, out=out, lse=lse)
    assert (out[90:] == 3).all() and (lse[90:] == 3).all() and not (out[:90] == 3).all(-1).any()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_pages_that_are_not_there(ds, dim, dtype):
    """Table entries out of range leave their tokens out, whatever lies in shared memory by then."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, [90, 40], [200, 0], 4, 2, dim, 16)
    pool[-2:] = 0xff                    # pages of no sequence: all scales NaN
    table[0, 2], table[0, 9], table[0, 17] = -1, len(pool), 1 << 30
    table[1, 0] = -7
    check(ds, q, dtype, pool, table, lengths, starts)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_what_is_not_seen_leaves_no_trace(ds, dim, dtype):
    """Tokens whose keys or values are NaN: rows before them do not notice, later ones are NaN in
    the channels that the value's group has, or in all for a key."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, [150, 100], [60, 128], 2, 1, dim, 16)
    nan = np.array([0xff, 0x7f], dtype=np.uint8)

    def poison(seq, pos, which, group):
        at = dim + which * (dim // 16) + 2 * group
        pool[table[seq, pos // 16], 0, pos % 16, at:at + 2] = nan

    poison(0, 100, 1, 0)
    poison(0, 131, 1, dim // 32 - 1)
    poison(0, 170, 0, 1)
    poison(1, 3, 1, 1)                  # seen by every row
    poison(1, 227, 1, 0)                # by the last one
    out, _ = check(ds, q, dtype, pool, table, lengths, starts)
    assert torch.isfinite(out[:40].float()).all() and torch.isnan(out[41, :, :32].float()).all()
    # free slots behind the last token hold NaN too
    pool[table[0, 13], 0, 3:] = 0xff
    pool[table[0, 13], 0, 2] = pool[table[0, 13], 0, 1]
    check(ds, q, dtype, pool, table, lengths, starts)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_that_are_no_numbers(ds, dtype):
    rng = np.random.default_rng(6)
    q, pool, table, lengths, starts = chunk(rng, [140], [20], 2, 1, 64, 16)
    q[5, 0, 3], q[17, 1, 60], q[139, 0, 0] = np.nan, np.inf, -np.inf
    qt = dev(q).to(DTYPES[dtype])
    out, lse = ds.kv4_chunk_attention(qt, dev(pool), dev(table), dev(lengths), dev(starts))
    bad = torch.isnan(out.float()).all(-1)
    want = torch.zeros_like(bad)
    want[5, 0] = want[17, 1] = want[139, 0] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(out.float()).any(-1), want)
    clean = torch.where(torch.isfinite(qt), qt, torch.zeros_like(qt))
    other, olse = ds.kv4_chunk_attention(clean, dev(pool), dev(table), dev(lengths), dev(starts))
    assert torch.equal(out[~want], other[~want]) and torch.equal(lse[~want], olse[~want])


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-4, 1e-38])
def test_scale(ds, scale):
    rng = np.random.default_rng(7)
    check(ds, *chunk_args(rng, [70], [100], 4, 2, 64, 16, "bf16"), scale=scale)
    check(ds, *chunk_args(rng, [70], [100], 2, 1, 256, 16, "fp16"), scale=scale)


def test_no_scale_is_even_attention(ds):
    """Scores of any size times 0 are 0, and times the smallest numbers what they are."""
    rng = np.random.default_rng(16)
    q, pool, table, lengths, starts = chunk(rng, [70], [100], 2, 1, 64, 16, spread=1e4)
    for scale in (0.0, 1e-40, -1e-36):
        check(ds, q * np.float32(1e30), "bf16", pool, table, lengths, starts, scale=scale)


@pytest.mark.parametrize("dtype,spread", [("bf16", 1e-30), ("bf16", 1e-6), ("bf16", 1e4), ("fp16", 1e-3), ("fp16", 2e3),
                                          ("fp16", 1e-6)])
def test_values_of_every_size(ds, dtype, spread):
    """Keys and values far from 1, queries so that scores are not."""
    rng = np.random.default_rng(8)
    q, pool, table, lengths, starts = chunk(rng, [40, 90], [100, 0], 4, 2, 64, 16, spread=spread)
    scale = 0.125 / max(spread, 1e-5)
    check(ds, q, dtype, pool, table, lengths, starts, scale=scale)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_that_grow_and_fall(ds, dim, dtype):
    """Value scales from one end of their range to the other within a sequence: small ones first, so
    that what is held of them has to make room, then large ones first."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, [70, 140], [450, 450], 2, 1, dim, 16)
    for seq in range(2):
        size = np.exp2(np.linspace(-24, 12, int(lengths[seq])))
        k, v = rng.standard_normal((2, 1, int(lengths[seq]), dim)).astype(np.float32)
        v *= (size if seq == 0 else size[::-1])[:, None].astype(np.float32)
        rec = model.encode(k[0], v[0])
        for pos in range(int(lengths[seq])):
            pool[table[seq, pos // 16], 0, pos % 16] = rec[pos]
    check(ds, q, dtype, pool, table, lengths, starts)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_of_either_sign_and_every_code(ds, dim, dtype):
    """Records that kv4_append does not make: any codes, scales below 0, 0, subnormal and the smallest."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, [80, 130], [70, 0], 2, 1, dim, 16)
    pool = rng.integers(0, 256, pool.shape, dtype=np.uint8)
    n = dim // 32
    scales = (rng.standard_normal((*pool.shape[:-1], 2 * n)) * 0.2).astype(np.float16)
    scales[rng.random(scales.shape) < 0.1] = 0
    scales[rng.random(scales.shape) < 0.1] *= np.float16(2.0 ** -14)
    pool[..., dim:dim + 4 * n] = scales.view(np.uint8)
    check(ds, q, dtype, pool, table, lengths, starts)


def test_growing_scores(ds):
    """Each tile's largest score is well above the last one's, so that outputs are scaled again and again."""
    rng = np.random.default_rng(9)
    for dim, dtype in ((64, "bf16"), (128, "fp16"), (256, "bf16")):
        q, _, table, lengths, starts = chunk(rng, [130], [700], 2, 1, dim, 64)
        k = rng.standard_normal((len(table[0]) + 2, 1, 64, dim)).astype(np.float32) * 0.1
        v = rng.standard_normal(k.shape).astype(np.float32)
        for i, page in enumerate(table[0]):
            k[page] += 0.25 * (i + 1)
        q = np.abs(q)
        check(ds, q, dtype, model.encode(k, v), table, lengths, starts, scale=0.5)


@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 0), (3, 5), (8, 8), (0, 24)])
def test_strided_queries(ds, offset, gap):
    rng = np.random.default_rng(offset + gap)
    heads, dim = 4, 64
    q, pool, table, lengths, starts = chunk(rng, [30, 50], [10, 0], heads, 2, dim, 16)
    wide = torch.full((80 * heads * (dim + gap) + 64,), float("nan"), dtype=torch.bfloat16, device=DEV)
    qt = wide.as_strided(q.shape, (heads * (dim + gap), dim + gap, 1), offset)
    qt.copy_(dev(q))
    check(ds, qt, "bf16", pool, table, lengths, starts)


def test_pools_of_more_than_32_bits(ds):
    """Pages whose bytes start beyond 2^32, in a pool with gaps between its pages."""
    rng = np.random.default_rng(10)
    q, pool, table, lengths, starts = chunk(rng, [60], [100], 4, 2, 128, 32)
    n_pages, page = len(pool), pool[0].size
    room = torch.zeros((n_pages - 1) * (1 << 30) + page, dtype=torch.uint8, device=DEV)
    far = room.as_strided(pool.shape, (1 << 30, *dev(pool[:1]).stride()[1:]))
    far.copy_(dev(pool))
    a = ds.kv4_chunk_attention(dev(q).bfloat16(), far, dev(table), dev(lengths), dev(starts))
    b = ds.kv4_chunk_attention(dev(q).bfloat16(), dev(pool), dev(table), dev(lengths), dev(starts))
    assert (n_pages - 1) * (1 << 30) > 1 << 32
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_agrees_with_decode_attention(ds):
    """A chunk of as many tokens for each sequence is what kv4_attention does with `queries`."""
    rng = np.random.default_rng(11)
    q, pool, table, lengths, starts = chunk(rng, [4, 4, 4], [900, 33, 0], 16, 2, 128, 64)
    qt = dev(q).half()
    out, lse = check(ds, qt, "fp16", pool, table, lengths, starts)
    other, olse = ds.kv4_attention(qt.view(3, 4, 16, 128), dev(pool), dev(table), dev(lengths))
    assert (lse - olse.view(12, 16)).abs().max() < 2.0 ** -16
    assert (out.float() - other.view(12, 16, 128).float()).abs().max() < 2.0 ** -8


def test_graphs_streams_and_workspaces(ds):
    rng = np.random.default_rng(12)
    q, pool, table, lengths, starts = chunk(rng, [300, 20], [900, 4000], 8, 2, 128, 64)
    args = [dev(q).bfloat16(), dev(pool), dev(table), dev(lengths), dev(starts)]
    want = ds.kv4_chunk_attention(*args)
    # a workspace full of anything, exactly as large as asked for; results do not depend on the run
    size = ds.ds_kv4_chunk_attention_workspace(
        ds.ds_kv4_cache_t(args[1].data_ptr(), args[1].stride(0), args[2].data_ptr(), args[2].stride(0), len(pool),
                          64, 2, 128, *table.shape), 2, 320, 8)
    space = torch.full((size + 256,), 0xff, dtype=torch.uint8, device=DEV)
    got = ds.kv4_chunk_attention(*args, workspace=space[:size])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (space[size:] == 0xff).all()
    with pytest.raises(ValueError):
        ds.kv4_chunk_attention(*args, workspace=space[:size - 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ds.kv4_chunk_attention(*args, stream=side)
    again = ds.kv4_chunk_attention(*args)
    torch.cuda.synchronize()
    for x in (got, again):
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.kv4_chunk_attention(*args, out=out, lse=lse)
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    args[3].fill_(200), args[4].copy_(dev(np.array([0, 20, 320], dtype=np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    want = ds.kv4_chunk_attention(*args)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_nothing_to_do(ds):
    rng = np.random.default_rng(13)
    q, pool, table, lengths, starts = chunk(rng, [5], [5], 2, 1, 64, 16)
    pool_t, table_t, len_t = dev(pool), dev(table), dev(lengths)
    out, lse = ds.kv4_chunk_attention(dev(q[:0]).half(), pool_t, table_t, len_t, dev(starts[:1] * 0))
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out = torch.full((5, 2, 64), 2.0, dtype=torch.float16, device=DEV)
    ds.kv4_chunk_attention(dev(q).half(), pool_t, table_t, len_t, dev(np.zeros(1, dtype=np.int32)), out=out)
    ds.kv4_chunk_attention(dev(q).half(), pool_t, table_t, len_t, dev(np.zeros(2, dtype=np.int32)), out=out)
    assert (out == 2).all()


def test_refusals(ds):
    rng = np.random.default_rng(14)
    q, pool, table, lengths, starts = chunk(rng, [5], [5], 2, 1, 64, 16)
    q, pool, table, lengths, starts = dev(q).half(), dev(pool), dev(table), dev(lengths), dev(starts)
    call = ds.kv4_chunk_attention
    for bad in (lambda: call(q.cpu(), pool, table, lengths, starts), lambda: call(q[0], pool, table, lengths, starts),
                lambda: call(q.transpose(1, 2), pool, table, lengths, starts),
                lambda: call(q, pool, table, lengths, starts.long()),
                lambda: call(q, pool, table, lengths, starts[None]),
                lambda: call(q, pool, table, lengths, starts[:0]),
                lambda: call(q, pool, table, lengths[:0], starts),
                lambda: call(q, pool, table, lengths, torch.cat((starts, starts))),
                lambda: call(q, pool, table, lengths, starts, seqs=torch.zeros(3, dtype=torch.int32, device=DEV)),
                lambda: call(q, pool, table, lengths, starts, out=q[:4]),
                lambda: call(q, pool, table, lengths, starts, lse=torch.zeros((5, 2), device=DEV).half()),
                lambda: call(q[..., :32], pool, table, lengths, starts)):
        with pytest.raises((ValueError, ds.DSError)):
            bad()
    with pytest.raises(ds.DSError):
        call(q.float(), pool, table, lengths, starts)
    with pytest.raises(ds.DSError):
        call(torch.cat((q, q), 1)[:, :3], pool.repeat(1, 2, 1, 1), table, lengths, starts)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,before", [([3, 70, 1], [0, 40, 0]), ([5, 2], [6001, 130])])
def test_infinite_queries_whose_scores_have_one_sign(ds, dim, dtype, new, before):
    """Every key's channel is 7 (1 + 2^-10), or -8 times that, whose parts both have its sign: an
    infinite channel of a query makes all scores -inf, of one token or of thousands and over
    several CTAs, and no NaN comes up by itself.  Rows that see a token are NaN, others are not."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, new, before, 4, 2, dim, 16)
    n = dim // 32
    pool[:, 0, :, :dim // 2], pool[:, 1, :, :dim // 2] = 0xff, 0x00
    pool[..., dim:dim + 2 * n] = np.full(n, 0x3c01, dtype=np.uint16).view(np.uint8)
    q[0, 0, 3], q[1, 1, dim - 1], q[-1, 2, 5] = -np.inf, -np.inf, np.inf
    q[2, 0, 7], q[2, 3, 1] = np.inf, -np.inf
    out, lse = check(ds, q, dtype, pool, table, lengths, starts)
    assert torch.isnan(out[0, 0].float()).all() and torch.isnan(lse[-1, 2])
    # the tokens that such a row sees are not there: it sees nothing
    table = table.copy()
    table[:, 0] = -1
    if before[0] == 0:
        out, lse = check(ds, q, dtype, pool, table, lengths, starts)
        assert (out[:3] == 0).all() and (lse[:3] == -float("inf")).all()
    else:
        table[0, :] = len(pool)
        out, lse = check(ds, q, dtype, pool, table, lengths, starts)
        assert (out[:5] == 0).all() and (lse[:5] == -float("inf")).all()
        table[0, 200] = 0               # one page of all
        out, lse = check(ds, q, dtype, pool, table, lengths, starts)
        assert torch.isnan(out[0, 0].float()).all() and torch.isnan(lse[1, 1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("most", [65504.0, 9000.0])
def test_keys_beyond_16_bits(ds, dim, dtype, most):
    """Key scales of either sign up to fp16's largest, with any codes: channels up to 2^19.  Most of
    them, one in thirty, and one group of one token.  (With bf16 queries scales are exact up to
    64640.)"""
    rng = np.random.default_rng(dim)
    most = min(most, 64640.0) if dtype == "bf16" else most
    q, pool, table, lengths, starts = chunk(rng, [80, 130, 9], [70, 0, 300], 2, 1, dim, 16)
    n = dim // 32
    pool[..., :dim // 2] = rng.integers(0, 256, (*pool.shape[:-1], dim // 2), dtype=np.uint8)
    plain = pool.copy()
    for some in (0.7, 1 / 30):
        scales = (rng.standard_normal((*pool.shape[:-1], n)) * 0.2).astype(np.float16)
        large = rng.random(scales.shape) < some
        scales[large] = rng.choice([-1.0, 1.0], large.sum()) * np.exp2(rng.uniform(11, np.log2(most), large.sum()))
        scales[0, 0, :8, 0], scales[1, 0, :8, n - 1] = most, -most
        pool[..., dim:dim + 2 * n] = scales.view(np.uint8)
        for scale in (1e-6, 1e-4):
            check(ds, q, dtype, pool, table, lengths, starts, scale=scale)
    pool = plain
    pool[table[2, 18], 0, 3, dim:dim + 2] = np.array([most], dtype=np.float16).view(np.uint8)
    check(ds, q, dtype, pool, table, lengths, starts, scale=1e-5)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits", [0x7c00, 0xfc00, 0x7fff, 0xffff, 0x7e00])
def test_key_scales_that_are_no_numbers(ds, dim, dtype, bits):
    """An infinite scale is as good as a NaN: rows that see it are NaN, rows before it are not."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, [90], [30], 2, 1, dim, 16)
    clean = check(ds, q, dtype, pool, table, lengths, starts)
    at = dim + 2 * (dim // 32 - 1)
    pool[table[0, 4], 0, 6, at:at + 2] = np.array([bits], dtype=np.uint16).view(np.uint8)      # token 70
    out, lse = ds.kv4_chunk_attention(dev(q).to(DTYPES[dtype]), dev(pool), dev(table), dev(lengths), dev(starts))
    assert torch.isnan(out[40:].float()).all() and torch.isnan(lse[40:]).all()
    assert torch.equal(out[:40], clean[0][:40]) and torch.equal(lse[:40], clean[1][:40])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [2.0 ** 8, 2.0 ** 10, 2.0 ** 12, 2.0 ** 14, 2.0 ** 18, 2.0 ** 21, -2.0 ** 23, 2.0 ** 30,
                                   2.0 ** 90, 3e38])
@pytest.mark.parametrize("new,before", [([40, 3], [300, 4001]), ([4, 30], [2900, 0])])
def test_scores_far_from_zero(ds, dim, dtype, scale, new, before):
    """Scores of up to 2^13 times scales up to the largest, whose products round to 2^100 and are
    beyond 32 bits at last.  Queries have one channel and key scales are 1, so that scores are
    exact: they differ by 2^10 times the scale, and a row's output is the mean of the values of
    its largest scores' tokens.  Half of the rows' scores grow along the sequence from far below 0,
    or fall; long sequences are many CTAs'.

    Bounds: the weights of these tokens are equal, so that their mean is off by one weight's
    rounding 2^-11, the values' 2^-11 and the sums' 2^-18; lse by 2^-21 of it."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, new, before, 4, 1, dim, 16)
    n = dim // 32
    q[:] = 0
    rows = np.arange(len(q))
    q[:, 0, 5], q[:, 1, 5], q[:, 2, dim - 2], q[:, 3, dim - 2] = 1024, -1024, 1024, -1024
    places = model.channel_places(dim)[0]
    codes = rng.integers(0, 16, (*pool.shape[:-1], dim))
    for seq, (a, b) in enumerate(((5, dim - 2), (dim - 2, 5))):
        pos = np.arange(lengths[seq])
        for channel, rising in ((a, True), (b, False)):
            c = pos * 15 // lengths[seq] if rising else rng.integers(0, 16, len(pos))
            codes[table[seq, pos // 16], 0, pos % 16, places[channel]] = c
    pool[..., :dim // 2] = codes[..., 0::2] | codes[..., 1::2] << 4
    pool[..., dim:dim + 2 * n] = np.ones(n, dtype=np.float16).view(np.uint8)
    qt = dev(q).to(DTYPES[dtype])
    out, lse = ds.kv4_chunk_attention(qt, dev(pool), dev(table), dev(lengths), dev(starts), scale=scale)
    ref, rlse, spread, _ = model.chunk_attention(qt.double().cpu().numpy(), pool, table, lengths, starts,
                                                 float(np.float32(scale)))
    t = (2.0 ** -10 + 2.0 ** -18) * spread + 2.0 ** -24 * 8
    lo, hi = (torch.from_numpy(x).to(qt.dtype).double().numpy() for x in (ref - t, ref + t))
    got = out.double().cpu().numpy()
    assert ((lo <= got) & (got <= hi)).all()
    with np.errstate(over="ignore"):
        wide = rlse.astype(np.float32)
    glse = lse.cpu().numpy()
    f = np.isfinite(wide)
    assert np.array_equal(glse[~f], wide[~f])
    assert (np.abs(glse[f].astype(np.float64) - rlse[f]) <= 2.0 ** -21 * (1 + np.abs(rlse[f]))).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,before", [([90], [30]), ([20], [100]), ([130], [0])])
def test_weights_of_fp16_queries_hold_22_bits(ds, dim, new, before):
    """Values that fp16 holds (codes times a power of two), in pairs that nearly cancel: an output
    is a difference of weights.  What is left of its bound is 2^-22 of a weight, the sums' cut-offs
    and the scores' (as in `check`; scores are small here).  With weights of 11 bits the 64-bit
    model itself is outside it."""
    rng = np.random.default_rng(dim)
    q, pool, table, lengths, starts = chunk(rng, new, before, 2, 1, dim, 16)
    n = dim // 32
    pos = np.arange(lengths[0])
    codes = np.where(pos % 2 == 0, 0xff, 0x11).astype(np.uint8)            # 15 and 1: 7 and -7
    pool[table[0, pos // 16], 0, pos % 16, dim // 2:dim] = codes[:, None]
    pool[..., dim + 2 * n:dim + 4 * n] = np.ones(n, dtype=np.float16).view(np.uint8)
    qt = (dev(q) * 0.25).half()
    scale = dim ** -0.5 * 0.125
    out, _ = ds.kv4_chunk_attention(qt, dev(pool), dev(table), dev(lengths), dev(starts), scale=scale)
    x = qt.double().cpu().numpy()
    ref, _, spread, reach = model.chunk_attention(x, pool, table, lengths, starts, float(np.float32(scale)))
    t = (2.0 ** -22 + 2 * 2.0 ** -17 * reach[..., None] + 2.0 ** -18 + lengths[0] * 2.0 ** -26) * spread
    lo, hi = (torch.from_numpy(y).half().double().numpy() for y in (ref - t, ref + t))
    got = out.double().cpu().numpy()
    assert ((lo <= got) & (got <= hi)).all(), np.max(np.abs(got - ref) / t)
    # the mistake, in the model
    k, v = model.decode(pool[table[0, pos // 16], 0, pos % 16], dim)
    coarse = np.zeros_like(ref)
    for j in range(len(x)):
        see = lengths[0] - len(x) + 1 + j
        w = np.exp(float(np.float32(scale)) * (x[j] @ k[:see].T))
        coarse[j] = w.astype(np.float16).astype(np.float64) @ v[:see] / w.sum(-1, keepdims=True)
    assert not ((lo <= coarse) & (coarse <= hi)).all()
