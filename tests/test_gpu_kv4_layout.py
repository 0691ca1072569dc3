"""How attention over the 4-bit cache lays its work out, where that can be seen or can go wrong."""
import numpy as np
import pytest

import oracle.kv4 as model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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


def shared_pages(rng, batch, length, hk, page, dim):
    """A pool of one sequence's pages and a table whose rows hold them in orders of their own."""
    n = -(-length // page)
    k, v = rng.standard_normal((2, n, hk, page, dim)).astype(np.float32)
    return model.encode(k, v), np.array([rng.permutation(n) for _ in range(batch)], dtype=np.int32)


def bound(ref, spread, reach, n):
    """What the output may be off by before its rounding: 2^-11 of a weight (or 2^-36 of scales
    of about 1 for n tokens' codes), scores and sums in 32 bits (2^-18 of their terms' sizes)."""
    move = 2.0 ** -18 * (1 + reach)
    return (2.0 ** -11 + 2 * move[..., None]) * spread + n * 2.0 ** -36


def within(got, ref, t):
    lo, hi = (torch.from_numpy(x).to(got.dtype).double().numpy() for x in (ref - t, ref + t))
    return bool(((lo <= got.double().cpu().numpy()) & (got.double().cpu().numpy() <= hi)).all())


@pytest.mark.parametrize("dim,group,k,slots", [(128, 8, 1024, 2), (128, 4, 513, 2), (64, 8, 1000, 2),
                                               (256, 16, 500, 1), (128, 16, 1400, 1)])
@pytest.mark.parametrize("more", [1.02, 1.4])
def test_listed_units_between_one_wave_and_two_are_cut(ds, dim, group, k, slots, more):
    """A little more units than CTAs: they are cut between no more CTAs than the GPU holds
    (`slots` an SM), which the workspace's size shows, and joined."""
    rng = np.random.default_rng(dim + k)
    hk, page = 4, 64
    ctas = slots * torch.cuda.get_device_properties(0).multi_processor_count
    batch = -(-int(ctas * more) // hk)
    pool, table = shared_pages(rng, batch, 1500, hk, page, dim)
    cache = ds.ds_kv4_cache_t(1 << 20, pool[0].size, 1 << 20, table.shape[1], len(pool), page, hk, dim, batch,
                              table.shape[1])
    rows = 8 if group <= 8 else 16
    each = 16 + 2 * rows * (dim + 2) * 4       # a record of the unit and two partial results
    assert ds.ds_kv4_attention_workspace(cache, batch, 1, hk * group, k) == ctas * each
    lengths = np.full(batch, 1500, dtype=np.int32)
    lengths[1], lengths[2] = 0, 70
    idx = np.array([rng.permutation(1500)[:k] for _ in range(batch)], dtype=np.int32)[:, None]
    idx[-1, 0, ::3] = -1
    q = dev(rng.standard_normal((batch, 1, hk * group, dim)).astype(np.float32)).bfloat16()
    out, lse = ds.kv4_attention(q, dev(pool), dev(table), dev(lengths), indices=dev(idx))
    some = np.array([0, 1, 2, batch // 2, batch - 2, batch - 1], dtype=np.int32)
    ref, rlse, spread, reach = model.attention(q[some].double().cpu().numpy(), pool, table, lengths, dim ** -0.5,
                                               idx[some], some)
    assert within(out[some], ref, bound(ref, spread, reach, k))
    assert np.allclose(lse[some].cpu().numpy(), rlse, rtol=0, atol=1e-4)


# Warps of a CTA and tokens of a tile, by head dimension and rows of a unit.
WARPS = {(64, 8): 8, (128, 8): 8, (256, 8): 12, (64, 16): 8, (128, 16): 12, (256, 16): 8}
TILE = {64: 32, 128: 32, 256: 16}


def check_some(ds, q, pool, table, lengths, indices=None, pairs=((0, 0), (1, 2), (-1, -1))):
    """Attention against the model for some (sequence, key/value head) pairs, twice."""
    dim, group, hk = q.shape[3], q.shape[2] // pool.shape[1], pool.shape[1]
    args = (q, dev(pool), dev(table), dev(lengths))
    at = None if indices is None else dev(indices)
    out, lse = ds.kv4_attention(*args, indices=at)
    again = ds.kv4_attention(*args, indices=at)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b, g in pairs:
        b, g = b % len(q), g % hk
        rows = slice(g * group, (g + 1) * group)
        one = np.array([b], dtype=np.int32)
        ref, rlse, spread, reach = model.attention(
            q[b:b + 1, :, rows].double().cpu().numpy(), pool[:, g:g + 1], table, lengths, dim ** -0.5,
            None if indices is None else indices[b:b + 1], one)
        n = int(lengths[b]) if indices is None else indices.shape[2]
        assert within(out[b:b + 1, :, rows], ref, bound(ref, spread, reach, n)), (b, g)
        assert np.allclose(lse[b:b + 1, :, rows].cpu().numpy(), rlse, rtol=0, atol=1e-4)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [3, 16])
@pytest.mark.parametrize("page", [16, 48, 64, 7])
def test_long_units_within_a_cta(ds, dim, group, page):
    """So many long units that a warp takes dozens of a unit's tiles: its ring of copies goes round,
    and pages are looked up again, many times."""
    rng = np.random.default_rng(dim + group + page)
    batch, hk = 48, 8
    tile, warps = TILE[dim], WARPS[dim, 8 if group <= 8 else 16]
    longest = 2 * 40 * tile * warps + 11          # half of a unit: 40 tiles a warp, above 32 and any ring
    lengths = rng.integers(longest // 2, longest, batch).astype(np.int32)
    lengths[0], lengths[1], lengths[-1] = longest, longest - tile * warps, longest - 1
    assert batch * hk >= 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pool, table = shared_pages(rng, batch, longest, hk, page, dim)
    q = dev(rng.standard_normal((batch, 1, hk * group, dim)).astype(np.float32)).bfloat16()
    check_some(ds, q, pool, table, lengths)


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 8), (256, 2), (128, 16)])
def test_long_lists_within_a_cta(ds, dim, group):
    rng = np.random.default_rng(dim + group)
    batch, hk, page = 48, 8, 64
    k = 40 * TILE[dim] * WARPS[dim, 8 if group <= 8 else 16] + 5
    length = k + k // 3
    pool, table = shared_pages(rng, batch, length, hk, page, dim)
    lengths = np.full(batch, length, dtype=np.int32)
    lengths[1] = length // 2
    idx = rng.integers(0, length, (batch, 1, k)).astype(np.int32)
    idx[-1, 0, k // 3:k // 2] = -1
    q = dev(rng.standard_normal((batch, 1, hk * group, dim)).astype(np.float32)).bfloat16()
    check_some(ds, q, pool, table, lengths, idx)


@pytest.mark.parametrize("dim,group", [(64, 8), (128, 8), (256, 8)])
def test_long_drafts_within_a_cta(ds, dim, group):
    """Three queries: units of 16 rows, the last of 8, with limits of their own."""
    rng = np.random.default_rng(dim)
    batch, hk, page = 24, 8, 32
    longest = 2 * 40 * TILE[dim] * WARPS[dim, 16] + 3
    lengths = rng.integers(longest // 2, longest, batch).astype(np.int32)
    lengths[0], lengths[1], lengths[-1] = longest, 1, longest - 2
    pool, table = shared_pages(rng, batch, longest, hk, page, dim)
    q = dev(rng.standard_normal((batch, 3, hk * group, dim)).astype(np.float32)).half()
    check_some(ds, q, pool, table, lengths)
