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
