"""ds_kv4_chunk_attention answers for its arguments before any CUDA call, and the 64-bit model of
chunks is that of decode attention where they meet (CPU only)."""
import numpy as np
import pytest

import oracle.kv4 as model
import top_selection_deepselect_gb300 as ds
from test_kv4_abi import BAD_CACHES, FAKE, cache, status_of

EINVAL, EUNSUP = ds.DS_EINVAL, ds.DS_EUNSUPPORTED

CALL = dict(lengths=FAKE, seqs=None, starts=FAKE, batch=2, tokens=10, heads=4, dtype=ds.DS_BF16, q=FAKE,
            q_stride=(512, 128), scale=1.0, out=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=None)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ds.build()
    return ds.load_library()


def refuse(c=None, **change):
    return status_of(ds.ds_kv4_chunk_attention, cache=cache() if c is None else c,
                     **{n: change.get(n, v) for n, v in CALL.items()})


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(change, status):
    assert refuse(cache(**change)) == status
    assert status_of(ds.ds_kv4_chunk_attention_workspace, cache(**change), 2, 10, 4) == status


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(heads=0), EINVAL), (dict(heads=5), EINVAL),
    (dict(heads=-2), EINVAL), (dict(tokens=1 << 31), EUNSUP), (dict(tokens=1 << 30), EUNSUP)])
def test_bad_sizes(change, status):
    assert refuse(**change) == status
    sizes = {n: change.get(n, CALL[n]) for n in ("batch", "tokens", "heads")}
    assert status_of(ds.ds_kv4_chunk_attention_workspace, cache(), **sizes) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=ds.DS_FP32), EUNSUP), (dict(dtype=7), EUNSUP), (dict(lengths=None), EINVAL),
    (dict(starts=None), EINVAL), (dict(q=None), EINVAL), (dict(q=FAKE + 1), EINVAL), (dict(out=None), EINVAL),
    (dict(out=FAKE + 8), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL)])
def test_bad_pointers_and_types(change, status):
    assert refuse(**change) == status


def test_tables_that_are_too_long():
    assert refuse(cache(max_pages=1 << 27, table_stride=1 << 27)) == EUNSUP


def test_nothing_to_do():
    assert refuse(batch=0, q=None, out=None) == ds.DS_OK
    assert refuse(tokens=0, workspace=None, workspace_bytes=0) == ds.DS_OK


def test_model_of_chunks_is_that_of_decoding():
    rng = np.random.default_rng(2)
    page, dim, n_pages = 4, 64, 9
    k, v = rng.standard_normal((2, n_pages, 2, page, dim)).astype(np.float32)
    pool = model.encode(k, v)
    table = np.array([[3, 0, -1, 8], [5, 6, 7, 99]], dtype=np.int32)
    lengths = np.array([14, 15], dtype=np.int32)
    q = rng.standard_normal((6, 4, dim))
    out, lse, spread, _ = model.chunk_attention(q, pool, table, lengths, [0, 3, 6], 0.3)
    want = model.attention(q.reshape(2, 3, 4, dim), pool, table, lengths, 0.3)
    for a, b in zip((out, lse, spread), want):
        assert np.allclose(a, np.asarray(b).reshape(a.shape), rtol=1e-12, atol=1e-13)


def test_starts_as_they_are_read():
    assert model.rising([-3, 5, 2, 40], 10).tolist() == [0, 5, 5, 10]
