"""include/ds_kv4.h: declared and exported functions agree, argument checks
answer before any CUDA call, and the 64-bit model of the records is sound
(CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest

import oracle.kv4 as model
import top_selection_deepselect_gb300 as ds

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: these calls fail their checks first
EINVAL, EUNSUP = ds.DS_EINVAL, ds.DS_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load_library()


def test_header_and_binding_agree(lib):
    with open(os.path.join(ROOT, "include", "ds_kv4.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ds_\w+)\s*\(", text, flags=re.M)
    assert sorted(set(names)) == sorted(ds.KV4_ENTRY_POINTS)
    for name in names:
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
        assert callable(getattr(ds, name))


@pytest.mark.parametrize("dim,size", [(64, 80), (128, 144), (256, 288)])
def test_record_bytes(dim, size):
    assert ds.kv4_record_bytes(dim) == size == model.record_bytes(dim)


@pytest.mark.parametrize("dim", [0, -64, 32, 96, 512])
def test_record_bytes_refuses_other_dimensions(dim):
    with pytest.raises(ds.DSError) as e:
        ds.kv4_record_bytes(dim)
    assert e.value.status == EUNSUP


def cache(**kw):
    a = dict(pool=FAKE, page_stride=2 * 16 * 144, table=FAKE, table_stride=8, n_pages=4,
             page_size=16, kv_heads=2, head_dim=128, max_seqs=3, max_pages=8)
    a.update(kw)
    return ds.ds_kv4_cache_t(*[a[name] for name, _ in ds.ds_kv4_cache_t._fields_])


def test_packed_descriptors_are_the_structures():
    """The byte strings that the torch wrappers pass have the structures' layout."""
    from top_selection_deepselect_gb300 import _kv4
    for pack, kind in [(_kv4._pack_cache, ds.ds_kv4_cache_t), (_kv4._pack_pool, ds.ds_page_pool_t),
                       (_kv4._pack_book, ds.ds_page_book_t)]:
        values = [1000 + i for i in range(len(kind._fields_))]
        assert pack(*values) == bytes(kind(*values))


BAD_CACHES = [
    (dict(pool=None), EINVAL), (dict(pool=FAKE + 8), EINVAL), (dict(table=None), EINVAL),
    (dict(page_stride=2 * 16 * 144 - 16), EINVAL), (dict(page_stride=2 * 16 * 144 + 8), EINVAL),
    (dict(table_stride=7), EINVAL), (dict(n_pages=0), EINVAL), (dict(page_size=0), EINVAL),
    (dict(kv_heads=0), EINVAL), (dict(max_seqs=0), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(head_dim=96), EUNSUP),
    (dict(n_pages=1 << 16, page_size=1 << 15, page_stride=2 * 144 << 15), EINVAL),
]


def status_of(call, *a, **kw):
    try:
        call(*a, **kw)
    except ds.DSError as e:
        assert ds.ds_last_error_detail()
        return e.status
    return ds.DS_OK


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_checks(lib, kw, status):
    c = cache(**kw)
    s2 = (256, 128)
    assert status_of(ds.ds_kv4_append, c, FAKE, FAKE, 1, 1, FAKE, s2, FAKE, s2, None) == status
    assert status_of(ds.ds_kv4_read, c, FAKE, FAKE, 1, 1, FAKE, FAKE, None) == status
    assert status_of(ds.ds_kv4_attention, c, FAKE, None, 1, 1, 2, 1, FAKE, (1, 1, 1), None, 0, 1.0,
                     FAKE, None, FAKE, 1 << 30, None) == status
    assert status_of(ds.ds_kv4_attention_workspace, c, 1, 1, 2, 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), EINVAL), (dict(tokens=1 << 31), EUNSUP), (dict(seq=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
    (dict(dtype=3), EUNSUP), (dict(k=FAKE + 1), EINVAL), (dict(tokens=0, k=None, v=None), ds.DS_OK)])
def test_append_checks(lib, kw, status):
    a = dict(seq=FAKE, pos=FAKE, tokens=4, dtype=ds.DS_BF16, k=FAKE, v=FAKE)
    a.update(kw)
    assert status_of(ds.ds_kv4_append, cache(), a["seq"], a["pos"], a["tokens"], a["dtype"], a["k"],
                     (256, 128), a["v"], (256, 128), None) == status
    if kw.get("k") != FAKE + 1:
        assert status_of(ds.ds_kv4_read, cache(), a["seq"], a["pos"], a["tokens"], a["dtype"],
                         a["k"], a["v"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), EINVAL), (dict(queries=-1), EINVAL), (dict(heads=0), EINVAL),
    (dict(heads=3), EINVAL), (dict(k=-1), EINVAL), (dict(k=4), EINVAL),
    (dict(indices=FAKE, k=0), EINVAL), (dict(dtype=ds.DS_FP32), EUNSUP), (dict(dtype=9), EUNSUP),
    (dict(lengths=None), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL),
    (dict(q=FAKE + 1), EINVAL), (dict(out=FAKE + 2), EINVAL), (dict(batch=1 << 30, queries=4), EUNSUP),
    (dict(batch=0, q=None, out=None), ds.DS_OK), (dict(queries=0), ds.DS_OK)])
def test_attention_checks(lib, kw, status):
    a = dict(lengths=FAKE, batch=2, queries=1, heads=4, dtype=ds.DS_BF16, q=FAKE, indices=None, k=0,
             out=FAKE)
    a.update(kw)
    assert status_of(ds.ds_kv4_attention, cache(), a["lengths"], None, a["batch"], a["queries"],
                     a["heads"], a["dtype"], a["q"], (512, 512, 128), a["indices"], a["k"], 1.0,
                     a["out"], None, FAKE, 1 << 40, None) == status


def pool(**kw):
    a = dict(pool=FAKE, layer_stride=4096, page_stride=1024, page_bytes=1024, layers=2, n_pages=4)
    a.update(kw)
    return ds.ds_page_pool_t(*[a[name] for name, _ in ds.ds_page_pool_t._fields_])


def book(**kw):
    a = dict(table=FAKE, table_stride=8, lengths=FAKE, refs=FAKE, max_seqs=3, max_pages=8,
             page_size=16, n_pages=4)
    a.update(kw)
    return ds.ds_page_book_t(*[a[name] for name, _ in ds.ds_page_book_t._fields_])


@pytest.mark.parametrize("kw", [
    dict(pool=None), dict(pool=FAKE + 4), dict(layer_stride=8), dict(page_stride=1008),
    dict(page_stride=1032), dict(page_bytes=0), dict(page_bytes=24), dict(layers=0), dict(n_pages=0)])
def test_pool_checks(lib, kw):
    p = pool(**kw)
    assert status_of(ds.ds_pages_copy, p, FAKE, FAKE, 1, None) == EINVAL
    assert status_of(ds.ds_pages_fork, p, book(), FAKE, FAKE, 1, FAKE, FAKE, 4096, None) == EINVAL
    assert status_of(ds.ds_pages_compact, p, book(), FAKE, FAKE, FAKE, 4096, None) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(refs=None), dict(lengths=None), dict(table_stride=7), dict(max_seqs=0),
    dict(max_pages=0), dict(page_size=0), dict(n_pages=0), dict(max_pages=1 << 20, page_size=1 << 11,
                                                               table_stride=1 << 20)])
def test_book_checks(lib, kw):
    b = book(**kw)
    assert status_of(ds.ds_pages_reserve, b, FAKE, FAKE, 1, FAKE, FAKE, 4096, None) == EINVAL
    assert status_of(ds.ds_pages_fork, pool(), b, FAKE, FAKE, 1, FAKE, FAKE, 4096, None) == EINVAL
    assert status_of(ds.ds_pages_free, b, FAKE, 1, None) == EINVAL
    if "lengths" not in kw:   # a compaction does not use the lengths
        assert status_of(ds.ds_pages_compact, pool(), b, FAKE, FAKE, FAKE, 4096, None) == EINVAL


def test_more_pages_or_entries_than_are_counted_in_32_bits(lib):
    most, big = 1 << 30, 1 << 60
    for n in (most + 1, 2 ** 31 - 1):
        for rc in (status_of(ds.ds_pages_reserve, book(n_pages=n), FAKE, FAKE, 1, FAKE, FAKE, big, None),
                   status_of(ds.ds_pages_reserve, book(), FAKE, FAKE, n, FAKE, FAKE, big, None),
                   status_of(ds.ds_pages_fork, pool(n_pages=n), book(n_pages=n), FAKE, FAKE, 1, FAKE, FAKE,
                             big, None),
                   status_of(ds.ds_pages_fork, pool(), book(), FAKE, FAKE, n, FAKE, FAKE, big, None),
                   status_of(ds.ds_pages_free, book(), FAKE, n, None),
                   status_of(ds.ds_pages_copy, pool(), FAKE, FAKE, n, None),
                   status_of(ds.ds_pages_compact, pool(n_pages=n), book(n_pages=n), FAKE, FAKE, FAKE, big,
                             None)):
            assert rc == EUNSUP


def test_workspace_bytes_of_the_wrappers(lib):
    from top_selection_deepselect_gb300 import _kv4
    for n_pages in (1, 7, 8192, 1 << 30):
        for n in (0, 1, 1000, 1 << 30):
            assert _kv4._pages_bytes(n_pages, n) == ds.ds_pages_workspace(n_pages, n)


def test_page_list_and_workspace_checks(lib):
    need = ds.ds_pages_workspace(4, 2)
    assert ds.ds_pages_workspace(4, 0) > 0
    for a, n, ws, size, st in [(None, 2, FAKE, need, FAKE), (FAKE, -1, FAKE, need, FAKE),
                               (FAKE, 2, None, need, FAKE), (FAKE, 2, FAKE + 4, need, FAKE),
                               (FAKE, 2, FAKE, need - 1, FAKE), (FAKE, 2, FAKE, need, None)]:
        assert status_of(ds.ds_pages_reserve, book(), a, FAKE, n, st, ws, size, None) == EINVAL
        assert status_of(ds.ds_pages_fork, pool(), book(), a, FAKE, n, st, ws, size, None) == EINVAL
    assert status_of(ds.ds_pages_copy, pool(), None, FAKE, 1, None) == EINVAL
    assert status_of(ds.ds_pages_copy, pool(), None, None, 0, None) == ds.DS_OK
    assert status_of(ds.ds_pages_free, book(), None, 1, None) == EINVAL
    assert status_of(ds.ds_pages_free, book(), None, 0, None) == ds.DS_OK
    assert status_of(ds.ds_pages_compact, pool(), book(), None, FAKE, FAKE, 4096, None) == EINVAL
    assert status_of(ds.ds_pages_compact, pool(n_pages=5), book(), FAKE, FAKE, FAKE, 4096,
                     None) == EINVAL


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_model_of_the_records(dim):
    for places in model.channel_places(dim):
        assert sorted(places) == list(range(dim))
    rng = np.random.default_rng(dim)
    k, v = rng.standard_normal((2, 5, 3, dim)).astype(np.float32)
    v[0, 0] = 0
    rec = model.encode(k, v)
    assert rec.shape == (5, 3, model.record_bytes(dim))
    for x, y in zip((k, v), model.decode(rec, dim)):
        top = np.abs(x).reshape(5, 3, -1, 32).max(-1).repeat(32, -1)
        # half a step, the step rounded to fp16
        assert (np.abs(x - y) <= top / 14 * (1 + 2.0 ** -9) + 1e-7).all()
    assert (model.decode(rec, dim)[1][0, 0] == 0).all()


def test_model_poisons_groups_that_are_not_finite():
    x = np.ones((1, 64), dtype=np.float32)
    x[0, 3] = np.inf
    x[0, 40] = 1e30
    k, _ = model.decode(model.encode(x, x), 64)
    assert np.isnan(k[0, :32]).all()
    assert k[0, 40] == 7 * 65504.0 and (k[0, 41:] == 0).all()
