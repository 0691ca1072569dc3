"""Pages of a cache on the GPU against the model, every byte and every count."""
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


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).to(DEV)


class Both:
    """The same state on the GPU and in the model."""

    def __init__(self, ds, n_pages, max_seqs, max_pages, page, layers=2, heads=1, rec=16, seed=0,
                 spare_columns=0):
        rng = np.random.default_rng(seed)
        self.ds, self.page = ds, page
        self.pool = rng.integers(0, 256, (layers, n_pages, heads, page, rec), dtype=np.uint8)
        table = np.full((max_seqs, max_pages), -1, dtype=np.int32)
        self.m = model.Book(table, np.zeros(max_seqs, np.int32), np.zeros(n_pages, np.int32), page)
        self.d_pool = dev(self.pool, np.uint8)
        wide = np.full((max_seqs, max_pages + spare_columns), -77, dtype=np.int32)
        wide[:, :max_pages] = -1
        self.wide = dev(wide)
        self.table = self.wide[:, :max_pages]
        self.lengths, self.refs = dev(self.m.lengths), dev(self.m.refs)

    def check(self):
        assert np.array_equal(self.table.cpu().numpy(), self.m.table)
        assert np.array_equal(self.lengths.cpu().numpy(), self.m.lengths)
        assert np.array_equal(self.refs.cpu().numpy(), self.m.refs)
        assert np.array_equal(self.d_pool.cpu().numpy(), self.pool)
        assert (self.wide[:, self.table.shape[1]:] == -77).all()

    def reserve(self, seqs, tokens):
        st = self.ds.pages_reserve(self.table, self.lengths, self.refs, dev(seqs), dev(tokens),
                                   self.page)
        want = self.m.reserve(seqs, tokens)
        assert tuple(st.tolist()) == want
        self.check()
        return want

    def fork(self, src, dst):
        st = self.ds.pages_fork(self.d_pool, self.table, self.lengths, self.refs, dev(src), dev(dst))
        want = self.m.fork(self.pool, src, dst)
        assert tuple(st.tolist()) == want
        self.check()
        return want

    def free(self, seqs):
        self.ds.pages_free(self.table, self.lengths, self.refs, dev(seqs), self.page)
        self.m.free(seqs)
        self.check()

    def compact(self):
        remap, st = self.ds.pages_compact(self.d_pool, self.table, self.refs)
        want, counts = self.m.compact(self.pool)
        assert tuple(st.tolist()) == counts
        assert np.array_equal(remap.cpu().numpy(), want)
        self.check()
        return counts


@pytest.mark.parametrize("page,n_pages,rec", [(1, 40, 16), (16, 60, 80), (7, 33, 144), (64, 2000, 16)])
def test_a_life_of_sequences(ds, page, n_pages, rec):
    """Random steps, with entries out of range and repeated ones among them."""
    rng = np.random.default_rng(page)
    b = Both(ds, n_pages, 12, 20, page, rec=rec, seed=page, spare_columns=3)
    short = moved = 0
    for _ in range(60):
        op = rng.integers(0, 10)
        if op < 4:
            n = rng.integers(0, 7)
            short += b.reserve(rng.integers(-1, 13, n), rng.integers(-1, 4 * page + 2, n))[0] > 0
        elif op < 6:
            n = rng.integers(0, 5)
            b.fork(rng.integers(-1, 13, n), rng.integers(-1, 13, n))
        elif op < 8:
            b.free(rng.integers(-1, 13, rng.integers(0, 4)))
        else:
            moved += b.compact()[1]
    assert moved > 0
    if n_pages < 50:
        assert short > 0


def test_nothing_changes_when_pages_are_short(ds):
    b = Both(ds, 10, 4, 6, 8)
    assert b.reserve([0, 1], [40, 20]) == (0, 8)
    assert b.reserve([2, 0], [16, 1]) == (1, 0)             # three pages wanted, two free
    assert b.reserve([1], [40]) == (2 + 1, 0)               # two beyond the row, one of three not free
    assert b.reserve([2], [2 ** 31 - 1])[0] > 0
    assert b.reserve([2], [16]) == (0, 2)
    assert b.fork([1], [3]) == (1, 0)                       # 20 tokens: the last page is not full
    assert b.fork([0], [3]) == (0, 0)                       # 40 tokens: all pages are shared
    b.free([0])
    b.free([3, 3])


def test_children_share_full_pages_and_own_the_last(ds):
    b = Both(ds, 64, 16, 8, 4, layers=3, heads=2, rec=80)
    b.reserve([0, 1], [14, 8])
    assert b.fork([0] * 7 + [1] * 3, range(2, 12)) == (0, 7)
    assert b.m.refs.max() == 8
    b.free(range(0, 12, 2))
    assert b.compact()[1] > 0
    b.free([1])
    b.free(range(16))
    assert b.m.refs.max() == 0
    assert b.compact() == (0, 0)


def test_long_lists(ds):
    """More entries than the bookkeeping CTA has threads, and thousands of pages."""
    n = 2500
    rng = np.random.default_rng(1)
    b = Both(ds, 9001, 2 * n, 3, 2, layers=1)
    b.reserve(rng.permutation(n), rng.integers(1, 7, n))
    b.fork(np.arange(n), n + rng.permutation(n))
    b.free(rng.permutation(2 * n)[:n])
    assert b.compact()[1] > 100
    b.reserve(rng.integers(0, 2 * n, n), np.ones(n, int))
    b.compact()


@pytest.mark.parametrize("n_pages", [1, 31, 32, 33, 1024, 1025])
@pytest.mark.parametrize("live", ["none", "all", "odd", "last"])
def test_compaction_of_every_kind_of_pool(ds, n_pages, live):
    b = Both(ds, n_pages, n_pages, 1, 1, layers=1)
    keep = {"none": [], "all": list(range(n_pages)), "odd": list(range(1, n_pages, 2)),
            "last": [n_pages - 1]}[live]
    b.reserve(range(n_pages), [1] * n_pages)
    b.free([s for s in range(n_pages) if s not in set(keep)])
    b.compact()


@pytest.mark.parametrize("shape", [(1, 9, 16), (2, 9, 3, 5, 80), (3, 6, 70000), (1, 5, 16400)])
def test_copy(ds, shape):
    rng = np.random.default_rng(2)
    host = rng.integers(0, 256, shape, dtype=np.uint8)
    pool = dev(host, np.uint8)
    src, dst = [0, 3, -1, 1, 0, 99], [2, 4, 1, -1, shape[1], 2]
    ds.pages_copy(pool, dev(src), dev(dst))
    host[:, 2], host[:, 4] = host[:, 0], host[:, 3]
    assert np.array_equal(pool.cpu().numpy(), host)
    ds.pages_copy(pool, dev([]), dev([]))


def test_copy_of_other_types_and_strides(ds):
    """Pages of a bf16 cache, and a pool whose layers lie inside the pages."""
    rng = np.random.default_rng(3)
    base = torch.from_numpy(rng.standard_normal((6, 3, 4, 8))).to(DEV).bfloat16()
    want = base.clone()
    want[4], want[5] = want[1], want[0]
    ds.pages_copy(base.transpose(0, 1), dev([1, 0]), dev([4, 5]))
    assert torch.equal(base, want)


def test_copy_beyond_32_bits(ds):
    pool = torch.zeros((2, 70, 1 << 25), dtype=torch.uint8, device=DEV)    # 4.4 GB
    pool[1, 68].random_(0, 256)
    ds.pages_copy(pool, dev([68]), dev([69]))
    assert torch.equal(pool[1, 69], pool[1, 68]) and pool[1, 69].any() and not pool[0, 69].any()


def test_refusals(ds):
    b = Both(ds, 8, 4, 4, 4)
    lists = dev([0]), dev([1])
    with pytest.raises(ValueError):
        ds.pages_copy(b.d_pool, lists[0].long(), lists[1])
    with pytest.raises(ValueError):
        ds.pages_copy(b.d_pool.cpu(), *lists)
    with pytest.raises(ValueError):
        ds.pages_copy(b.d_pool[..., ::2], *lists)
    for overlapping in (b.d_pool[:, :1].expand(-1, 8, -1, -1, -1), b.d_pool[:1].expand(2, -1, -1, -1, -1)):
        with pytest.raises(ValueError):
            ds.pages_copy(overlapping, *lists)
    with pytest.raises(ValueError):
        ds.pages_free(b.table[:1].expand(4, -1), b.lengths, b.refs, lists[0], 4)
    with pytest.raises(ValueError):
        ds.pages_fork(b.d_pool[0], b.table, b.lengths, b.refs, *lists)
    with pytest.raises(ValueError):
        ds.pages_reserve(b.table, b.lengths[:2], b.refs, *lists, 4)
    with pytest.raises(ds.DSError) as e:
        ds.pages_reserve(b.table, b.lengths, b.refs, *lists, 0)
    assert e.value.status == ds.DS_EINVAL
    with pytest.raises(ds.DSError):
        ds.pages_compact(b.d_pool, b.table, b.refs[:4].clone())
    with pytest.raises(ds.DSError):
        ds.pages_copy(b.d_pool.view(2, 8, -1)[:, :, :24], *lists)
    with pytest.raises(ds.DSError):
        ds.pages_free(b.table, b.lengths, b.refs, dev([0]), -1)
    b.check()


def test_reserve_for_negative_lengths(ds):
    """They count as 0, the smallest ones too."""
    low = -2 ** 31
    seqs, tokens = [4, 3, 1, 3, 0, 2], [5, 17, 16, 9, 1, 33]
    for lengths in ([low, low, low, low, low], [low + 3, low + 2, low + 1, low, -1], [-7, low + 5, 0, low + 1, low + 4]):
        table, got, refs = dev(np.full((5, 4), -1)), dev(lengths), dev(np.zeros(9))
        status = ds.pages_reserve(table, got, refs, dev(seqs), dev(tokens), 16)
        assert status.tolist() == [0, 8]
        assert got.tolist() == [1, 16, 33, 17, 5]
        assert table[:, :3].tolist() == [[4, -1, -1], [3, -1, -1], [5, 6, 7], [1, 2, -1], [0, -1, -1]]
        assert refs.tolist() == [1] * 8 + [0]
