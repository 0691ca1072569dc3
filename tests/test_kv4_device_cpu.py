"""The cache's wrappers launch on their tensors' device, whichever is current, on a host without
any: devices, streams and the library's functions are stand-ins that note what they are asked."""
import contextlib
import weakref

import pytest

torch = pytest.importorskip("torch")

import top_selection_deepselect_gb300 as ds
from top_selection_deepselect_gb300 import _kv4

MINE = 1


class On:
    """A CPU tensor that says it is on a CUDA device."""
    def __init__(self, x, index=MINE):
        self.x, self.index = x, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.x, name)

    def __getitem__(self, at):
        return On(self.x[at], self.index)


class Stream:
    def __init__(self, device_index):
        self.device_index = device_index


@pytest.fixture
def cuda(monkeypatch):
    """Device 0 is current; calls notes (function, device current then, stream's device)."""
    ds.build()
    t = _kv4._Torch().find()
    t.now, t.stream, t.calls = 0, None, []

    @contextlib.contextmanager
    def on_device(index):
        before, t.now = t.now, index
        yield
        t.now = before

    @contextlib.contextmanager
    def on_stream(stream):
        before = t.now, t.stream
        t.now, t.stream = stream.device_index, stream
        yield
        t.now, t.stream = before

    def handle(index):
        assert index == MINE
        return 7 if t.stream is None else 9

    def library(name):
        def call(*args):
            t.calls.append((name, t.now, args[-1]))
            return 0
        return call

    def workspace(*args):
        t.calls.append(("workspace", t.now, None))
        args[-1]._obj.value = 64
        return 0

    t.current, t.on_device, t.on_stream, t.raw_stream = lambda: t.now, on_device, on_stream, handle
    t.capturing = lambda: t.calls.append(("capturing", t.now, None)) or False
    t.empty = lambda shape, dtype, device: On(torch.empty(shape, dtype=dtype))
    t.empty_like = lambda x: On(torch.empty_like(x.x))
    for name in ("append", "read", "attention", "copy", "reserve", "fork", "free", "compact"):
        setattr(t, name, library(name))
    t.workspace = workspace
    monkeypatch.setattr(_kv4, "_t", t)
    monkeypatch.setattr(_kv4, "_attention_bytes", {})
    return t


def tensors():
    def i32(*shape):
        return On(torch.zeros(shape, dtype=torch.int32))
    pool = On(torch.zeros((4, 2, 16, 144), dtype=torch.uint8))
    layers = On(torch.zeros((3, 4, 2, 16, 144), dtype=torch.uint8))
    x = On(torch.zeros((5, 2, 128)))
    q = On(torch.zeros((3, 1, 4, 128), dtype=torch.bfloat16))
    table, lengths, refs, some, pair = i32(3, 4), i32(3), i32(4), i32(5), i32(2)
    return {
        "append": lambda **kw: ds.kv4_append(pool, table, some, some, x, x, **kw),
        "read": lambda **kw: ds.kv4_read(pool, table, some, some, 128, torch.float32, **kw),
        "attention": lambda **kw: ds.kv4_attention(q, pool, table, lengths, **kw),
        "copy": lambda **kw: ds.pages_copy(layers, pair, pair, **kw),
        "reserve": lambda **kw: ds.pages_reserve(table, lengths, refs, pair, pair, 16, **kw),
        "fork": lambda **kw: ds.pages_fork(layers, table, lengths, refs, pair, pair, **kw),
        "free": lambda **kw: ds.pages_free(table, lengths, refs, pair, 16, **kw),
        "compact": lambda **kw: ds.pages_compact(layers, table, refs, **kw)}


NAMES = sorted(tensors())


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, MINE])
def test_the_tensors_device_is_current_at_the_launch(cuda, name, current):
    cuda.now = current
    tensors()[name]()
    assert [c[2] for c in cuda.calls if c[0] == name] == [7]
    assert {c[1] for c in cuda.calls} == {MINE}
    assert cuda.now == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_the_tensors_device(cuda, name):
    tensors()[name](stream=Stream(MINE))
    assert [c[2] for c in cuda.calls if c[0] == name] == [9]
    assert {c[1] for c in cuda.calls} == {MINE}
    assert cuda.now == 0


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, MINE])
def test_a_stream_of_another_device_is_refused(cuda, name, current):
    cuda.now = current
    with pytest.raises(ValueError):
        tensors()[name](stream=Stream(0))
    assert not cuda.calls


@pytest.mark.parametrize("name", ["attention", "reserve", "fork", "compact"])
def test_a_workspace_is_the_calls_own(cuda, name):
    """What a call allocates beside its results ends with it: memory that is kept by a stream's handle
    would be another stream's when CUDA gives the handle out again."""
    given = []

    def empty(shape, dtype, device):
        x = On(torch.empty(shape, dtype=dtype))
        if dtype == torch.uint8:
            given.append(weakref.ref(x))
        return x

    cuda.empty, cuda.now = empty, MINE
    call = tensors()[name]
    for _ in range(3):
        call()
    assert len(given) == 3 and all(x() is None for x in given)
