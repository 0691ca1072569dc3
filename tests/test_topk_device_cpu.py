"""topk and topk_long_row launch on their tensor's device, whichever is current, on a host without
any: devices, streams and the library's functions are stand-ins that note what they are asked."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import top_selection_deepselect_gb300 as ds
from top_selection_deepselect_gb300 import _binding

MINE = 1


class On:
    """A CPU tensor that says it is on a CUDA device."""
    is_cuda = True

    def __init__(self, x):
        self.x = x

    def get_device(self):
        return MINE

    def __getattr__(self, name):
        return getattr(self.x, name)


@pytest.fixture
def cuda(monkeypatch):
    state = types.SimpleNamespace(now=0, calls=[])

    @contextlib.contextmanager
    def device(index):
        before, state.now = state.now, index
        yield
        state.now = before

    def library(name, answer):
        def call(*args):
            state.calls.append((name, state.now, args[-1]))
            return answer
        return call

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.now)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device: types.SimpleNamespace(cuda_stream=7, device_index=MINE))
    for name, answer in [("ds_topk_ex", None), ("ds_topk_long_row", None), ("ds_topk_long_row_workspace", 64)]:
        monkeypatch.setattr(_binding, name, library(name, answer))
    return state


CALLS = [lambda **kw: ds.topk(On(torch.zeros((3, 64))), 4, 16, 16, **kw),
         lambda **kw: ds.topk_long_row(On(torch.zeros(64)), 4, 16, 16, **kw)]


@pytest.mark.parametrize("call", CALLS, ids=["topk", "topk_long_row"])
@pytest.mark.parametrize("current", [0, MINE])
def test_the_tensors_device_is_current_at_the_launch(cuda, call, current):
    cuda.now = current
    idx, val = call()
    assert idx.shape == val.shape and idx.shape[-1] == 4
    assert {c[1] for c in cuda.calls} == {MINE} and cuda.calls[-1][2] == 7
    assert cuda.now == current
    call(stream=types.SimpleNamespace(cuda_stream=9, device_index=MINE))
    assert {c[1] for c in cuda.calls} == {MINE} and cuda.calls[-1][2] == 9


@pytest.mark.parametrize("call", CALLS, ids=["topk", "topk_long_row"])
def test_a_stream_of_another_device_is_refused(cuda, call):
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(cuda_stream=9, device_index=0))
    assert not cuda.calls
