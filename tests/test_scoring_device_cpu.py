"""The wrappers of chunk attention and log probabilities launch on their tensors' device, whichever is
current: with the stand-ins of test_kv4_device_cpu."""
import pytest

torch = pytest.importorskip("torch")

import top_selection_deepselect_gb300 as ds
from test_kv4_device_cpu import MINE, On, Stream, cuda  # noqa: F401
from top_selection_deepselect_gb300 import _kv4, _logprob


class Library:
    def __init__(self, t):
        for name in ("ds_token_logprobs", "ds_token_logprobs_backward"):
            setattr(self, name, self.noting(t, name))

    @staticmethod
    def noting(t, name):
        def call(*args):
            t.calls.append((name, t.now, args[-1]))
            return 0
        return call


@pytest.fixture
def device(cuda, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_logprob, "_t", cuda)
    monkeypatch.setattr(_logprob, "_lib", lambda library=Library(cuda): library)
    cuda.chunk = Library.noting(cuda, "chunk")
    cuda.chunk_workspace = lambda *args: cuda.workspace(*args)
    assert _kv4._t is cuda
    return cuda


def calls():
    def i32(*shape):
        return On(torch.zeros(shape, dtype=torch.int32))
    pool = On(torch.zeros((4, 2, 16, 144), dtype=torch.uint8))
    q = On(torch.zeros((5, 4, 128), dtype=torch.bfloat16))
    x, f = On(torch.zeros((3, 50))), On(torch.zeros(3))
    return {
        "chunk": lambda **kw: ds.kv4_chunk_attention(q, pool, i32(3, 4), i32(3), i32(4), **kw),
        "ds_token_logprobs": lambda **kw: ds.token_logprobs(x, i32(3), 2, **kw),
        "ds_token_logprobs_backward": lambda **kw: ds.token_logprobs_backward(x, i32(3), f, f, f, **kw)}


NAMES = sorted(calls())


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, MINE])
def test_the_tensors_device_is_current_at_the_launch(device, name, current):
    device.now = current
    calls()[name]()
    assert [c[2] for c in device.calls if c[0] == name] == [7]
    assert {c[1] for c in device.calls} == {MINE}
    assert device.now == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_the_tensors_device(device, name):
    calls()[name](stream=Stream(MINE))
    assert [c[2] for c in device.calls if c[0] == name] == [9]
    assert {c[1] for c in device.calls} == {MINE}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, MINE])
def test_a_stream_of_another_device_is_refused(device, name, current):
    device.now = current
    with pytest.raises(ValueError):
        calls()[name](stream=Stream(0))
    assert not device.calls


def test_a_tangent_is_refused(device, monkeypatch):
    """There is no forward-mode derivative, and a result without one would say that it is 0."""
    from torch.autograd import forward_ad
    monkeypatch.setattr(_kv4, "_cuda", lambda name, x: MINE)
    device.now = MINE
    tokens = On(torch.zeros(3, dtype=torch.int32))
    with forward_ad.dual_level():
        for primal in (torch.zeros((3, 50)), torch.zeros((3, 50), requires_grad=True)):
            x = forward_ad.make_dual(primal, torch.ones((3, 50)))
            with pytest.raises(NotImplementedError):
                ds.token_logprobs(x, tokens, 2)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                ds.token_logprobs(x, tokens, 2)
    assert not device.calls
