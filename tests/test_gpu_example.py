"""examples/selected_decode.py runs, and what it must leave holds."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "selected_decode.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as ds
    ds.build()
    spec = importlib.util.spec_from_file_location("selected_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_sequences_branch_end_and_move(example):
    r = example.run()
    assert torch.isfinite(r["hidden"].float()).all() and torch.isfinite(r["drafts"].float()).all()
    # parent and children hold the same tokens: the same next token gives the same state
    assert torch.equal(r["branched"][1], r["branched"][0])
    assert torch.equal(r["branched"][2], r["branched"][0])
    # the pages moved, what they hold did not change
    assert torch.equal(r["after"], r["before"][1:])
    assert r["moved"] > 0
    held = {p for row in r["table"] for p in row if p >= 0}
    assert held == set(range(r["live"]))
    n = 128 + 4 + 3 + 1
    assert [x for x in r["lengths"] if x] == [n, n]
    full = n // 16
    assert sorted(r["refs"], reverse=True)[:full] == [2] * full
    assert sum(r["refs"]) == 2 * -(-n // 16)


def test_selecting_every_token_is_attending_every_token(example):
    """With k at least as long as the sequences, selected steps equal plain ones but for the order of sums."""
    a, b = (example.run(prompts=(40, 17), steps=3, k=k) for k in (256, 0))
    diff = (a["hidden"].float() - b["hidden"].float()).abs().max()
    # two layers of bf16 states of size about 3: a few units of 2^-8 relative
    assert diff <= 2.0 ** -4
