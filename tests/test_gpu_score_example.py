"""examples/score_text.py runs: chunks, scores and gradients together, as a program uses them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "score_text.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as ds
    ds.build()
    spec = importlib.util.spec_from_file_location("score_text", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_scores_are_those_of_the_logits(example):
    """Log probabilities, entropy and alternatives against log_softmax in 64 bits.  Chunks make their logits with
    products of other sizes than all rows together do, which may round a bf16 logit the other way: off by a unit,
    2^-7 of the largest logit at most, and log probabilities by two of these."""
    import top_selection_deepselect_gb300 as ds
    r = example.run()
    bf16 = r["hidden"] @ r["model"].head
    logits = bf16.double()
    logp = torch.log_softmax(logits, -1)
    scored = r["following"] >= 0
    assert scored.sum() == len(scored) - len(r["texts"]) and not r["logprob"][~scored].any()
    want = logp.gather(1, r["following"].clamp(min=0).long()[:, None])[:, 0]
    got = ds.token_logprobs(bf16, r["following"], 4)
    # 3001 terms of sums in 32 bits: 2^-22 (3001 / 512 + 64 + 2 E|d|) with E|d| below 24, see test_gpu_logprob
    t = 2.0 ** -22 * 128 + 2.0 ** -21 * want.abs()
    assert ((got[0] - want).abs() <= t)[scored].all()
    assert (got[1] + (logp * logp.exp()).sum(-1)).abs().max() <= 2.0 ** -13
    assert (got[4] - logp.gather(1, got[3].long())).abs().max() <= 2.0 ** -14
    assert torch.equal(logits.gather(1, got[3][:, :1].long())[:, 0], logits.amax(-1))
    unit = 2.0 ** -7 * logits.abs().amax(-1)
    assert ((r["logprob"] - want).abs() <= 2 * unit + t)[scored].all()
    assert ((r["lse"] - got[2]).abs() <= unit + 2.0 ** -14).all()


def test_the_chunks_size_changes_nothing_but_roundings(example):
    """The keys and values of a token do not depend on how its text is cut, if the layers below agree; hidden states
    of two layers in bf16 then differ by a few units of 2^-8, and scores by as much of the logits' size."""
    model = example.Model(3001, 2, 8, 2, 64, 0, torch.device("cuda:0"))
    texts = [list(range(5, 155)), [7], list(range(300, 333))]
    a, b = (example.score(model, texts, chunk) for chunk in (1000, 37))
    assert torch.equal(a[1], b[1])
    assert (a[0] - b[0]).abs().max() <= 2.0 ** -3
    assert (a[2] - b[2]).abs().max() <= 0.5 and (a[2] - b[2]).abs().mean() <= 2.0 ** -5


def test_gradient_is_the_formulas_and_the_differences(example):
    """Against autograd through log_softmax in 64 bits on the same logits (whose gradient comes rounded to bf16, as
    here), and against differences of the 64-bit loss along a direction."""
    r = example.run()
    model, scored = r["model"], r["following"] >= 0

    def loss(head):
        logp = torch.log_softmax((r["hidden"].double() @ head), -1)
        lp = logp.gather(1, r["following"].clamp(min=0).long()[:, None])[:, 0]
        h = -(logp * logp.exp()).sum(-1)
        return -((r["advantage"] * lp + 0.01 * h)[scored]).sum() / scored.sum()

    head = model.head.double().requires_grad_()
    want, = torch.autograd.grad(loss(head), head)
    # logits and their gradient are bf16: 2^-9 relative each, the product's result too
    assert (r["grad"] - want).norm() <= 2.0 ** -6 * want.norm()
    step = 1e-4 * want / want.norm()
    with torch.no_grad():
        slope = (loss(head + step) - loss(head - step)) / 2e-4
    assert abs(slope - want.norm()) <= 1e-4 * want.norm()
    assert abs((r["grad"].double() * want).sum() / want.norm() - slope) <= 2.0 ** -6 * slope
