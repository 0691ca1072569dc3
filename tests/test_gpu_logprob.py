"""Log probabilities, entropy, alternatives and their gradient on the GPU against the 64-bit model,
within bounds derived from the roundings."""
import numpy as np
import pytest

import oracle.logprob as model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import top_selection_deepselect_gb300 as _ds
    _ds.build()
    _ds.load_library()
    return _ds


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if dtype is None else t.to(dtype)


def bounds(x, scale):
    """How far (lse, a log probability's offset, entropy) of each row may be off, and E|d|.

    d = (x - m) scale log2 e carries four roundings (of scale log2 e two, the difference, the
    product), so that 2^d is off by 2^-22 |d| relative, and by 2^-22 of the exponential itself.  A
    thread adds vocab / 512 pairs at most, then 8 + 8 + 8 joins follow, each a rounding, and each
    join or new maximum (64 at most on rows as random as these) a factor with 2^-22 of its own:
    rs = 2^-22 (vocab / 512 + 64 + 2 E|d|) relative covers S, and T twice as much.  lse and the
    entropy are rounded from 64 bits."""
    z = np.where(np.isneginf(x), -np.inf, x) * scale
    with np.errstate(all="ignore"):
        m = z.max(-1, keepdims=True)
        d = np.where(np.isneginf(z), 0, (z - m) / np.log(2))
        e = np.where(np.isneginf(z), 0, np.exp(z - m))
        mean = np.abs(e * d).sum(-1) / e.sum(-1)
    rs = 2.0 ** -22 * (x.shape[1] / 512 + 64 + 2 * np.nan_to_num(mean))
    return rs, rs, 3 * rs * (1 + np.nan_to_num(mean))


def same_but(got, want, t):
    """Equal where not finite, within t elsewhere."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    wild = ~np.isfinite(want)
    assert np.array_equal(got[wild & ~np.isnan(want)], want[wild & ~np.isnan(want)])
    assert (np.abs(got - want) <= t)[~wild].all(), np.nanmax(np.where(wild, 0, np.abs(got - want) / t))


def check_forward(ds, xt, tokens, k, scale=1.0, **kw):
    got = ds.token_logprobs(xt, tokens, k, scale=scale, **kw)
    torch.cuda.synchronize()
    x = xt.double().cpu().numpy()
    tok = tokens.cpu().numpy()
    ref = model.forward(x, tok, k, float(np.float32(scale)))
    tl, tp, te = bounds(x, scale)
    lp, h, lse, idx, top = (g.cpu().numpy() for g in got)
    assert np.array_equal(idx, ref[3])
    with np.errstate(invalid="ignore"):
        same_but(lse, ref[2], tl + 2.0 ** -22 * np.abs(ref[2]))
        same_but(lp, ref[0], tp + 2.0 ** -21 * np.abs(ref[0]))
        same_but(h, ref[1], te + 2.0 ** -22 * np.abs(ref[1]))
        same_but(top, ref[4], tp[:, None] + 2.0 ** -21 * np.abs(ref[4]))
    return got


def check_backward(ds, xt, tokens, idx, scale, g, out=None, which=(1, 1, 1, 1)):
    """The model's gradient, with bounds: log p is off by its rounding 2^-24 |log p| and by lse's
    error, p by that and 2^-22 (16-bit logits: the product with log2 e 2^-23 |log p| more), what p is
    multiplied with by k + 4 roundings of its terms; a final rounding to the logits' type."""
    rows, vocab = xt.shape
    x = xt.double().cpu().numpy()
    lp, h, lse, _, _ = ds.token_logprobs(xt, tokens, 0, scale=scale)
    use = [t if w else None for t, w in zip(g, which)]
    got = ds.token_logprobs_backward(xt, tokens, lse, h, grad_logprob=use[0], grad_entropy=use[1],
                                     grad_lse=use[2], idx=idx if which[3] else None, grad_top=use[3],
                                     scale=scale, out=out)
    torch.cuda.synchronize()
    gn = [(t if w else torch.zeros_like(t)).double().cpu().numpy() for t, w in zip(g, which)]
    tok, ind = tokens.cpu().numpy(), idx.cpu().numpy()
    s = float(np.float32(scale))
    ref = model.backward(x, tok, ind, s, *gn)
    _, rh, rlse, _, _ = model.forward(x, tok, 0, s)
    # rows of large sums are summed again and not taken from their rounded lse
    rlse = np.where(np.abs(rlse) < 1024, rlse, 0)
    tl, _, te = bounds(x, scale)
    with np.errstate(all="ignore"):
        logp = np.stack([model.log_probs(row * s)[0] for row in x])
        p = np.where(np.isneginf(logp), 0, np.exp(logp))
        logp = np.where(np.isneginf(logp), 0, logp)
        dl = (2.0 ** -23 * np.abs(logp) + (tl + 2.0 ** -22 * np.abs(rlse))[:, None])
        dp = dl + 2.0 ** -22 + 2.0 ** -23 * np.abs(logp)
        size = np.abs(gn[0]) + np.abs(gn[2]) + np.abs(gn[3]).sum(-1)
        inner = size[:, None] + np.abs(gn[1])[:, None] * (np.abs(logp) + rh[:, None])
        t = p * (np.abs(gn[1])[:, None] * (dl + te[:, None]) + inner * (dp + (ind.shape[1] + 4) * 2.0 ** -23))
        t = s * (t + 2.0 ** -22 * (ind.shape[1] + 2) * size[:, None] * (p > 0)) + 1e-30
    lo, hi = (torch.from_numpy(v).to(xt.dtype).double().numpy() for v in (ref - t, ref + t))
    got_n = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got_n), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert ((lo <= got_n) & (got_n <= hi))[fine].all()
    return got


def logits(rng, rows, vocab, dtype, spread=3.0):
    return dev((rng.standard_normal((rows, vocab)) * spread).astype(np.float32)).to(DTYPES[dtype])


def some_tokens(rng, rows, vocab):
    return dev(rng.integers(0, vocab, rows).astype(np.int32))


def some_grads(rng, rows, k):
    return [dev(rng.standard_normal(s).astype(np.float32)) for s in ((rows,), (rows,), (rows,), (rows, k))]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 2, 2), (5, 31, 31), (2, 33, 32), (4, 1000, 0),
                                          (3, 8191, 5), (2, 8193, 32), (3, 50257, 20), (1, 131072, 32),
                                          (1, 300001, 7), (320, 8200, 1)])
def test_forward(ds, dtype, rows, vocab, k):
    rng = np.random.default_rng(vocab + k)
    check_forward(ds, logits(rng, rows, vocab, dtype), some_tokens(rng, rows, vocab), k)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 2, 2), (2, 33, 32), (4, 1000, 0), (3, 8191, 5),
                                          (2, 50257, 32), (1, 131072, 3), (320, 2100, 1)])
def test_backward(ds, dtype, rows, vocab, k):
    rng = np.random.default_rng(vocab * 3 + k)
    x, tokens = logits(rng, rows, vocab, dtype), some_tokens(rng, rows, vocab)
    idx = ds.token_logprobs(x, tokens, k, scale=0.8)[3]
    check_backward(ds, x, tokens, idx, 0.8, some_grads(rng, rows, k))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("which", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (0, 0, 0, 0)])
def test_each_gradient_alone(ds, dtype, which):
    rng = np.random.default_rng(7)
    x, tokens = logits(rng, 3, 777, dtype), some_tokens(rng, 3, 777)
    idx = ds.token_logprobs(x, tokens, 4)[3]
    got = check_backward(ds, x, tokens, idx, 1.0, some_grads(rng, 3, 4), which=which)
    if not any(which):
        assert not got.any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 0), (3, 5), (8, 8), (7, 1)])
def test_rows_that_start_anywhere(ds, dtype, offset, gap):
    """Slices of a wider buffer; what lies around them is NaN and stays as it was."""
    rng = np.random.default_rng(offset * 10 + gap)
    rows, vocab = 4, 2051
    wide = torch.full((rows * (vocab + gap) + 64,), float("nan"), device=DEV, dtype=DTYPES[dtype])
    x = wide.as_strided((rows, vocab), (vocab + gap, 1), offset)
    x.copy_(logits(rng, rows, vocab, dtype))
    tokens = some_tokens(rng, rows, vocab)
    idx = check_forward(ds, x, tokens, 9, 1.3)[3]
    g = some_grads(rng, rows, 9)
    for shift in (0, 1, 8):
        room = torch.full((rows * (vocab + gap) + 64,), 7.0, device=DEV, dtype=DTYPES[dtype])
        out = room.as_strided((rows, vocab), (vocab + gap, 1), offset + shift)
        check_backward(ds, x, tokens, idx, 1.3, g, out=out)
        out.fill_(7.0)
        assert (room == 7.0).all()
    # in place: the same result
    want = check_backward(ds, x, tokens, idx, 1.3, g)
    lp, h, lse, _, _ = ds.token_logprobs(x, tokens, 0, scale=1.3)
    got = ds.token_logprobs_backward(x, tokens, lse, h, g[0], g[1], idx, g[3], g[2], 1.3, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [5, 777, 9001])
def test_masks(ds, dtype, vocab):
    """-inf here and there, nearly everywhere and everywhere; the type's lowest value; tokens without
    a probability and outside the vocabulary."""
    rng = np.random.default_rng(vocab)
    x = logits(rng, 9, vocab, dtype)
    x[0, ::2] = -float("inf")
    x[1, :] = -float("inf")
    x[2, :] = -float("inf")
    x[2, vocab // 2] = -3.0
    x[3, 1:] = torch.finfo(x.dtype).min
    x[4, :] = torch.finfo(x.dtype).min
    x[5, :] = -float("inf")
    x[5, -1] = torch.finfo(x.dtype).min
    x[6, :-1] = -float("inf")
    tokens = dev(np.array([0, 1, 0, 0, 2, 4, vocab - 1, -1, vocab], dtype=np.int32))
    k = min(5, vocab)
    got = check_forward(ds, x, tokens, k)
    assert got[0][7:].eq(0).all() and got[0][1].item() == -float("inf")
    idx = got[3]
    g = some_grads(rng, 9, k)
    grad = check_backward(ds, x, tokens, idx, 1.0, g)
    assert not grad[1].any()
    # entries of the list that are no tokens take no part
    idx = idx.clone()
    idx[:, 1] = -1
    idx[7, 2] = vocab
    check_backward(ds, x, tokens, idx, 1.0, g)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lift", [1000.0, -3e4, 2.0 ** 20])
def test_rows_far_from_zero(ds, dtype, lift):
    """lse in 32 bits says little about the probabilities of such rows."""
    rng = np.random.default_rng(12)
    steps = rng.integers(0, 3, (3, 2000)) * max(1.0, abs(lift) * 2.0 ** -7)
    x = dev((lift + steps).astype(np.float32)).to(DTYPES[dtype])
    tokens = some_tokens(rng, 3, 2000)
    idx = check_forward(ds, x, tokens, 4)[3]
    g = some_grads(rng, 3, 4)
    grad = check_backward(ds, x, tokens, idx, 1.0, g)
    lp, h, lse, _, _ = ds.token_logprobs(x, tokens)
    assert torch.equal(ds.token_logprobs_backward(x, tokens, lse, h, g[0], g[1], idx, g[3], g[2], out=x), grad)


def test_sums_beyond_32_bits(ds):
    """scale * logits is beyond fp32 and lse infinite; differences are not."""
    x = torch.full((2, 300), torch.finfo(torch.float32).min, device=DEV)
    x[1] = torch.finfo(torch.float32).max
    tokens = dev(np.array([5, 6], dtype=np.int32))
    lp, h, lse, _, top = ds.token_logprobs(x, tokens, 2, scale=4.0)
    assert lse.tolist() == [-float("inf"), float("inf")]
    want = -np.log(300.0)
    for t in (lp, -h, top[:, 0], top[:, 1]):
        assert (t.double() - want).abs().max() <= 2.0 ** -20
    grad = ds.token_logprobs_backward(x, tokens, lse, h, grad_logprob=torch.ones_like(lp), scale=4.0).double()
    assert (grad[0, 5] - 4 * 299 / 300).abs() <= 2.0 ** -18 and (grad[1, :6] + 4 / 300).abs().max() <= 2.0 ** -24


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_nan_and_infinity(ds, dtype):
    rng = np.random.default_rng(3)
    x = logits(rng, 6, 3000, dtype)
    x[1, 2999] = float("nan")
    x[2, 5] = float("inf")
    x[3, :] = float("nan")
    x[4, 7:50] = float("nan")
    tokens = dev(np.array([3, 3, 5, 0, 1, 2], dtype=np.int32))
    got = check_forward(ds, x, tokens, 32)
    assert torch.isnan(got[0][1:5]).all() and torch.isfinite(got[0][5])
    g = some_grads(rng, 6, 32)
    grad = check_backward(ds, x, tokens, got[3], 1.0, g)
    assert torch.isnan(grad[1:5]).all() and torch.isfinite(grad[5]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 40000), (310, 40000)])
def test_ties_and_sorted_rows(ds, dtype, rows, vocab):
    """Constant, ascending, descending and few-valued rows: most logits are candidates, or equal."""
    rng = np.random.default_rng(rows)
    base = np.arange(vocab, dtype=np.float32)
    kinds = [np.full(vocab, 1.5), base / 4096, -base / 4096, rng.integers(0, 3, vocab) * 0.5, base // 64,
             np.where(base < 3, -0.0, 0.0)]
    x = np.stack([kinds[i % 6] for i in range(rows)]).astype(np.float32) if rows > 6 else None
    if x is not None:
        check_rows = list(range(6))
        xt = dev(x).to(DTYPES[dtype])
        tokens = some_tokens(rng, rows, vocab)
        got = ds.token_logprobs(xt, tokens, 32)
        ref = model.forward(xt[:6].double().cpu().numpy(), tokens[:6].cpu().numpy(), 32, 1.0)
        assert np.array_equal(got[3][check_rows].cpu().numpy(), ref[3])
        again = got[3].cpu().numpy()
        for i in range(rows):
            assert np.array_equal(again[i], again[i % 6])
    else:
        for kind in kinds:
            xt = dev(kind[None].astype(np.float32)).to(DTYPES[dtype])
            got = ds.token_logprobs(xt, some_tokens(rng, 1, vocab), 32)
            assert got[3][0].cpu().tolist() == model.order(xt[0].double().cpu().numpy())[:32].tolist()


def test_large_logits_in_few_threads_places(ds):
    """Every 256 vectors the first 32 hold ever larger logits: neither bound on candidates helps."""
    rng = np.random.default_rng(11)
    rows, vocab = 310, 102400
    x = torch.zeros((rows, vocab), device=DEV)
    v = x[7].view(100, 256, 4)
    v[:, :32] = 1 + torch.arange(100, device=DEV)[:, None, None] + torch.rand((100, 32, 4), device=DEV)
    x[9] = torch.rand(vocab, device=DEV)
    got = ds.token_logprobs(x, some_tokens(rng, rows, vocab), 32)[3].cpu().numpy()
    for r in (0, 7, 9):
        assert got[r].tolist() == model.order(x[r].double().cpu().numpy())[:32].tolist()


@pytest.mark.parametrize("scale", [1e-3, 0.5, 30.0])
def test_scale(ds, scale):
    rng = np.random.default_rng(5)
    x, tokens = logits(rng, 3, 4097, "bf16"), some_tokens(rng, 3, 4097)
    idx = check_forward(ds, x, tokens, 3, scale)[3]
    check_backward(ds, x, tokens, idx, scale, some_grads(rng, 3, 3))


def test_the_token_among_the_alternatives_and_twice(ds):
    rng = np.random.default_rng(8)
    x, tokens = logits(rng, 4, 500, "fp32"), dev(np.array([3, 3, 499, 0], dtype=np.int32))
    idx = dev(np.array([[3, 3, 5], [1, 2, 3], [499, 0, 499], [7, 7, 7]], dtype=np.int32))
    check_backward(ds, x, tokens, idx, 1.0, some_grads(rng, 4, 3))


def test_autograd_is_the_explicit_call(ds):
    rng = np.random.default_rng(9)
    x = logits(rng, 5, 3001, "bf16").requires_grad_()
    tokens = some_tokens(rng, 5, 3001)
    logprob, entropy, lse, idx, top = ds.token_logprobs(x, tokens, 3, scale=0.9)
    assert not idx.requires_grad
    g = some_grads(rng, 5, 3)
    loss = (g[0] * logprob).sum() + (g[1] * entropy).sum() + (g[2] * lse).sum() + (g[3] * top).sum()
    got, = torch.autograd.grad(loss, x)
    with torch.no_grad():
        plain = ds.token_logprobs(x, tokens, 3, scale=0.9)
        want = ds.token_logprobs_backward(x, tokens, plain[2], plain[1], g[0], g[1], plain[3], g[3], g[2], 0.9)
    assert all(torch.equal(a, b) for a, b in zip((logprob, entropy, lse, idx, top), plain))
    assert torch.equal(got, want)
    # one output alone, and outputs that the caller has written into
    logprob, entropy, lse, _, _ = ds.token_logprobs(x, tokens)
    got, = torch.autograd.grad(logprob.sum(), x)
    with torch.no_grad():
        want = ds.token_logprobs_backward(x, tokens, plain[2], plain[1], torch.ones_like(plain[0]))
        again = ds.token_logprobs(x, tokens)
        want = ds.token_logprobs_backward(x, tokens, again[2], again[1], torch.ones_like(again[0]))
    assert torch.equal(got, want)
    logprob, entropy, lse, _, _ = ds.token_logprobs(x, tokens)
    loss = logprob.sum()
    lse.detach().zero_()
    with pytest.raises(RuntimeError):
        torch.autograd.grad(loss, x)


def test_streams_graphs_and_given_outputs(ds):
    rng = np.random.default_rng(10)
    x, tokens = logits(rng, 3, 20011, "bf16"), some_tokens(rng, 3, 20011)
    want = ds.token_logprobs(x, tokens, 6)
    grads = some_grads(rng, 3, 6)
    want_grad = ds.token_logprobs_backward(x, tokens, want[2], want[1], grads[0], grads[1], want[3], grads[3])
    outs = [torch.empty_like(w) for w in want]
    grad = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ds.token_logprobs(x, tokens, 6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def step():
        ds.token_logprobs(x, tokens, 6, logprob=outs[0], entropy=outs[1], lse=outs[2], idx=outs[3], top=outs[4])
        ds.token_logprobs_backward(x, tokens, outs[2], outs[1], grads[0], grads[1], outs[3], grads[3], out=grad)

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t in outs + [grad]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(grad, want_grad)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = ds.token_logprobs(x, tokens, 6)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_beyond_32_bits(ds):
    """17000 rows of 131072: the last rows start past element 2^31."""
    x = torch.zeros((17000, 131072), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x[-2:] = torch.randn((2, 131072), device=DEV, generator=g).bfloat16()
    tokens = torch.full((17000,), 70000, dtype=torch.int32, device=DEV)
    got = ds.token_logprobs(x, tokens, 4)
    rows = check_forward(ds, x[-2:].clone(), tokens[-2:], 4)
    for a, b in zip(got, rows):
        torch.testing.assert_close(a[-2:].double(), b.double(), rtol=2.0 ** -19, atol=2.0 ** -14)
    assert torch.equal(got[3][-2:], rows[3])
    grad = ds.token_logprobs_backward(x, tokens, got[2], got[1], torch.ones_like(got[0]), out=x)
    last = grad[-1].float()
    assert abs(last[70000].item() - 1) < 2.0 ** -7 and abs(last.sum().item()) < 0.05


def test_refusals(ds):
    x, tokens = torch.zeros((3, 8), device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    lp, h, lse, _, _ = ds.token_logprobs(x, tokens)
    for call in (lambda: ds.token_logprobs(x.cpu(), tokens), lambda: ds.token_logprobs(x[0], tokens),
                 lambda: ds.token_logprobs(x.t(), tokens), lambda: ds.token_logprobs(x, tokens.long()),
                 lambda: ds.token_logprobs(x, tokens[:2]), lambda: ds.token_logprobs(x[:1].expand(3, 8), tokens),
                 lambda: ds.token_logprobs(x, tokens, 2, idx=torch.zeros((3, 3), dtype=torch.int32, device=DEV)),
                 lambda: ds.token_logprobs_backward(x, tokens, lse, h, grad_top=torch.zeros((3, 2), device=DEV)),
                 lambda: ds.token_logprobs_backward(x, tokens, lse.double(), h),
                 lambda: ds.token_logprobs_backward(x, tokens, lse, h, out=x[:, :7]),
                 lambda: ds.token_logprobs_backward(
                     x, tokens, lse, h, out=torch.as_strided(torch.zeros(40, device=DEV), (3, 8), (7, 1)))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ds.token_logprobs(x.double(), tokens)
    buffer = torch.zeros(64, device=DEV)
    with pytest.raises(ValueError):
        ds.token_logprobs_backward(buffer[:24].view(3, 8), tokens, lse, h, out=buffer[4:28].view(3, 8))
    wide = torch.zeros((3, 16), device=DEV)
    ds.token_logprobs_backward(wide[:, :8], tokens, lse, h, out=wide[:, 8:])
    with pytest.raises(ds.DSError):
        ds.token_logprobs(x, tokens, 9)
    with pytest.raises(ds.DSError):
        ds.token_logprobs(x, tokens, -1)
    with pytest.raises(ValueError):
        ds.token_logprobs(x.requires_grad_(), tokens, lse=lse)
    empty = ds.token_logprobs(torch.zeros((0, 8), device=DEV), tokens[:0], 2)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0,), (0, 2), (0, 2)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,scale", [(1, 1.0), (1, 0.01), (310, 1.0)])
@pytest.mark.parametrize("k", [0, 5])
def test_rows_that_start_masked(ds, dtype, rows, scale, k):
    """The type's lowest value, or one as good as that, in all of a slice's first logits, and in
    all of a slice: what -inf is taken as in sums may not stand above the maximum so far."""
    rng = np.random.default_rng(rows + k)
    vocab = 40000
    lowest = torch.finfo(DTYPES[dtype]).min
    other = -6e4 if dtype == "fp16" else -1e31
    x = logits(rng, 6, vocab, dtype)
    x[0, :20000] = lowest
    x[1, :-1] = lowest
    x[2, :20000], x[2, 20000:39990] = other, -float("inf")
    x[3, :10000], x[3, 10000:30000] = -float("inf"), lowest
    x[4, ::2] = other
    x[5, 1:] = torch.linspace(lowest, other, vocab - 1, dtype=torch.float64).to(x.dtype)
    tokens = dev(np.array([30000, vocab - 1, 39995, 35000, 1, 0], dtype=np.int32))
    if rows == 1:
        for r in range(6):
            idx = check_forward(ds, x[r:r + 1], tokens[r:r + 1], k, scale)[3]
            check_backward(ds, x[r:r + 1], tokens[r:r + 1], idx, scale, some_grads(rng, 1, k))
        return
    one = check_forward(ds, x, tokens, k, scale)
    pick = torch.arange(rows, device=DEV) % 6
    all_rows = ds.token_logprobs(x[pick], tokens[pick], k, scale=scale)
    ref = model.forward(x.double().cpu().numpy(), tokens.cpu().numpy(), k, scale)
    tl, tp, te = bounds(x.double().cpu().numpy(), scale)
    for r in range(rows):
        a = r % 6
        assert abs(all_rows[2][r].item() - ref[2][a]) <= tl[a] + 2.0 ** -22 * abs(ref[2][a])
        assert abs(all_rows[0][r].item() - ref[0][a]) <= tp[a] + 2.0 ** -21 * abs(ref[0][a])
        assert abs(all_rows[1][r].item() - ref[1][a]) <= te[a] + 2.0 ** -22 * abs(ref[1][a])
    assert torch.equal(all_rows[3], one[3][pick])


@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 1e9, 1e10, 1e15, 1e20, 1e28, 1e35])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_so_far_from_zero_that_products_round(ds, size, sign):
    """Neighbouring numbers around a maximum whose product with the scale is known to some units,
    or to 2^100, only: differences are taken first."""
    rng = np.random.default_rng(13)
    lift = np.float32(sign * size)
    steps = rng.integers(0, 3, (3, 2000)).astype(np.float32) * np.spacing(np.abs(lift))
    steps[2] *= 1000
    x = dev(lift + steps)
    tokens = some_tokens(rng, 3, 2000)
    idx = check_forward(ds, x, tokens, 4)[3]
    check_backward(ds, x, tokens, idx, 1.0, some_grads(rng, 3, 4))
    check_forward(ds, x.to(torch.bfloat16), tokens, 4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 6])
@pytest.mark.parametrize("mask", [-1e7, -1e9, -1e10, -1e15, -1e20, -1e28])
def test_masks_of_any_size(ds, dtype, rows, mask):
    """A large negative number in all of a slice's first logits, or in all logits, or a mixture."""
    rng = np.random.default_rng(14)
    vocab = 40000
    x = logits(rng, 6, vocab, dtype)
    x[0, :20000] = mask
    x[1, :-1] = mask
    x[2] = mask
    x[3, 1::2] = mask
    x[4, :20000], x[4, 20000:30000], x[4, 30000:] = mask, -float("inf"), mask / 2
    x[5, :30000], x[5, 30000:] = mask, -mask
    tokens = dev(np.array([30000, vocab - 1, 7, 0, 39995, 35000], dtype=np.int32))
    for r in range(0, 6, rows):
        idx = check_forward(ds, x[r:r + rows], tokens[r:r + rows], 3)[3]
        check_backward(ds, x[r:r + rows], tokens[r:r + rows], idx, 1.0, some_grads(rng, rows, 3))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 310])
def test_alternatives_found_one_by_one(ds, dtype, rows):
    """Ever larger logits in the places of 31 threads and none elsewhere: the 32nd of any threads'
    largest is 0, which thousands reach, so that each alternative is swept for.  Beside it the
    same with a NaN at token 0, which comes first, and in a place of the middle."""
    rng = np.random.default_rng(16)
    vocab, each = 102400, 4 if dtype == "fp32" else 8
    base = torch.zeros((vocab // (256 * each), 256, each), device=DEV)
    n = len(base)
    base[:, :31] = 1 + torch.arange(n, device=DEV)[:, None, None] + torch.from_numpy(
        rng.random((n, 31, each), dtype=np.float32)).to(DEV)
    kinds = torch.stack([base.reshape(-1)] * 4).to(DTYPES[dtype])
    kinds[1, 0] = float("nan")
    kinds[2, 50001] = float("nan")
    kinds[3, 0] = kinds[3, 1] = kinds[3, vocab - 1] = float("nan")
    want = [model.order(x.double().cpu().numpy())[:32] for x in kinds]
    for k in (1, 31, 32):
        if rows == 1:
            for kind, ref in zip(kinds, want):
                got = ds.token_logprobs(kind[None], some_tokens(rng, 1, vocab), k)[3].cpu().numpy()
                assert got[0].tolist() == ref[:k].tolist()
            continue
        got = ds.token_logprobs(kinds[torch.arange(rows, device=DEV) % 4], some_tokens(rng, rows, vocab), k)
        got = got[3].cpu().numpy()
        for r in range(rows):
            assert got[r].tolist() == want[r % 4][:k].tolist()


@pytest.mark.parametrize("scale", [2.0 ** -149, 1e9, 1e30, 2.5e38, 3.4e38])
def test_scales_at_the_ends_of_their_range(ds, scale):
    """Logits so that their products with the scale are some units, or nothing."""
    rng = np.random.default_rng(17)
    size = 1.0 if scale < 1 else 3.0 / scale
    x = dev((rng.standard_normal((3, 3001)) * size).astype(np.float32))
    x[1, 5:900] = -float("inf")
    tokens = some_tokens(rng, 3, 3001)
    idx = check_forward(ds, x, tokens, 3, scale)[3]
    check_backward(ds, x, tokens, idx, scale, [g * 0.1 for g in some_grads(rng, 3, 3)])


@pytest.mark.parametrize("lift", [40.7, 60.1, 100.3, 300.3, 500.3, 777.7, 1000.1, -90.6, -1016.9, 1024.3])
def test_gradient_does_not_show_how_lse_is_rounded(ds, lift):
    """Equal logits: p is 1 / vocab = 2^-10, log p = -10 ln 2.  lse is summed again from 64 on,
    relative to the maximum, where it is 10 ln 2 and not off by up to 2^-15 as that of 777.7 is; below,
    half a unit of it in its last place is 2^-19.  Besides, log2 may be off by a unit in the 10, which
    is 0.7 2^-20, and rounding log p, expf and the product by 2^-22 each: together below 2^-18."""
    x = torch.full((2, 1024), lift, device=DEV)
    tokens = dev(np.array([-1, -1], dtype=np.int32))
    _, h, lse, _, _ = ds.token_logprobs(x, tokens)
    got = ds.token_logprobs_backward(x, tokens, lse, h, grad_lse=torch.ones(2, device=DEV))
    assert (got.double() * 1024 - 1).abs().max().item() <= 2.0 ** -18
