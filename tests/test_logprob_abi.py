"""include/ds_logprob.h: declared and exported functions agree, argument checks answer before any
CUDA call, and the 64-bit model's gradient is that of its forward pass (CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest

import oracle.logprob as model
import top_selection_deepselect_gb300 as ds

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: these calls fail their checks first
EINVAL, EUNSUP = ds.DS_EINVAL, ds.DS_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    ds.build()
    return ds.load_library()


def test_header_and_binding_agree(lib):
    with open(os.path.join(ROOT, "include", "ds_logprob.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ds_\w+)\s*\(", text, flags=re.M)
    assert sorted(set(names)) == sorted(ds.LOGPROB_ENTRY_POINTS)
    for name in names:
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
        assert callable(getattr(ds, name))


def status_of(call, **kw):
    try:
        call(**kw)
    except ds.DSError as e:
        assert ds.ds_last_error_detail()
        return e.status
    return ds.DS_OK


FORWARD = dict(logits=FAKE, dtype=ds.DS_BF16, rows=2, vocab=100, row_stride=100, tokens=FAKE, k=4, scale=1.0,
               logprob=FAKE, entropy=FAKE, lse=FAKE, idx=FAKE, top=FAKE, stream=None)
BACKWARD = dict(logits=FAKE, dtype=ds.DS_BF16, rows=2, vocab=100, row_stride=100, tokens=FAKE, k=4, idx=FAKE,
                scale=1.0, lse=FAKE, entropy=FAKE, grad_logprob=FAKE, grad_entropy=FAKE, grad_lse=FAKE,
                grad_top=FAKE, grad=FAKE, grad_stride=100, stream=None)
BOTH = [(dict(dtype=3), EUNSUP), (dict(dtype=-1), EUNSUP), (dict(rows=-1), EINVAL), (dict(vocab=0), EINVAL),
        (dict(vocab=1 << 31, row_stride=1 << 31, grad_stride=1 << 31), EUNSUP), (dict(rows=1 << 27), EUNSUP),
        (dict(row_stride=99), EINVAL), (dict(k=-1), EINVAL), (dict(k=33), EUNSUP),
        (dict(k=4, vocab=3), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
        (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(logits=None), EINVAL),
        (dict(logits=FAKE + 1), EINVAL), (dict(tokens=None), EINVAL), (dict(lse=None), EINVAL),
        (dict(entropy=None), EINVAL), (dict(idx=None), EINVAL)]


@pytest.mark.parametrize("change,status", BOTH + [(dict(logprob=None), EINVAL), (dict(top=None), EINVAL)])
def test_forward_refuses(lib, change, status):
    args = {n: change.get(n, v) for n, v in FORWARD.items()}
    assert status_of(ds.ds_token_logprobs, **args) == status


@pytest.mark.parametrize("change,status", BOTH + [(dict(grad=None), EINVAL), (dict(grad=FAKE + 1), EINVAL),
                                                  (dict(grad_stride=99), EINVAL)])
def test_backward_refuses(lib, change, status):
    args = {n: change.get(n, v) for n, v in BACKWARD.items()}
    assert status_of(ds.ds_token_logprobs_backward, **args) == status


def test_no_rows_is_nothing_to_do(lib):
    assert status_of(ds.ds_token_logprobs, **{**FORWARD, "rows": 0, "logits": None, "tokens": None}) == ds.DS_OK
    assert status_of(ds.ds_token_logprobs_backward, **{**BACKWARD, "rows": 0, "grad": None}) == ds.DS_OK


def test_models_gradient_is_its_differences():
    """Central differences in 64 bits: error about step^2 times a third derivative of size one, and
    2^-52 over the step: 1e-9 covers both at a step of 1e-5."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 9)) * 2
    x[1, 3] = -np.inf
    x[3] = -np.inf
    tokens, idx = np.array([2, 5, -1, 1]), np.array([[0, 2, 0], [4, -1, 8], [1, 2, 3], [0, 1, 2]])
    g = [rng.standard_normal(4) for _ in range(3)] + [rng.standard_normal((4, 3))]

    def value(x):
        lp, h, lse, _, _ = model.forward(x, tokens, 0, 0.7)
        total = 0.0
        for r in range(3):
            total += g[0][r] * lp[r] + g[1][r] * h[r] + g[2][r] * lse[r]
            total += sum(w * (0.7 * x[r, i] - lse[r]) for i, w in zip(idx[r], g[3][r]) if i >= 0)
        return total

    got = model.backward(x, tokens, idx, 0.7, *g)
    assert not got[3].any()
    for r, i in np.ndindex(3, 9):
        if np.isneginf(x[r, i]):
            assert got[r, i] == 0
            continue
        up, down = x.copy(), x.copy()
        up[r, i] += 1e-5
        down[r, i] -= 1e-5
        assert abs((value(up) - value(down)) / 2e-5 - got[r, i]) < 1e-9


def test_model_by_hand():
    """Probabilities 1/2, 1/4, 1/4 and a token that cannot come."""
    x = np.array(
        [[np.log(0.25), np.log(0.5), -np.inf, np.log(0.25)]])
    lp, h, lse, idx, top = model.forward(x, np.array([1]), 4, 1.0)
    assert np.allclose([lp[0], h[0], lse[0]], [-np.log(2), 1.5 * np.log(2), 0.0], atol=1e-15)
    assert idx.tolist() == [[1, 0, 3, 2]]
    assert np.allclose(top[0, :3], [-np.log(2), -np.log(4), -np.log(4)]) and np.isneginf(top[0, 3])
    assert model.order([1.0, np.nan, -0.0, 0.0, np.inf]).tolist() == [1, 4, 0, 2, 3]
