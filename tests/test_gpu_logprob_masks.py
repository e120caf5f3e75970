"""Log probabilities of rows whose logits are large beside the rounding of their
products with log2 e: finite mask values of every size, and rows whose maximum
itself is large, against the 64-bit reference and bounds of tests/i8_ref.py."""
import numpy as np
import pytest

import i8_ref
import synth
from test_gpu_logprob import _check, q  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

# what masks become after a division by a temperature, and plain ones
MASKS = (-1e9, -1e9 / 0.33, -1e9 / 0.4, -1e9 / 0.61, -5e9, -1e10, -1e18, -1e20, -1e30)


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("v,shares", [(1000, (0.5, 0.9, 0.99)), (4096, (0.5, 0.9, 0.999)),
                                      (30000, (0.9, 0.9999)), (262144, (0.9,))])
def test_finite_masks(q, v, shares, t):  # noqa: F811
    """Visible logits of ordinary size, the others at a finite mask value."""
    rng = synth.rng("lpfinite", str(v))
    x = rng.normal(size=(len(MASKS) * len(shares), v)) * 2.5
    for i, mask in enumerate(MASKS):
        for j, share in enumerate(shares):
            x[i * len(shares) + j, rng.random(v) < share] = mask
    x[:, v // 3] = 1.25                       # one visible at least
    tokens = np.array([[v // 3, v - 1]] * len(x), np.int32)
    for n_top in (0, 20):
        _check(q, x, t, tokens, n_top)


def test_fully_masked_rows(q):  # noqa: F811
    """Every logit at the mask: the uniform distribution."""
    for v in (700, 20000, 70001):
        x = np.repeat(np.array(MASKS + (-3.4028235e38, -1e4, -65504.0, -1e6, -3e7))[:, None], v, 1)
        out = _check(q, x, "fp32", np.zeros((len(x), 1), np.int32), 5)
        assert (out.top_ids.cpu().numpy() == np.arange(5)).all()


MAXIMA = (1e6, 2.0 ** 23 + 1, 2.0 ** 24 - 1, 2.0 ** 24, 2.0 ** 24 + 2, 3.7e7, 1e8, 1.5e9,
          1509949440.0, 1.86e9, 2.5e9, 3439329280.0, 4e9, 2.0 ** 33, 1e11, 1e20, 3.4e38)


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [5, 1000, 20000, 70001])
def test_large_maxima(q, v, t):  # noqa: F811
    """Rows whose maximum is large, of either sign: alone above the others, a
    few steps above its neighbours, repeated."""
    rng = synth.rng("lplarge", str(v))
    rows = []
    for top in MAXIMA + tuple(-a for a in MAXIMA):
        below = top - abs(top) * rng.random(v) * 0.5
        below[rng.integers(0, v)] = top
        rows.append(below)
        near = np.full(v, top)
        k = rng.integers(1, 40, v)
        rows.append(np.where(rng.random(v) < 0.3, near, near - k * (abs(top) * 2.0 ** -23)))
    x = np.clip(np.array(rows), -3.3e38, 3.3e38)
    tokens = np.array([[0, v - 1]] * len(x), np.int32)
    for n_top in (0, 3):
        _check(q, x, t, tokens, n_top)


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [2000, 50257])
def test_wide_rows(q, v, t):  # noqa: F811
    """Logits spread over both signs, and references that rise by far on the way."""
    rng = synth.rng("lpwide", str(v))
    x = np.empty((8, v))
    x[0] = (rng.random(v) * 2 - 1) * 1e9
    x[1] = np.sort((rng.random(v) * 2 - 1) * 1e9)
    x[2] = np.where(np.arange(v) < v // 2, 3.0e9, 2.0 ** 33)
    x[3] = np.where(np.arange(v) == v - 1, 2.0 ** 33, 3.01e9)
    x[4] = np.where(np.arange(v) < v // 2, -2.5e9, rng.normal(size=v))
    x[5] = np.where(np.arange(v) == v - 2, 0.5, -1.7e9)
    x[6] = np.where(np.arange(v) == v - 2, 1.0e7, -1.0e7)
    x[7] = np.linspace(-2.0 ** 25, -2.0 ** 24 + 3, v)
    tokens = np.array([[v // 2, v - 2]] * 8, np.int32)
    for n_top in (0, 7):
        _check(q, x, t, tokens, n_top)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [1, 40, 1000, 40000])
def test_signs(q, v, t):  # noqa: F811
    """No log probability above 0, no entropy below 0, no log sum exp below the
    largest logit; with one visible token the entropy and its log probability
    are next to 0."""
    rng = synth.rng("lpsigns", str(v))
    x = np.full((400, v), -np.inf)
    at = rng.integers(0, v, 400)
    x[np.arange(400), at] = rng.normal(size=400) * np.exp(rng.normal(size=400) * 2)
    x[0, at[0]] = 0.36999786
    x[100:200][np.isneginf(x[100:200])] = -3e4           # (0 beside the visible one)
    # one token far above the others, and rows of a few equal tokens
    x[200:300] = np.where(np.isneginf(x[200:300]), -20.0, 5.0 + rng.random((100, 1)))
    x[300:] = np.where(rng.random((100, v)) < 0.5, x[300:], rng.normal(size=(100, 1)) * 7)
    out = _check(q, x, t, at[:, None].astype(np.int32), 1)
    top = np.max(x, axis=1)
    import torch
    top = torch.tensor(top).to(i8_ref.torch_type(t)).float().cuda()
    assert bool((out.lse >= top).all())
    assert bool((out.entropy >= 0).all())
    assert bool((out.logprob <= 0).all()) and bool((out.top_logprobs <= 0).all())
