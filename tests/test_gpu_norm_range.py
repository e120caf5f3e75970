"""Norms of 16-bit rows computed in 32 bits where those are short: a value far
above a row's spread, against the 64-bit reference."""
import numpy as np
import pytest

import i8_ref
import ops_ref
import synth
from gpu_cases import to_gpu
from i8_ref import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


def _norm(x, weight, bias, eps, layer):
    """(value, bound): with p the mean in 32 bits and q what is left of it, d = (x -
    p) - q takes two roundings of |d| + U |mean| and |d|, and q one of U |mean|;
    squares, their root and three products 71 u, as in ops_ref; means and sums
    over threads are in 64 bits."""
    value, b = ops_ref.norm(x, weight, bias, eps, layer)       # (b: the 64-bit arithmetic)
    mean = x.mean(axis=1, keepdims=True) if layer else np.zeros((len(x), 1))
    d = x - mean
    r = np.abs(weight) / np.sqrt((d * d).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    return value, b + 1.01 * U * (73 * np.abs(d) * r + 2 * U * np.abs(mean) * r + np.abs(value) * (bias is not None))


def _vec(rng, n, size=0.2, middle=1.0):
    return (rng.normal(size=n) * size + middle).astype(np.float32)


def _check(q, x, t, eps, layer, what, bias=None, rng=None):
    """Rows x (numpy), as t holds them."""
    g = to_gpu(x.astype(np.float32)).to(i8_ref.torch_type(t))
    w = _vec(rng, x.shape[1])
    out = q.norm_rows(g, to_gpu(w), bias=None if bias is None else to_gpu(bias), eps=eps, layer=layer,
                      dtype=i8_ref.torch_type(t))
    value, bound = _norm(g.double().cpu().numpy(), w.astype(np.float64),
                         None if bias is None else bias.astype(np.float64), eps, layer)
    ops_ref.assert_rounded(out.y.double().cpu().numpy(), value, bound, t, what)


@pytest.mark.parametrize("n", [5, 64, 500, 1003, 2048, 4096, 8192, 14336, 40000])
@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_outlier_channels(q, t, n):
    """One value of 3000, or two of either sign, before others of about 1: the
    others keep their bits."""
    rng = synth.rng("normoutlier", t, str(n))
    x = rng.normal(size=(24, n))
    for i in range(24):
        at = 8 * rng.integers(0, (n + 7) // 8)                 # the first of eight neighbours
        x[i, at] = 3000.0
        if i % 2:
            x[i, (at + n // 2) % n] = -3000.0
    for layer in (False, True):
        _check(q, x, t, 1e-5, layer, (n, layer), rng=rng)
    _check(q, x + 100.0, t, 1e-5, True, (n, "far"), bias=_vec(rng, n, 0.1, 0.0), rng=rng)
