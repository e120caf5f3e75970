"""Norms of 16-bit rows computed in 32 bits where those are short: a value far
above a row's spread, rows at the ends of bfloat16's range, against the 64-bit
reference."""
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


N_RANGE = [1, 5, 100, 505, 900, 2040, 4096, 8200, 20000, 65536]


@pytest.mark.parametrize("size", [2e-40, 1e-39, 4e-39, 3e-38, 1e36, 1e37, 3e37, 8e37])
@pytest.mark.parametrize("layer", [False, True])
def test_ends_of_bfloat16(q, size, layer):
    """Subnormal rows without an eps, and rows whose differences, or the sums of
    them, leave 32 bits."""
    rng = synth.rng("normends", str(size), str(layer))
    for n in N_RANGE[layer:]:
        x = np.clip(rng.normal(size=(3, n)) * size, -3.38e38, 3.38e38)
        x[:, 0] = size                                         # (no row of zeros)
        _check(q, x, "bf16", 0.0, layer, (size, n), rng=rng)


@pytest.mark.parametrize("n", N_RANGE[1:])
def test_largest_bfloat16_values(q, n):
    """Values at the end itself, of either sign: one among the others' negatives,
    halves, all but one alike."""
    rng = synth.rng("normlargest", str(n))
    big = 3.3895314e38
    x = np.full((4, n), -big)
    x[0, n // 2] = big
    x[1, : n // 2] = big
    x[2, 1:] = big
    x[3] = rng.uniform(-1, 1, n) * big
    for layer in (False, True):
        _check(q, x, "bf16", 0.0, layer, (n, layer), bias=_vec(rng, n, 0.1, 0.0), rng=rng)


@pytest.mark.parametrize("size", [1e-39, 1e38])
@pytest.mark.parametrize("n", [100, 900, 4096, 9000])
def test_ends_in_the_norm_after_a_block(q, n, size):
    """post_weight's norm of such rows, into an ordinary stream, gated."""
    rng = synth.rng("normpostends", str(n), str(size))
    for layer in (False, True):
        x = np.clip(rng.normal(size=(3, n)) * size, -3.38e38, 3.38e38)
        g = to_gpu(x.astype(np.float32)).bfloat16()
        r = to_gpu(rng.normal(size=(3, n)).astype(np.float32)).bfloat16()
        pw, w, gate = _vec(rng, n), _vec(rng, n), _vec(rng, n, 0.1, 0.5)
        import torch
        out = q.residual_norm_rows(g, r, to_gpu(w), post_weight=to_gpu(pw), gate=to_gpu(gate), eps=0.0, layer=layer,
                                   dtype=torch.bfloat16)
        a, b = _norm(g.double().cpu().numpy(), pw.astype(np.float64), None, 0.0, layer)
        rv, gv = r.double().cpu().numpy(), gate.astype(np.float64)
        ops_ref.assert_rounded(out.residual.double().cpu().numpy(), gv * a + rv,
                               np.abs(gv) * b + (3 * U + ops_ref.REL64) * (np.abs(gv * a) + np.abs(rv)), "bf16", "residual")
        value, bound = _norm(out.residual.double().cpu().numpy(), w.astype(np.float64), None, 0.0, layer)
        ops_ref.assert_rounded(out.y.double().cpu().numpy(), value, bound, "bf16", "y")
