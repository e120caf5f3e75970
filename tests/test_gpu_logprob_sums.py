"""Sums of logprob_rows within the roundings of the additions that the kernel
makes, and rows in which one logit left out or taken twice shows."""
import numpy as np
import pytest

import i8_ref
import synth
from gpu_cases import to_gpu
from test_gpu_logprob import _run, q  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def test_equal_terms(q):  # noqa: F811
    """A chain of equal terms rounds to one side.  512 rows are not cut into
    parts: a lane of 256 has 1024 of 262144 fp32 logits, 16 a turn.  Each lane
    gets one logit c above the others, so that their terms are exp(-c) = 2^-1 (1 +
    0.55 * 2^-14): added one by one, those beyond sums of 2^8 would each round up
    by 0.45 * 2^-14, 1.3e-5 of the sum of the row.

    The bound: 16 additions of a turn, 64 of turns, 6 in a wave and 4 of waves, a
    move of the reference per turn that changes nothing; (|d| + 3) 2u of each
    term, |d| < 1.  lse: that, 3u of log S and u of its own; entropy: the sums'
    error at most twice, times 1 + |W / S|, and the roundings of log S and W / S."""
    import torch
    m, v = 512, 262144
    c = np.float32(np.log(2.0) - np.log1p(0.55 * 2.0 ** -14))
    row = np.zeros(v, np.float32)
    row[:1024] = c
    logits = to_gpu(row).expand(m, v).contiguous()
    out = q.logprob_rows(logits, n_top=0, ws=q.logprob_workspace(m, v, 0, "cuda"))
    d = row.astype(np.float64) - float(c)
    s = np.exp(d).sum()
    lse = float(c) + np.log(s)
    mean = (np.exp(d) * d).sum() / s
    rel = i8_ref.U * (16 + 64 + 6 + 4 + 2 * (1 + 3))
    assert rel < 6e-6                              # the fault above is twice this
    tol = 1.01 * (rel + 4 * i8_ref.U * lse)
    assert float((out.lse.double() - lse).abs().max()) <= tol
    tol = 1.01 * (2 * rel * (1 + abs(mean)) + 4 * i8_ref.U * (np.log(s) + abs(mean)))
    assert float((out.entropy.double() - (np.log(s) - mean)).abs().max()) <= tol
    assert torch.equal(out.lse, out.lse[:1].expand(m))


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 2), (7, 1), (3, 5)])
@pytest.mark.parametrize("m,v", [(7, 13), (7, 1003), (7, 16384), (7, 50257), (7, 262144), (1, 262143),
                                 (520, 5003)])
def test_every_logit_counts_once(q, m, v, offset, pad, t):  # noqa: F811
    """Logits of 0 among -infinity: S is their number, exactly.  lse = entropy =
    log S, off by 1 ulp of log2, the constant's and the product's rounding: 4u of
    it, less than one logit in 262144 (3.8e-6) makes."""
    rng = synth.rng("lpcount", str(v))
    i = np.arange(v)
    parts = 1 if m >= 512 else max(1, min(1024 // m, v // 16384, 64))
    size = -(-v // parts)
    size = -(-size // 8) * 8
    kinds = [i >= 0, (i < 20) | (i >= v - 20),                     # all; both ends
             (i % size < 9) | (i % size >= size - 9),              # both sides of every part
             rng.random(v) < 0.5, i % 2 == 0, i % 8 == 7,
             (i % 1024 < 9) | (i % 1024 >= 1015)]                  # both sides of a wave's loads
    x = np.stack([np.where(kinds[j % len(kinds)], 0.0, -np.inf) for j in range(m)])
    out, _ = _run(q, x, t, None, min(v, 3), offset=offset, pad=pad)
    n = (x == 0).sum(axis=1)
    tol = 4 * i8_ref.U * np.log(n)
    assert ((1.0 / n > tol)).all()
    for got in (out.lse, out.entropy):
        err = np.abs(got.double().cpu().numpy() - np.log(n))
        assert (err <= tol).all(), (m, v, np.argwhere(err > tol).ravel()[:4])
