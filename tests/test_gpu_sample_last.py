"""u of 1 and above: the last kept token that has mass, in rows that nothing
cuts and whose tail weighs a few units of 2^-52 of the largest weight."""
import numpy as np
import pytest

import synth
from test_gpu_sample import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


def _heads(n):
    """fp32 logits of weights near 2^-20 whose whole units of 2^-52 are above
    them by 0.4 to 0.45 of a unit (the library's weight is off by 1e-4 of one)."""
    x = np.arange(np.float32(-13.86), np.float32(-13.83), np.float32(2.0 ** -20), dtype=np.float32)
    units = np.exp(x.astype(np.longdouble)) * 2.0 ** 52
    up = np.ceil(units) - units
    return x[(up > 0.4) & (up < 0.45)][:n]


@pytest.mark.parametrize("m", [1, 8])
def test_last_token_with_mass(q, m):
    """The listed tokens' units are 16 more than their weights, the tail's three
    are not listed: sums in floating point end before the tail."""
    rng = synth.rng("samplelast", str(m))
    v = 50257
    heads = _heads(40)
    assert len(heads) == 40
    x = np.full((m, v), -np.inf, np.float32)
    x[:, 0] = 0.0
    x[:, 4:164:4] = heads
    tail = np.sort(rng.choice(np.arange(30000, v), (m, 5), replace=False), axis=1)
    for i in range(m):
        x[i, tail[i, :3]] = np.float32(-52 * np.log(2.0))      # a unit each: the last by its index
        x[i, tail[i, 3:]] = -50.0                              # none
    for u in (1.0, 1.5, np.inf):
        out, _, _ = _run(q, x, "fp32", u=u)
        assert out.ids.tolist() == tail[:, 2].tolist()
        assert out.kept.tolist() == [46] * m


def test_last_token_of_a_listed_row(q):
    """The same where the list holds the whole row."""
    x = np.full((2, 50257), -np.inf, np.float32)
    x[:, 0] = 0.0
    x[:, 400] = np.float32(-52 * np.log(2.0))
    x[:, 40000] = -60.0
    out, _, _ = _run(q, x, "fp32", u=1.0)
    assert out.ids.tolist() == [400, 400] and out.kept.tolist() == [3, 3]
