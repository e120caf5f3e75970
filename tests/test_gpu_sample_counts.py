"""How many tokens a row has: stretches whose every vector is finite, with and
without logits after the last vector, and banned tokens at their ends."""
import numpy as np
import pytest

import i8_ref
import synth
from test_gpu_sample import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


# whole stretches (4096 logits of a short row in fp32; parts of 2048 or 4096), one logit more or
# less, a few after the last vector
@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [4095, 4096, 4099, 8192, 32771, 65536, 262144])
def test_kept_of_rows_that_nothing_cuts(q, v, t):
    rng = synth.rng("samplecounts", str(v), t)
    x = rng.normal(size=(8, v))
    x[1, 0] = x[2, v - 1] = -np.inf
    x[3, v // 2:v // 2 + 9] = -np.inf
    x[4, rng.random(v) < 0.5] = -np.inf
    x[5, 1:] = -np.inf
    x[6, :-1] = -np.inf
    x[7, ::8] = -np.inf
    want = [int((r > -np.inf).sum()) for r in x]
    for kw in (dict(), dict(top_k=v), dict(min_p=1e-30), dict(top_p=1.0)):
        out = _check(q, x, t, most_open=1.0, u=rng.random(8), **kw)
        assert out.kept.tolist() == want, kw
