"""Sampling from rows whose finite logits lie further apart than fp32's range
(masks of either sign near the type's ends), at temperatures that give such
logits weight, infinity among them, against the definition by sorting
(tests/ops_ref.py)."""
import numpy as np
import pytest

import synth
from test_gpu_sample import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


def _rows(rng, v, end):
    i = np.arange(v)
    return np.stack([np.where(i % 2, 0.88 * end, -0.88 * end),         # halves
                     np.where(i % 50, 0.88 * end, -0.88 * end),        # few far ones: a list holds them
                     np.where(rng.random(v) < 0.5, end, -end),         # the ends themselves
                     rng.uniform(-1, 1, v) * end,                      # all over the range
                     np.where(rng.random(v) < 0.6, -end, rng.normal(size=v) * 3)])


# head and tail of the order: targets among the far logits too
HEADS = [dict(), dict(top_p=0.9), dict(min_p=0.05), "most", "half"]


@pytest.mark.parametrize("temperature", [8e36, 3e37, 1e38, 3.4e38, np.inf])
@pytest.mark.parametrize("t,v", [("fp32", 1000), ("fp32", 20000), ("bf16", 4096), ("bf16", 50257), ("bf16", 262144)])
def test_logits_further_apart_than_the_range(q, t, v, temperature):
    rng = synth.rng("samplefar", t, str(v), str(temperature))
    x = _rows(rng, v, 3.4028234e38 if t == "fp32" else 3.3895314e38)
    for head in HEADS:
        kw = {"most": dict(top_k=v - 7), "half": dict(top_k=v // 2 + 9, top_p=0.99)}[head] if isinstance(head, str) else head
        _check(q, x, t, most_open=1.0, u=np.array([0.03, 0.5, 0.9, 0.99, 1 - 2.0 ** -24]), temperature=temperature, **kw)


@pytest.mark.parametrize("t,v", [("fp32", 3000), ("bf16", 50257)])
def test_infinite_temperature_and_masks(q, t, v):
    """Every token that -infinity does not ban weighs the same."""
    rng = synth.rng("samplefarmask", t, str(v))
    x = rng.normal(size=(3, v)) * 2
    x[0, rng.random(v) < 0.3] = -np.inf
    x[1, 5:] = -np.inf
    out = _check(q, x, t, u=[0.2, 0.7, 0.95], temperature=np.inf)
    assert out.kept.tolist() == [int((r > -np.inf).sum()) for r in x]
