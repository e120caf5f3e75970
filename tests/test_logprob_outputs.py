"""Outputs of logprob_rows that a call does not want."""
import numpy as np
import pytest
import torch

import moe_expert_ffn_q8_amd as q
from test_binding_checks import FakeGpu, f32, u8


@pytest.mark.parametrize("none", [("lse",), ("entropy",), ("lse", "entropy")])
def test_binding_takes_none(none):
    """lse and entropy may be missing; the other checks still run (no GPU: the
    call ends at a workspace of the wrong type)."""
    out = q.LogprobOut(f32(2), f32(2), f32(2), None, None)._replace(**dict.fromkeys(none))
    tokens = FakeGpu(2, torch.int32)
    with pytest.raises(TypeError, match="ws"):
        q.logprob_rows(f32((2, 100)), tokens, ws=f32(64), out=out)
    with pytest.raises(ValueError, match="logprob"):
        q.logprob_rows(f32((2, 100)), tokens, ws=u8(256), out=out._replace(logprob=f32(3)))
    with pytest.raises(ValueError, match="lacks"):
        q.logprob_rows(f32((2, 100)), tokens, ws=u8(256), out=out._replace(logprob=None))


@pytest.mark.gpu
@pytest.mark.parametrize("m,v", [(3, 1000), (2, 70001)])
def test_without_lse_or_entropy(m, v):
    """The outputs that are wanted have the same bits."""
    x = torch.randn(m, v, device="cuda") * 2.5
    tokens = torch.tensor(np.arange(m, dtype=np.int32), device="cuda")
    ws = q.logprob_workspace(m, v, 5, "cuda")
    want = q.logprob_rows(x, tokens, n_top=5, ws=ws)
    for none in (("lse",), ("entropy",), ("lse", "entropy")):
        out = q.logprob_outputs(m, 1, 5, "cuda")._replace(**dict.fromkeys(none))
        got = q.logprob_rows(x, tokens, n_top=5, ws=ws, out=out)
        for name in q.LogprobOut._fields:
            if name not in none:
                assert torch.equal(getattr(got, name), getattr(want, name)), name
