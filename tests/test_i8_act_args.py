"""Arguments of the products with an activation and a residual: strides whose
byte offsets would not fit are refused, and an output type that is asked for is
not replaced by the residual's (without a GPU; the addresses are never read)."""
import pytest
import torch

import moe_expert_ffn_q8_amd as q
from test_binding_checks import FakeGpu, f32
from test_i8_abi import A, BF16, F32, I8, SHAPE, UNSUP, i8


@pytest.mark.parametrize("change,status", [
    (dict(res=A, r_stride=(1 << 32) + 1), UNSUP), (dict(res=A, r_stride=1 << 62), UNSUP),
    (dict(res=A, r_stride=(1 << 63) - 1, y_type=BF16), UNSUP), (dict(y_stride=(1 << 32) + 1), UNSUP),
    (dict(res=A, y_stride=1 << 61), UNSUP), (dict(res=A, r_stride=-(1 << 62)), SHAPE)])
def test_strides_beyond_the_range(change, status):
    a = dict(x=A, x_type=I8, x_stride=64, x_scale=A, w=A, w_stride=64, w_scale=A, bias=None, act=4, res=None,
             r_stride=8, y=A, y_type=F32, y_stride=8, n=8, k=64, m=4, ws=A, ws_bytes=1 << 20)
    a.update(change)
    assert q.raw.i8_matmul_act(*a.values(), None) == status


def test_output_type_asked_for(monkeypatch):
    """A dtype beside a residual of another type is an error; without one y is
    of the residual's type, or fp32."""
    kw = dict(x=i8((4, 64)), w=i8((6, 64)), w_scale=f32(6), x_scale=f32(4))
    bf16 = FakeGpu((4, 6), torch.bfloat16)
    made = []

    real = torch.empty

    def empty(shape, dtype=None, device=None):
        if device is None:
            return real(shape, dtype=dtype)
        made.append(dtype)
        return FakeGpu(shape, dtype)

    monkeypatch.setattr(q._lib.torch, "empty", empty)
    for t in (torch.float32, torch.float16):
        with pytest.raises(TypeError, match="residual"):
            q.i8_matmul_act(**kw, residual=bf16, dtype=t)
    # (a bias of a wrong length ends the call after y is made, before the library)
    for extra, want in ((dict(residual=bf16), torch.bfloat16), (dict(residual=bf16, dtype=torch.bfloat16), torch.bfloat16),
                        (dict(), torch.float32), (dict(dtype=torch.float16), torch.float16)):
        del made[:]
        with pytest.raises(ValueError, match="bias"):
            q.i8_matmul_act(**kw, bias=f32(5), **extra)
        assert made == [want], extra
