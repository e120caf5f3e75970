"""Arguments of the products with an activation and a residual: strides whose
byte offsets would not fit are refused (without a GPU; the addresses are never
read)."""
import pytest

import moe_expert_ffn_q8_amd as q
from test_i8_abi import A, BF16, F32, I8, SHAPE, UNSUP


@pytest.mark.parametrize("change,status", [
    (dict(res=A, r_stride=(1 << 32) + 1), UNSUP), (dict(res=A, r_stride=1 << 62), UNSUP),
    (dict(res=A, r_stride=(1 << 63) - 1, y_type=BF16), UNSUP), (dict(y_stride=(1 << 32) + 1), UNSUP),
    (dict(res=A, y_stride=1 << 61), UNSUP), (dict(res=A, r_stride=-(1 << 62)), SHAPE)])
def test_strides_beyond_the_range(change, status):
    a = dict(x=A, x_type=I8, x_stride=64, x_scale=A, w=A, w_stride=64, w_scale=A, bias=None, act=4, res=None,
             r_stride=8, y=A, y_type=F32, y_stride=8, n=8, k=64, m=4, ws=A, ws_bytes=1 << 20)
    a.update(change)
    assert q.raw.i8_matmul_act(*a.values(), None) == status
