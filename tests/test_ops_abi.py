"""Argument checks of the operators around the products of a token step: every
bad argument is refused on the host, by the C ABI with its documented status
and by the binding with an exception, before any pointer is used (these run
without a GPU; the addresses are never read)."""
import pytest
import torch

import moe_expert_ffn_q8_amd as q
from test_binding_checks import FakeGpu, f32, i32, u8
from test_i8_abi import A, ALIGN, BF16, F16, F32, I8, NULL, OK, PRODUCT, SHAPE, UNSUP, WS, Strided, i8

lib = q.raw


@pytest.mark.parametrize("change,status", PRODUCT + [
    (dict(bias=A + 2), ALIGN), (dict(act=-1), UNSUP), (dict(act=6), UNSUP),
    (dict(res=A + 2), ALIGN), (dict(res=A + 1, y_type=BF16), ALIGN), (dict(res=A, r_stride=7), SHAPE)])
def test_act_status(change, status):
    a = dict(x=A, x_type=I8, x_stride=64, x_scale=A, w=A, w_stride=64, w_scale=A, bias=None, act=4, res=None,
             r_stride=8, y=A, y_type=F32, y_stride=8, n=8, k=64, m=4, ws=A, ws_bytes=1 << 20)
    a.update(change)
    assert lib.i8_matmul_act(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(type=I8, k=65), SHAPE),
    (dict(m=(1 << 27) + 1), UNSUP), (dict(n=1 << 31), UNSUP), (dict(k=(1 << 20) + 1, stride=1 << 21, y_stride=1 << 21), UNSUP),
    (dict(type=4), UNSUP), (dict(type=-1), UNSUP), (dict(y_type=I8), UNSUP), (dict(m=0, table=None), OK),
    (dict(table=None), NULL), (dict(tokens=None), NULL), (dict(y=None), NULL), (dict(type=I8, scale=None), NULL),
    (dict(stride=63), SHAPE), (dict(y_stride=63), SHAPE), (dict(stride=(1 << 32) + 64), UNSUP),
    (dict(table=A + 2), ALIGN), (dict(table=A + 1, type=F16), ALIGN), (dict(type=I8, table=A + 8), ALIGN),
    (dict(type=I8, stride=72), ALIGN), (dict(type=I8, scale=A + 2), ALIGN), (dict(tokens=A + 2), ALIGN),
    (dict(y=A + 2), ALIGN), (dict(y=A + 1, y_type=BF16), ALIGN)])
def test_embed_status(change, status):
    a = dict(table=A, type=F32, stride=64, scale=A, tokens=A, by=1.0, y=A, y_type=F32, y_stride=64, m=4, n=9, k=64)
    a.update(change)
    assert lib.embed_rows(*a.values(), None) == status


@pytest.mark.parametrize("r8", [0, 1])
@pytest.mark.parametrize("change,status", [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=48), SHAPE), (dict(k=0), SHAPE), (dict(m=0, w=None), OK),
    (dict(w=None), NULL), (dict(tokens=None), NULL), (dict(y=None), NULL), (dict(w=A + 2), ALIGN),
    (dict(tokens=A + 1), ALIGN), (dict(y=A + 2), ALIGN), (dict(y_stride=32), SHAPE), (dict(y_type=3), UNSUP),
    (dict(k=(1 << 20) + 32, y_stride=1 << 21), UNSUP)])
def test_q8_0_embed_status(change, status, r8):
    a = dict(w=A, r8=r8, tokens=A, by=1.0, y=A, y_type=F32, y_stride=64, m=4, n=9, k=64)
    a.update(change)
    assert lib.q8_0_embed_rows(*a.values(), None) == status


NORM = [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(y_type=I8, n=48), SHAPE), (dict(n=65537, x_row_stride=1 << 17), UNSUP),
    (dict(m=(1 << 27) + 1), UNSUP), (dict(x_type=I8), UNSUP), (dict(y_type=4), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(eps=float("nan")), UNSUP), (dict(eps=float("inf")), UNSUP), (dict(m=0, x=None), OK),
    (dict(x=None), NULL), (dict(weight=None), NULL), (dict(y=None), NULL), (dict(y_type=I8, y_scale=None), NULL),
    (dict(x_row_stride=63), SHAPE), (dict(y_row_stride=63), SHAPE), (dict(x=A + 2), ALIGN), (dict(y=A + 2), ALIGN),
    (dict(weight=A + 2), ALIGN), (dict(bias=A + 2), ALIGN), (dict(y_type=I8, y=A + 8), ALIGN),
    (dict(y_type=I8, y_row_stride=72), ALIGN), (dict(y_type=I8, y_scale=A + 2), ALIGN),
    (dict(x_row_stride=(1 << 32) + 64), UNSUP)]


@pytest.mark.parametrize("change,status", NORM)
def test_norm_status(change, status):
    a = dict(x=A, x_type=F32, x_row_stride=64, weight=A, bias=None, eps=1e-5, layer=0, y=A, y_type=F32,
             y_row_stride=64, y_scale=A, m=4, n=64)
    a.update(change)
    assert lib.norm_rows(*a.values(), None) == status


@pytest.mark.parametrize("change,status", NORM + [
    (dict(residual=None), NULL), (dict(residual_out=None), NULL), (dict(post_bias=A), NULL),
    (dict(residual_type=I8), UNSUP), (dict(gate=A, gate_type=I8), UNSUP), (dict(residual=A + 2), ALIGN),
    (dict(residual_out=A + 2), ALIGN), (dict(residual_row_stride=60), SHAPE), (dict(residual_out_row_stride=60), SHAPE),
    (dict(gate=A, gate_row_stride=60), SHAPE), (dict(gate=A, gate_row_stride=-64), SHAPE), (dict(gate=A + 2), ALIGN),
    (dict(post_weight=A + 2), ALIGN), (dict(post_weight=A, post_bias=A + 1), ALIGN)])
def test_residual_norm_status(change, status):
    a = dict(x=A, residual=A, residual_out=A, weight=A, y=A, y_scale=A, x_row_stride=64, residual_row_stride=64,
             residual_out_row_stride=64, y_row_stride=64, residual_scale=1.0, eps=1e-5)
    m, n = change.get("m", 4), change.get("n", 64)
    a.update({k: v for k, v in change.items() if k not in ("m", "n")})
    assert lib.residual_norm_rows(q.ResidualNormDesc(**a), m, n, None) == status


def test_residual_norm_without_desc():
    assert lib.residual_norm_rows(None, 1, 64, None) == NULL


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), SHAPE), (dict(v=0), SHAPE), (dict(v=(1 << 24) + 1, stride=1 << 25), UNSUP), (dict(m=(1 << 23) + 1), UNSUP),
    (dict(type=I8), UNSUP), (dict(type=-1), UNSUP), (dict(m=0, logits=None), OK), (dict(stride=99), SHAPE),
    (dict(logits=None), NULL), (dict(u=None), NULL), (dict(ids=None), NULL), (dict(logprob=None), NULL),
    (dict(kept=None), NULL), (dict(logits=A + 2), ALIGN), (dict(logits=A + 1, type=F16), ALIGN), (dict(u=A + 1), ALIGN),
    (dict(temperature=A + 2), ALIGN), (dict(top_k=A + 2), ALIGN), (dict(top_p=A + 2), ALIGN), (dict(min_p=A + 2), ALIGN),
    (dict(ids=A + 2), ALIGN), (dict(logprob=A + 2), ALIGN), (dict(kept=A + 2), ALIGN), (dict(ws=A + 64), ALIGN),
    (dict(ws=None), WS), (dict(ws_bytes=0), WS), (dict(stride=(1 << 32) + 1), UNSUP)])
def test_sample_status(change, status):
    a = dict(logits=A, type=F32, stride=100, u=A, temperature=None, top_k=None, top_p=None, min_p=None, ids=A, logprob=A,
             kept=A, m=2, v=100, ws=A, ws_bytes=1 << 30)
    a.update(change)
    assert lib.sample_rows(*a.values(), None) == status


def test_sample_workspace_bytes():
    assert lib.sample_workspace_bytes(0, 10) >= 256
    for m, v in ((1, 10), (8, 262144), (512, 50257)):
        assert 0 < lib.sample_workspace_bytes(m, v) < 1 << 31
    for m, v in ((-1, 10), (1, 0), (1, (1 << 24) + 1), ((1 << 23) + 1, 10)):
        assert lib.sample_workspace_bytes(m, v) == 0


def test_a_workspace_serves_smaller_calls():
    """Room made for m rows of n logits is enough for fewer of either, of any
    type."""
    need = lambda m, v: q.sample_workspace_bytes(m, v)
    for m in (1, 2, 7, 64, 511, 512, 513, 2048, 2049, 5000):
        for v in (10, 4096, 4097, 32000, 65536, 262144, 1 << 24):
            assert all(need(a, b) <= need(m, v) for a in {1, m // 2, max(1, m - 1)} - {0} for b in {1, v // 2, v - 1, v})


# --- the binding -------------------------------------------------------------

def _bad(fn, ok, exc, match, **kw):
    with pytest.raises(exc, match=match):
        fn(**{**ok, **kw})


def test_binding_act():
    ok = dict(x=i8((4, 64)), w=i8((6, 64)), w_scale=f32(6), x_scale=f32(4), y=f32((4, 6)), residual=f32((4, 6)))
    bad = lambda *a, **kw: _bad(q.i8_matmul_act, ok, *a, **kw)
    bad(ValueError, "act: 'tanh'", act="tanh")
    bad(ValueError, "residual: shape", residual=f32((4, 7)))
    bad(TypeError, "residual", residual=FakeGpu((4, 6), torch.bfloat16))
    bad(TypeError, "residual", residual=i8((4, 6)))
    bad(ValueError, "several devices", residual=f32((4, 6), 1))
    bad(ValueError, "rows must be contiguous", residual=Strided((4, 6), torch.float32))
    bad(ValueError, "bias", bias=f32(5))


def test_binding_embed():
    ok = dict(table=f32((9, 64)), tokens=i32(4), y=f32((4, 64)))
    bad = lambda *a, **kw: _bad(q.embed_rows, ok, *a, **kw)
    bad(TypeError, "tokens", tokens=FakeGpu(4, torch.int64))
    bad(ValueError, "tokens", tokens=i32((4, 1)))
    bad(ValueError, "y: shape", y=f32((4, 63)))
    bad(ValueError, "y: shape", tokens=i32(3))
    bad(TypeError, "y:", y=i8((4, 64)))
    bad(TypeError, "table:", table=FakeGpu((9, 64), torch.float64))
    bad(ValueError, "table_scale", table=i8((9, 64)))
    bad(ValueError, "table_scale", table=i8((9, 64)), table_scale=f32(8))
    bad(ValueError, "table_scale", table_scale=f32(9))
    bad(ValueError, "several devices", tokens=i32(4, 1))
    ok = dict(w=u8(9 * 2 * 34), tokens=i32(4), n=9, k=64, y=f32((4, 64)))
    bad = lambda *a, **kw: _bad(q.q8_0_embed_rows, ok, *a, **kw)
    bad(ValueError, "w: the shape", n=10)
    bad(ValueError, "w: the shape", r8=True)
    bad(ValueError, "several devices", y=f32((4, 64), 1))


def test_binding_norm():
    ok = dict(x=f32((4, 64)), weight=f32(64), y=f32((4, 64)))
    bad = lambda *a, **kw: _bad(q.norm_rows, ok, *a, **kw)
    bad(TypeError, "x:", x=i8((4, 64)))
    bad(ValueError, "weight", weight=f32(63))
    bad(TypeError, "weight", weight=FakeGpu(64, torch.bfloat16))
    bad(ValueError, "bias", bias=f32(65))
    bad(ValueError, "y: shape", y=f32((4, 65)))
    bad(ValueError, "y_scale", y_scale=f32(4))
    bad(ValueError, "y_scale", y=i8((4, 64)), y_scale=f32(5))
    bad(ValueError, "several devices", weight=f32(64, 1))
    ok.update(residual=f32((4, 64)), residual_out=f32((4, 64)))
    bad = lambda *a, **kw: _bad(q.residual_norm_rows, ok, *a, **kw)
    bad(ValueError, "residual: shape", residual=f32((4, 63)))
    bad(TypeError, "residual_out", residual_out=FakeGpu((4, 64), torch.float16))
    bad(ValueError, "residual_out: shape", residual_out=f32((5, 64)))
    bad(ValueError, "gate", gate=f32(63))
    bad(ValueError, "gate: shape", gate=f32((3, 64)))
    bad(TypeError, "gate", gate=i32(64))
    bad(ValueError, "post_weight", post_weight=f32(2))
    bad(ValueError, "post_bias", post_bias=f32(64))
    bad(ValueError, "several devices", gate=f32((4, 64), 1))


def test_binding_sample():
    ok = dict(logits=f32((2, 100)), u=f32(2), ws=u8(1 << 20), out=q.SampleOut(i32(2), f32(2), i32(2)))
    bad = lambda *a, **kw: _bad(q.sample_rows, ok, *a, **kw)
    bad(TypeError, "logits", logits=i8((2, 100)))
    bad(ValueError, "u:", u=f32(3))
    bad(TypeError, "u", u=FakeGpu(2, torch.float64))
    bad(ValueError, "temperature", temperature=f32(1))
    bad(TypeError, "top_k", top_k=f32(2))
    bad(ValueError, "top_p", top_p=f32(5))
    bad(ValueError, "min_p", min_p=f32(5))
    bad(ValueError, "ids", out=q.SampleOut(i32(3), f32(2), i32(2)))
    bad(TypeError, "kept", out=q.SampleOut(i32(2), f32(2), f32(2)))
    bad(ValueError, "several devices", ws=u8(1 << 20, 1))
    with pytest.raises(q.Q8Error):
        q.sample_workspace(2, 0, "cpu")
