"""Argument checks of the 8-bit products with token and channel scales and of
the log probabilities: every bad argument is refused on the host, by the C ABI
with its documented status and by the binding with an exception, before any
pointer is used (these run without a GPU; the addresses are never read)."""
import pytest
import torch

import moe_expert_ffn_q8_amd as q
from test_binding_checks import FakeGpu, f32, i32, u8

OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4, -5
A = 1 << 20
F32, F16, BF16, I8 = 0, 1, 2, 3
lib = q.raw


def i8(shape, dev=0):
    return FakeGpu(shape, torch.int8, dev)


@pytest.mark.parametrize("change,status", [
    (dict(k=33), SHAPE), (dict(k=0), SHAPE), (dict(k=-32), SHAPE), (dict(k=131072), UNSUP),
    (dict(n_rows=-1), SHAPE), (dict(n_rows=0, x=None), OK), (dict(n_rows=(1 << 27) + 1), UNSUP),
    (dict(x_type=3), UNSUP), (dict(x_type=-1), UNSUP), (dict(x_type=4), UNSUP),
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(scale=None), NULL),
    (dict(x_stride=32), SHAPE), (dict(q_stride=32), SHAPE),
    (dict(x=A + 4), ALIGN), (dict(q=A + 8), ALIGN), (dict(scale=A + 2), ALIGN),
    (dict(x_stride=66), ALIGN), (dict(x_type=F16, x_stride=68), ALIGN), (dict(q_stride=72), ALIGN),
    (dict(x_stride=1 << 21), UNSUP), (dict(q_stride=(1 << 22) + 16), UNSUP),
])
def test_quantize_status(change, status):
    a = dict(x=A, x_type=F32, x_stride=64, q=A, q_stride=64, scale=A, n_rows=2, k=64)
    a.update(change)
    assert lib.i8_quantize_rows(a["x"], a["x_type"], a["x_stride"], a["q"], a["q_stride"],
                                a["scale"], a["n_rows"], a["k"], None) == status


PRODUCT = [
    (dict(k=48), SHAPE), (dict(k=0), SHAPE), (dict(k=131072, x_stride=131072, w_stride=131072), UNSUP),
    (dict(n=-1), SHAPE), (dict(m=-1), SHAPE), (dict(n=0, w=None), OK), (dict(m=0, x=None), OK),
    (dict(n=(1 << 27) + 1), UNSUP), (dict(m=(1 << 27) + 1), UNSUP),
    (dict(x_type=4), UNSUP), (dict(y_type=I8), UNSUP), (dict(y_type=-1), UNSUP),
    (dict(x=None), NULL), (dict(x_scale=None), NULL), (dict(w=None), NULL),
    (dict(w_scale=None), NULL), (dict(y=None), NULL),
    (dict(x_stride=32), SHAPE), (dict(w_stride=32), SHAPE), (dict(y_stride=7), SHAPE),
    (dict(x=A + 8), ALIGN), (dict(w=A + 4), ALIGN), (dict(x_stride=72), ALIGN),
    (dict(w_stride=72), ALIGN), (dict(y=A + 2), ALIGN), (dict(y=A + 1, y_type=F16), ALIGN),
    (dict(x_scale=A + 2), ALIGN), (dict(w_scale=A + 1), ALIGN),
    (dict(x_stride=(1 << 22) + 16), UNSUP), (dict(w_stride=(1 << 22) + 16), UNSUP),
    # activations that are not codes: the workspace
    (dict(x_type=F32, ws=None), WS), (dict(x_type=BF16, ws_bytes=256), WS),
    (dict(x_type=F16, ws=A + 128), ALIGN), (dict(x_type=F32, x_stride=66), ALIGN),
]


def _product(fn, change):
    a = dict(x=A, x_type=I8, x_stride=64, x_scale=A, w=A, w_stride=64, w_scale=A, bias=None, y=A,
             y_type=F32, y_stride=8, n=8, k=64, m=4, ws=A, ws_bytes=1 << 20)
    a.update(change)
    order = ["x", "x_type", "x_stride", "x_scale", "w", "w_stride", "w_scale", "bias", "y", "y_type",
             "y_stride", "n", "k", "m", "ws", "ws_bytes"]
    if fn is lib.i8_up_gate_swiglu:
        order.remove("bias")
    return fn(*[a[o] for o in order], None)


@pytest.mark.parametrize("change,status", PRODUCT + [(dict(bias=A + 2), ALIGN)])
def test_matmul_status(change, status):
    assert _product(lib.i8_matmul, change) == status


@pytest.mark.parametrize("change,status", PRODUCT)
def test_up_gate_status(change, status):
    assert _product(lib.i8_up_gate_swiglu, change) == status


def test_workspace_bytes():
    assert lib.i8_workspace_bytes(1, 64) == 256
    assert lib.i8_workspace_bytes(0, 64) == 256
    assert lib.i8_workspace_bytes(16, 4096) >= 16 * 4100
    for m, k in ((-1, 64), (1, 33), (1, 0), (1, 131072)):
        assert lib.i8_workspace_bytes(m, k) == 0
    assert lib.logprob_workspace_bytes(4, 1000, 5) >= 256
    for m, v, n in ((-1, 10, 1), (1, 0, 0), (1, 10, 11), (1, 10, -1), (1, 100, 65),
                    (1, (1 << 30) + 1, 1), ((1 << 24) + 1, 10, 1)):
        assert lib.logprob_workspace_bytes(m, v, n) == 0


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), SHAPE), (dict(v=0), SHAPE), (dict(v=-5), SHAPE), (dict(top=-1), SHAPE),
    (dict(v=4, top=5), SHAPE), (dict(given=-1), SHAPE), (dict(stride=99), SHAPE),
    (dict(top=65), UNSUP), (dict(given=1025), UNSUP), (dict(type=3), UNSUP), (dict(type=-1), UNSUP),
    (dict(v=(1 << 30) + 1, stride=1 << 31), UNSUP), (dict(m=(1 << 24) + 1), UNSUP),
    (dict(m=0, logits=None), OK),
    (dict(logits=None), NULL), (dict(tokens=None), NULL), (dict(logprob=None), NULL),
    (dict(ids=None), NULL), (dict(tops=None), NULL),
    (dict(logits=A + 2), ALIGN), (dict(logits=A + 1, type=BF16), ALIGN), (dict(tokens=A + 2), ALIGN),
    (dict(logprob=A + 1), ALIGN), (dict(lse=A + 2), ALIGN), (dict(entropy=A + 2), ALIGN),
    (dict(ids=A + 2), ALIGN), (dict(tops=A + 2), ALIGN), (dict(ws=A + 64), ALIGN),
    (dict(ws=None), WS), (dict(ws_bytes=0), WS),
])
def test_logprob_status(change, status):
    a = dict(logits=A, type=F32, stride=100, tokens=A, given=1, logprob=A, lse=A, entropy=A, ids=A,
             tops=A, m=2, v=100, top=5, ws=A, ws_bytes=1 << 30)
    a.update(change)
    order = ["logits", "type", "stride", "tokens", "given", "logprob", "lse", "entropy", "ids", "tops",
             "m", "v", "top", "ws", "ws_bytes"]
    assert lib.logprob_rows(*[a[o] for o in order], None) == status


# --- the binding -------------------------------------------------------------

class Strided(FakeGpu):
    """A stand-in whose columns are not contiguous."""

    def stride(self, i=None):
        st = tuple(2 * s for s in super().stride())
        return st if i is None else st[i]


def test_binding_quantize():
    with pytest.raises(TypeError, match="x:"):
        q.i8_quantize_rows(i8((2, 64)))
    with pytest.raises(ValueError, match="rows must be contiguous"):
        q.i8_quantize_rows(Strided((2, 64), torch.float32))
    with pytest.raises(ValueError, match="q: shape"):
        q.i8_quantize_rows(f32((2, 64)), q=i8((2, 32)), scale=f32(2))
    with pytest.raises(ValueError, match="scale"):
        q.i8_quantize_rows(f32((2, 64)), q=i8((2, 64)), scale=f32(3))
    with pytest.raises(ValueError, match="several devices"):
        q.i8_quantize_rows(f32((2, 64)), q=i8((2, 64), 1), scale=f32(2))
    with pytest.raises(ValueError, match="GPU tensor"):
        q.i8_quantize_rows(torch.zeros(2, 64))


@pytest.mark.parametrize("fn,rows,out", [(q.i8_matmul, 6, "y"), (q.i8_up_gate_swiglu, 12, "h")])
def test_binding_products(fn, rows, out):
    ok = dict(x=i8((4, 64)), w=i8((rows, 64)), w_scale=f32(rows), x_scale=f32(4))
    ok[out] = f32((4, 6))

    def bad(exc, match, **kw):
        with pytest.raises(exc, match=match):
            fn(**{**ok, **kw})

    bad(ValueError, "w: rows of 32", w=i8((rows, 32)))
    bad(TypeError, "w:", w=f32((rows, 64)))
    bad(ValueError, "w_scale", w_scale=f32(rows + 1))
    bad(TypeError, "w_scale", w_scale=FakeGpu(rows, torch.float16))
    bad(ValueError, "x_scale", x_scale=None)
    bad(ValueError, "x_scale", x_scale=f32(3))
    bad(ValueError, "x_scale", x=f32((4, 64)))              # scales with rows that are not codes
    bad(ValueError, f"{out}: shape", **{out: f32((4, 7))})
    bad(TypeError, f"{out}:", **{out: i8((4, 6))})
    bad(ValueError, "several devices", w=i8((rows, 64), 1))
    bad(ValueError, "several devices", **{out: f32((4, 6), 1)})
    bad(ValueError, "rows must be contiguous", x=Strided((4, 64), torch.int8))
    bad(ValueError, "2 dimensions", x=i8((64,)))
    if fn is q.i8_matmul:
        bad(ValueError, "bias", bias=f32(5))
    else:
        bad(ValueError, "gate and up", w=i8((11, 64)), w_scale=f32(11))


def test_binding_workspaces():
    for args in ((1, 33), (-1, 64)):
        with pytest.raises(q.Q8Error):
            q.i8_workspace(*args, "cpu")
    with pytest.raises(q.Q8Error):
        q.logprob_workspace(2, 100, 65, "cpu")


def test_binding_logprob():
    out = q.LogprobOut(f32(2), f32(2), f32(2), i32((2, 3)), f32((2, 3)))
    ok = dict(logits=f32((2, 100)), tokens=i32(2), n_top=3, ws=u8(256), out=out)

    def bad(exc, match, **kw):
        with pytest.raises(exc, match=match):
            q.logprob_rows(**{**ok, **kw})

    bad(TypeError, "logits", logits=i8((2, 100)))
    bad(ValueError, "rows must be contiguous", logits=Strided((2, 100), torch.float32))
    bad(TypeError, "tokens", tokens=FakeGpu(2, torch.int64))
    bad(ValueError, "tokens", tokens=i32(3))
    bad(ValueError, "tokens", tokens=i32((3, 1)))
    bad(ValueError, "lse", out=out._replace(lse=f32(3)))
    bad(ValueError, "top_ids", out=out._replace(top_ids=i32((2, 4))))
    bad(ValueError, "lacks", out=out._replace(top_logprobs=None))
    bad(ValueError, "lacks", out=out._replace(logprob=None))
    bad(ValueError, "several devices", ws=u8(256, 1))
    bad(TypeError, "ws", ws=f32(64))
