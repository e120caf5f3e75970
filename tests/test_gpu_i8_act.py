"""8-bit products with an activation and a residual in their epilogue on the GPU
against 64-bit references (tests/ops_ref.py), on every kernel that runs them."""
import numpy as np
import pytest

import i8_ref
import ops_ref
import synth
from gpu_cases import to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


class Case:
    def __init__(self, m, k, n, tag="", sigma=None):
        rng = synth.rng("i8act", str(m), str(k), str(n), tag)
        self.rng = rng
        self.cx = rng.integers(-128, 128, size=(m, k)).astype(np.int8)
        self.cw = rng.integers(-128, 128, size=(n, k)).astype(np.int8)
        # values of a few units, where the activations bend
        s = (3.0 if sigma is None else sigma) / (74.0 * 74.0 * np.sqrt(k))
        self.sx = (np.sqrt(s) * rng.uniform(0.5, 1.5, m)).astype(np.float32)
        self.sw = (np.sqrt(s) * rng.uniform(0.5, 1.5, n)).astype(np.float32)
        self.bias = rng.normal(size=n).astype(np.float32)
        self.res = rng.normal(size=(m, n)).astype(np.float32)

    def gpu(self, t):
        import torch
        r = to_gpu(self.res).to(i8_ref.torch_type(t))
        return to_gpu(self.cx), to_gpu(self.sx), to_gpu(self.cw), to_gpu(self.sw), to_gpu(self.bias), r


def _check(q, c, t, act, bias=True, residual=True, y=None, r=None):
    cx, sx, cw, sw, b, r0 = c.gpu(t)
    r = r0 if r is None else r
    out = q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b if bias else None, act=act,
                          residual=r if residual else None, y=y, dtype=i8_ref.torch_type(t))
    ref, bound = ops_ref.product_act(c.cx, c.sx, c.cw, c.sw, c.bias if bias else None, act,
                                     r0.double().cpu().numpy() if residual else None)
    i8_ref.assert_close(out.double().cpu().numpy(), ref, bound, t, act)
    return out


# (m, k, n) on each kernel: streamed (1 to 64 rows, small matrices), tiles of 128 and of
# 256, whole and in halves (q8v_i8_form)
SIZES = [(1, 32, 1), (1, 768, 2048), (3, 96, 37), (13, 1120, 300), (16, 4128, 513), (33, 256, 1000), (64, 512, 4100),
         (200, 160, 77), (150, 288, 9000), (333, 96, 5001), (1024, 256, 16390), (2050, 64, 8200)]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_sizes(q, m, k, n, t):
    c = Case(m, k, n)
    acts = ops_ref.ACTS if m * n < 200000 else ("none", "gelu_tanh")
    for i, act in enumerate(acts):
        _check(q, c, t, act, bias=i % 2 == 0, residual=i % 3 != 1)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,k,n", [(300, 1024, 4100), (300, 1056, 4100), (130, 2080, 6000), (97, 1312, 8192),
                                   (512, 4128, 3001), (320, 14336, 4096)])
def test_halves_of_k(q, m, k, n, t):
    """Few outputs and a long k: halves of k side by side, of one and of
    different lengths, the second ending inside a step; bits as i8_matmul."""
    import torch
    c = Case(m, k, n, "halves")
    for act, bias, residual in (("none", True, True), ("silu", False, False)):
        _check(q, c, t, act, bias=bias, residual=residual)
    cx, sx, cw, sw, b, r = c.gpu(t)
    plain = q.i8_matmul(cx, cw, sw, x_scale=sx, bias=b, dtype=i8_ref.torch_type(t))
    assert torch.equal(q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, dtype=i8_ref.torch_type(t)), plain)


def test_forms(q):
    """The sizes above reach every kernel."""
    forms = {q.raw.q8v_i8_form(n, k, m, 0) for m, k, n in SIZES}
    assert forms >= {0, 1, 2, 3} or forms >= {0, 1, 2, 4} or forms >= {0, 1, 2, 5}, forms


@pytest.mark.parametrize("act", ops_ref.ACTS)
@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_activations_over_their_range(q, act, t):
    """Values from far left to far right of every activation's bend."""
    for m, k, n in ((5, 64, 700), (260, 64, 9000)):
        for sigma in (0.05, 3.0, 40.0):
            _check(q, Case(m, k, n, str(sigma), sigma), t, act, residual=sigma == 3.0)


@pytest.mark.parametrize("m,k,n", [(2, 256, 300), (40, 512, 700), (300, 128, 9001)])
def test_same_bits(q, m, k, n):
    """None of both is i8_matmul; a row does not depend on the others; float
    tokens are those quantized before; in place is the same."""
    import torch
    c = Case(m, k, n, "bits")
    cx, sx, cw, sw, b, r = c.gpu("bf16")
    for t in (torch.float32, torch.float16, torch.bfloat16):
        plain = q.i8_matmul(cx, cw, sw, x_scale=sx, bias=b, dtype=t)
        assert torch.equal(q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, dtype=t), plain)
    whole = q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act="gelu", residual=r)
    assert whole.dtype == torch.bfloat16
    for i in (0, m - 1):
        one = q.i8_matmul_act(cx[i:i + 1], cw, sw, x_scale=sx[i:i + 1], bias=b, act="gelu", residual=r[i:i + 1])
        assert torch.equal(one[0], whole[i])
    y = r.clone()
    q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act="gelu", residual=y, y=y)
    assert torch.equal(y, whole)
    x = to_gpu(c.rng.normal(size=(m, k)).astype(np.float32))
    ws = q.i8_workspace(m, k, "cuda")
    qx, qs = q.i8_quantize_rows(x)
    for act in ("silu", "relu2"):
        assert torch.equal(q.i8_matmul_act(x, cw, sw, act=act, residual=r, ws=ws),
                           q.i8_matmul_act(qx, cw, sw, x_scale=qs, act=act, residual=r))


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (5, 8)])
def test_row_starts(q, offset, pad, t):
    """Residual and output rows that start anywhere, of different strides."""
    import torch
    tt = i8_ref.torch_type(t)
    for m, k, n in ((3, 64, 45), (70, 96, 130), (300, 64, 9003)):
        c = Case(m, k, n, "start")
        rb = torch.full((m * (n + pad + 1) + offset,), 1e4, dtype=tt, device="cuda")
        r = rb[offset:].view(m, n + pad + 1)[:, :n]
        r.copy_(to_gpu(c.res))
        yb = torch.full((m * (n + pad) + offset + 9,), -7.0, dtype=tt, device="cuda")
        y = yb[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
        _check(q, c, t, "gelu_tanh", y=y, r=r)
        body = yb[offset:offset + m * (n + pad)].view(m, n + pad)
        assert bool((body[:, n:] == -7).all()) and bool((yb[:offset] == -7).all())
        assert bool((yb[offset + m * (n + pad):] == -7).all())


def test_not_finite(q):
    """Infinities and NaN of scales and residuals go where they belong."""
    import torch
    c = Case(3, 64, 40, "nf")
    cx, sx, cw, sw, b, r = c.gpu("fp32")
    sx[1] = float("nan")
    r[2, 5], r[0, 7] = float("inf"), float("nan")
    for act in ops_ref.ACTS:
        y = q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act=act, residual=r)
        assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[0, 7])) and float(y[2, 5]) == float("inf")
        y[1], y[0, 7], y[2, 5] = 0, 0, 0
        assert bool(torch.isfinite(y).all())
    assert q.i8_matmul_act(cx[:0], cw, sw, x_scale=sx[:0], residual=r[:0]).shape == (0, 40)
