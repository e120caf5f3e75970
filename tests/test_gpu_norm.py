"""Norm rows and the residual stream's update on the GPU against 64-bit
references (tests/ops_ref.py), codes exactly."""
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


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _tensor(rng, m, n, t, pad=0, offset=0, size=1.0, middle=0.0):
    """Rows of n values of type t, n + pad apart, `offset` into their buffer."""
    import torch
    tt = i8_ref.torch_type(t)
    buf = torch.full((m * (n + pad) + offset + 8,), 1e4, dtype=tt, device="cuda")
    x = buf[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    v = rng.normal(size=(m, n)) * size + middle
    v[:, rng.integers(0, n, max(1, n // 300))] *= 12
    x.copy_(to_gpu(v.astype(np.float32)))
    return x


def _vec(rng, n, size=0.2, middle=1.0):
    return to_gpu((rng.normal(size=n) * size + middle).astype(np.float32))


def _narrow(yt, *streams):
    """Whether a call with these rows is computed in 32 bits."""
    import torch
    half = (torch.float16, torch.bfloat16)
    return yt in ("fp16", "bf16") and all(s is None or s.dtype in half for s in streams)


def _check_y(q, x, weight, bias, eps, layer, out, t, what, narrow=None):
    """y of the rows x (as the norm read them)."""
    narrow = _narrow(t, x) if narrow is None else narrow
    if t == "i8":
        y, _ = ops_ref.norm(_host(x), _host(weight), _host(bias), eps, layer)
        codes, scale = i8_ref.quantize(y.astype(np.float32))
        assert np.array_equal(out.y.cpu().numpy(), codes), what
        assert np.array_equal(out.y_scale.cpu().numpy(), scale, equal_nan=True), what
    else:
        value, bound = ops_ref.norm(_host(x), _host(weight), _host(bias), eps, layer, narrow)
        ops_ref.assert_rounded(_host(out.y), value, bound, t, what)


N_ANY = [1, 2, 7, 8, 63, 64, 100, 513, 768, 1003, 1025, 2048, 2049, 4096, 4097, 5632, 8200, 14336, 16385, 32768,
         32769, 65536]


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("n", N_ANY)
def test_norm_sizes(q, n, layer):
    rng = synth.rng("norm", str(n), str(layer))
    for m, xt, yt in ((1, "fp32", "bf16"), (3, "bf16", "fp32"), (6, "fp16", "fp16"), (65, "bf16", "bf16")):
        if m * n > 1 << 20:
            continue
        x = _tensor(rng, m, n, xt)
        w, b = _vec(rng, n), _vec(rng, n, 0.1, 0.0) if layer else None
        out = q.norm_rows(x, w, bias=b, eps=1e-5, layer=layer, dtype=i8_ref.torch_type(yt))
        assert out.residual is None and out.y_scale is None
        _check_y(q, x, w, b, 1e-5, layer, out, yt, (m, n, xt, yt))


@pytest.mark.parametrize("xt", i8_ref.TYPES)
@pytest.mark.parametrize("m,n", [(1, 32), (4, 96), (5, 768), (257, 2048), (9, 4096), (3, 14336), (2, 65536), (1030, 64)])
def test_norm_codes(q, m, n, xt):
    """Codes as the reference's, and those of the quantizer on the fp32 rows."""
    import torch
    rng = synth.rng("normq", str(m), str(n), xt)
    x, w = _tensor(rng, m, n, xt), _vec(rng, n)
    out = q.norm_rows(x, w, dtype=torch.int8)
    _check_y(q, x, w, None, 1e-5, False, out, "i8", (m, n))
    codes, scale = q.i8_quantize_rows(q.norm_rows(x, w).y)
    assert torch.equal(codes, out.y) and torch.equal(scale, out.y_scale)


CASES = [dict(), dict(post=True), dict(gate="channel"), dict(gate="row", alpha=0.5),
         dict(post=True, gate="row", layer=True, post_bias=True), dict(post=True, gate="channel", alpha=0.0),
         dict(layer=True, alpha=-1.5), dict(layer=True, post=True, gate="channel")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()) or "plain")
@pytest.mark.parametrize("m,n", [(1, 768), (3, 100), (130, 352), (17, 2048), (5, 4099), (2, 14336), (2, 40000)])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("fp16", "fp32", "i8"), ("fp32", "fp32", "fp32"),
                                   ("bf16", "fp32", "fp16"), ("fp32", "fp16", "i8")], ids="-".join)
def test_residual(q, m, n, types, case):
    xt, rt, yt = types
    if yt == "i8":
        n = n // 32 * 32
    rng = synth.rng("resnorm", str(m), str(n), xt, rt, str(sorted(case)))
    x, r = _tensor(rng, m, n, xt), _tensor(rng, m, n, rt, size=3.0)
    layer, alpha = case.get("layer", False), case.get("alpha", 1.0)
    w, b = _vec(rng, n), _vec(rng, n, 0.1, 0.0) if layer else None
    pw = _vec(rng, n) if case.get("post") else None
    pb = _vec(rng, n, 0.1, 0.0) if case.get("post_bias") else None
    gate = {None: None, "channel": _vec(rng, n, 0.1, 0.5), "row": _tensor(rng, m, n, xt)}[case.get("gate")]
    import torch
    yd = torch.int8 if yt == "i8" else i8_ref.torch_type(yt)
    out = q.residual_norm_rows(x, r, w, bias=b, post_weight=pw, post_bias=pb, gate=gate, residual_scale=alpha,
                               eps=1e-6, layer=layer, dtype=yd)
    narrow = _narrow(yt, x, r, gate if case.get("gate") == "row" else None)
    value, bound = ops_ref.residual(_host(x), _host(r), _host(pw), _host(pb), _host(gate), alpha, 1e-6, layer, narrow)
    ops_ref.assert_rounded(_host(out.residual), value, bound, rt, "residual")
    _check_y(q, out.residual, w, b, 1e-6, layer, out, yt, "y", narrow)
    # what follows the stream's update is the plain norm of the stream
    if narrow == _narrow(yt, r):
        plain = q.norm_rows(out.residual, w, bias=b, eps=1e-6, layer=layer, dtype=yd)
        assert torch.equal(plain.y, out.y)
    # in place
    again = q.residual_norm_rows(x, r, w, bias=b, post_weight=pw, post_bias=pb, gate=gate, residual_scale=alpha,
                                 eps=1e-6, layer=layer, residual_out=r, dtype=yd)
    assert again.residual is r and torch.equal(r, out.residual) and torch.equal(again.y, out.y)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (7, 8), (2, 3)])
def test_row_starts(q, offset, pad, t):
    """Rows that start anywhere; what lies beside a row is neither read nor
    written."""
    import torch
    rng = synth.rng("normstart", str(offset), str(pad), t)
    for m, n in ((3, 5), (4, 1003), (2, 4100)):
        x, r, g = (_tensor(rng, m, n, t, pad, offset) for _ in range(3))
        w = _vec(rng, n)
        tt = i8_ref.torch_type(t)
        bufs = [torch.full((m * (n + pad) + offset + 8,), -7.0, dtype=tt, device="cuda") for _ in range(2)]
        ro, y = (b[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n] for b in bufs)
        out = q.residual_norm_rows(x, r, w, gate=g, residual_out=ro, y=y)
        value, bound = ops_ref.residual(_host(x), _host(r), None, None, _host(g), 1.0, 1e-5, False, _narrow(t, x))
        ops_ref.assert_rounded(_host(ro), value, bound, t, "residual")
        _check_y(q, ro, w, None, 1e-5, False, out, t, "y")
        for b in bufs:
            body = b[offset:offset + m * (n + pad)].view(m, n + pad)
            assert bool((body[:, n:] == -7).all()) and bool((b[:offset] == -7).all())
            assert bool((b[offset + m * (n + pad):] == -7).all())


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_rows_far_from_zero(q, t):
    """A mean far above the spread, 16-bit rows."""
    rng = synth.rng("normfar", t)
    x = _tensor(rng, 5, 900, t, middle=300.0)
    w, b = _vec(rng, 900), _vec(rng, 900, 0.1, 0.0)
    out = q.norm_rows(x, w, bias=b, layer=True, dtype=i8_ref.torch_type(t))
    _check_y(q, x, w, b, 1e-5, True, out, t, "y")


@pytest.mark.parametrize("size", [1e-25, 1e-12, 1e19, 1e30])
@pytest.mark.parametrize("layer", [False, True])
def test_rows_whose_squares_leave_32_bits(q, size, layer):
    """bfloat16 rows of very large and very small values, without an eps."""
    import torch
    rng = synth.rng("normsquares", str(size), str(layer))
    for n in (100, 4096):
        x = to_gpu((rng.normal(size=(3, n)) * size).astype(np.float32)).bfloat16()
        w = _vec(rng, n)
        out = q.norm_rows(x, w, eps=0.0, layer=layer, dtype=torch.bfloat16)
        _check_y(q, x, w, None, 0.0, layer, out, "bf16", (size, n))


def test_odd_rows(q):
    """Zero rows, constant rows, rows far from 0, infinities and NaN."""
    import torch
    n = 320
    rng = synth.rng("normodd")
    x = rng.normal(size=(8, n))
    x[0], x[1], x[2] = 0.0, 3.0, rng.normal(size=n) * 1e-30
    x[3] = 1e6 + rng.normal(size=n)
    x[4, 5], x[5, 7], x[6] = np.inf, np.nan, rng.normal(size=n) * 1e15
    x = to_gpu(x.astype(np.float32))
    w, b = _vec(rng, n), _vec(rng, n, 0.1, 0.0)
    for layer in (False, True):
        out = q.norm_rows(x, w, bias=b, layer=layer)
        good = [0, 1, 2, 3, 6, 7]
        value, bound = ops_ref.norm(_host(x)[good], _host(w), _host(b), 1e-5, layer)
        ops_ref.assert_rounded(_host(out.y)[good], value, bound, "fp32", "y")
        assert bool(torch.isnan(out.y[5]).all()) and bool(torch.isnan(out.y[4]).any())
        codes = q.norm_rows(x, w, bias=b, layer=layer, dtype=torch.int8)
        assert torch.isnan(codes.y_scale).tolist() == [False] * 4 + [True] * 2 + [False] * 2
        assert bool((codes.y[4:6] == 0).all())
    zero = q.norm_rows(x[:1], w, dtype=torch.int8)
    assert zero.y_scale.item() == 0 and bool((zero.y == 0).all())
    assert q.norm_rows(x[:0], w).y.shape == (0, n)


@pytest.mark.parametrize("n", [96, 4096])
def test_row_alone(q, n):
    """A row's outputs are the same bits whatever rows a call has."""
    import torch
    rng = synth.rng("normalone", str(n))
    x, r, w = _tensor(rng, 300, n, "bf16"), _tensor(rng, 300, n, "bf16"), _vec(rng, n)
    whole = q.residual_norm_rows(x, r, w, post_weight=w, dtype=torch.int8)
    for i in (0, 7, 299):
        one = q.residual_norm_rows(x[i:i + 1], r[i:i + 1], w, post_weight=w, dtype=torch.int8)
        assert all(torch.equal(a[0], b[i]) for a, b in zip(one, whole))


def test_many_rows(q):
    """More rows than one launch takes waves of; offsets past 2^32 bytes."""
    import torch
    m, n = 1 << 20, 2112
    x = torch.ones((m, n), dtype=torch.bfloat16, device="cuda")
    x[-1, :] = 2.0
    x[m // 2, 0] = 40.0
    w = torch.ones(n, device="cuda")
    out = q.norm_rows(x, w, eps=0.0, dtype=torch.bfloat16)
    assert bool((out.y[:m // 2] == 1).all()) and bool((out.y[-1] == 1).all())
    value, bound = ops_ref.norm(_host(x[m // 2:m // 2 + 1]), np.ones(n), None, 0.0, False, True)
    ops_ref.assert_rounded(_host(out.y[m // 2:m // 2 + 1]), value, bound, "bf16", "row")
