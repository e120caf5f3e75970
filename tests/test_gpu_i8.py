"""The 8-bit products with token and channel scales on the GPU against 64-bit
references (tests/i8_ref.py derives the bounds): codes and scales exactly,
products within their fp32 roundings and the output type's."""
import numpy as np
import pytest

import i8_ref
import synth
from gpu_cases import to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


def _typed(x, t):
    """x (fp32) on the GPU in type t, and the values it holds."""
    g = to_gpu(x.astype(np.float32)).to(i8_ref.torch_type(t))
    return g, g.float().cpu().numpy()


def _codes(rng, rows, k, low=-128):
    return rng.integers(low, 128, size=(rows, k), dtype=np.int64).astype(np.int8)


def _scales(rng, n):
    return (rng.uniform(0.5, 1.5, size=n) * 3e-3).astype(np.float32)


# --- row quantization ---------------------------------------------------------

@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (2, 768), (5, 2080), (37, 4096), (3, 14336),
                                    (700, 160), (2, 131040)])
def test_quantize_exact(q, t, rows, k):
    rng = synth.rng("i8q", t, str(rows), str(k))
    x, held = _typed(rng.normal(size=(rows, k)) * np.exp(rng.normal(size=(rows, 1)) * 3), t)
    c, s = q.i8_quantize_rows(x)
    rc, rs = i8_ref.quantize(held)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)


@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_quantize_edges(q, t):
    """Exact ties (scale 1 and powers of two), zero rows, signed zeros, rows of
    subnormals, of the largest values, with NaN and infinities."""
    k = 64
    rows = []
    half = np.arange(k) - 31.5
    rows.append(np.concatenate([half[:-1], [127]]))
    rows.append(np.concatenate([half[:-1], [-127]]) * 2.0 ** -8)
    rows.append(np.zeros(k))
    rows.append(np.where(np.arange(k) % 2, 0.0, -0.0))
    tiny = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -24, "bf16": 2.0 ** -133}[t]
    for n in (1, 63, 64, 127, 128, 200, 255):
        rows.append(np.where(np.arange(k) == 5, n * tiny, (np.arange(k) % (n + 1)) * tiny))
    big = {"fp32": 3.4028235e38, "fp16": 65504.0, "bf16": 3.3895314e38}[t]
    rows.append(np.linspace(-1, 1, k) * big)
    for bad in (np.nan, np.inf, -np.inf):
        rows.append(np.where(np.arange(k) == 40, bad, 1.0))
    rows.append(np.full(k, np.nan))
    x, held = _typed(np.array(rows), t)
    c, s = q.i8_quantize_rows(x)
    rc, rs = i8_ref.quantize(held)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(c.cpu().numpy(), rc)


@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_quantize_near_ties(q, t):
    """Values on and one step beside every (q + 1/2) * s."""
    rng = synth.rng("i8ties", t)
    import torch
    tt = i8_ref.torch_type(t)
    rows = []
    for _ in range(40):
        a = float(torch.tensor(rng.uniform(0.01, 100)).to(tt))
        s = float(np.float32(a) / np.float32(127))
        v = torch.tensor((np.arange(127) + 0.5) * s, dtype=torch.float64).to(tt)
        near = torch.cat([torch.nextafter(v, torch.zeros_like(v)), v,
                          torch.nextafter(v, torch.full_like(v, a)), torch.tensor([a, -a, 0.0], dtype=tt)])
        near = torch.cat([near, -near])[:736]
        near[-1] = a
        rows.append(near)
    x = torch.stack(rows).cuda()
    assert x.shape[1] % 32 == 0
    c, s = q.i8_quantize_rows(x)
    rc, rs = i8_ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)


def test_quantize_strides(q):
    """Slices of wider buffers; nothing beside the rows is written."""
    import torch
    rng = synth.rng("i8strides")
    wide = to_gpu(rng.normal(size=(9, 512)).astype(np.float32)).to(torch.bfloat16)
    x = wide[1:8, 64:64 + 352]
    buf = torch.full((9, 512), 77, dtype=torch.int8, device="cuda")
    c, s = q.i8_quantize_rows(x, q=buf[1:8, 32:32 + 352])
    rc, rs = i8_ref.quantize(x.float().cpu().numpy())
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    buf[1:8, 32:32 + 352] = 77
    assert bool((buf == 77).all())
    assert q.i8_quantize_rows(wide[:0])[0].shape == (0, 512)
    with pytest.raises(q.Q8Error):
        q.i8_quantize_rows(wide[:, 4:4 + 32])       # rows start off a 16-byte boundary
    with pytest.raises(q.Q8Error):
        q.i8_quantize_rows(wide[:1].expand(4, 512))   # rows on top of each other


# --- products -----------------------------------------------------------------

# one token to several tiles of tokens, ragged everywhere; k of one slice, odd
# numbers of slices, long
SHAPES = [(1, 1, 32), (1, 70, 64), (1, 768, 768), (1, 2051, 2080), (1, 129, 14336), (2, 33, 96),
          (3, 100, 160), (4, 64, 1056), (5, 513, 352), (7, 257, 4096), (8, 300, 288), (9, 1000, 768),
          (15, 67, 1024), (16, 130, 544), (17, 129, 416), (24, 515, 2048), (31, 40, 128),
          (33, 260, 1184), (47, 640, 96), (63, 191, 2048), (64, 512, 160), (65, 65, 992),
          (96, 385, 736), (100, 130, 1504), (127, 1030, 224), (129, 257, 608), (200, 300, 320),
          (255, 129, 1312), (256, 256, 512), (257, 513, 448), (300, 1000, 4096), (513, 770, 1120),
          (1030, 1290, 256)]
# enough outputs for the large tiles: whole rounds and halves (some of them past
# the last token), one round that is not split
LARGE = [(1100, 16640, 96), (1792, 8200, 64), (600, 14400, 160)]


def _operands(m, rows, k, *key):
    rng = synth.rng("i8", str(m), str(rows), str(k), *key)
    return (rng, _codes(rng, m, k), _scales(rng, m) * 10, _codes(rng, rows, k), _scales(rng, rows))


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(q, m, n, k, t):
    rng, cx, sx, cw, sw = _operands(m, n, k)
    bias = rng.normal(size=n).astype(np.float32) if (m + n) % 2 else None
    y = q.i8_matmul(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(sx),
                    bias=None if bias is None else to_gpu(bias), dtype=i8_ref.torch_type(t))
    ref, bound = i8_ref.product(cx, sx, cw, sw, bias)
    i8_ref.assert_close(y.double().cpu().numpy(), ref, bound, t, f"{m}x{n}x{k}")


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n_ff,k", SHAPES)
def test_up_gate(q, m, n_ff, k, t):
    _, cx, sx, cw, sw = _operands(m, 2 * n_ff, k, "ug")
    sx *= np.float32(30.0 / (np.sqrt(k) * 5500 * 3e-2))       # gates of a few units
    h = q.i8_up_gate_swiglu(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(sx),
                            dtype=i8_ref.torch_type(t))
    ref, bound = i8_ref.gated(cx, sx, cw, sw)
    i8_ref.assert_close(h.double().cpu().numpy(), ref, bound, t, f"{m}x{n_ff}x{k}")


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,rows,k", LARGE)
def test_large(q, m, rows, k, t):
    """Both forms, the output inside a wider buffer with rows at odd elements."""
    import torch
    rng, cx, sx, cw, sw = _operands(m, rows, k, "large")
    sx *= np.float32(30.0 / (np.sqrt(k) * 5500 * 3e-2))
    x, s, w, ws = to_gpu(cx), to_gpu(sx), to_gpu(cw), to_gpu(sw)
    bias = rng.normal(size=rows).astype(np.float32)
    for fn, cols, ref, kw in ((q.i8_matmul, rows, i8_ref.product(cx, sx, cw, sw, bias), "y"),
                              (q.i8_up_gate_swiglu, rows // 2, i8_ref.gated(cx, sx, cw, sw), "h")):
        buf = torch.full((m + 2, cols + 7), 5.5, dtype=i8_ref.torch_type(t), device="cuda")
        out = buf[1:m + 1, 3:3 + cols]
        extra = {"bias": to_gpu(bias)} if fn is q.i8_matmul else {}
        fn(x, w, ws, x_scale=s, **{kw: out}, **extra)
        i8_ref.assert_close(out.double().cpu().numpy(), *ref, t, f"{m}x{rows}x{k}")
        out.fill_(5.5)
        assert bool((buf == 5.5).all())


@pytest.mark.parametrize("t", i8_ref.TYPES + ("codes",))
@pytest.mark.parametrize("n", [70, 5000, 20000])
def test_few_long_rows(q, n, t):
    """Float rows of up to 16384 values together, and just more, have the bits of
    the quantizer's codes; so have codes wherever they are read from."""
    import torch
    for m, k in ((1, 8192), (1, 8224), (1, 16384), (1, 16416), (2, 4096), (2, 4128), (2, 8192),
                 (2, 8224), (3, 2720), (3, 2752), (4, 2048), (4, 2080), (4, 4096), (5, 1632)):
        rng, cx, sx, cw, sw = _operands(m, n, k, "few")
        w, ws = to_gpu(cw), to_gpu(sw)
        if t == "codes":
            codes, scale = to_gpu(cx), to_gpu(sx)
            x, kw = codes, {"x_scale": scale}
        else:
            x, _ = _typed(rng.normal(size=(m, k)) * np.arange(1, m + 1)[:, None], t)
            codes, scale = q.i8_quantize_rows(x)
            kw = {"ws": q.i8_workspace(m, k, "cuda")}
        # (eight rows are beyond the form that quantizes inside)
        many = codes.repeat(8, 1), scale.repeat(8)
        for fn in (q.i8_matmul, q.i8_up_gate_swiglu):
            y = fn(x, w, ws, **kw)
            z = fn(many[0], w, ws, x_scale=many[1])
            assert torch.equal(y, z[:m]), (fn.__name__, m, k)


@pytest.mark.parametrize("m", [1, 3, 16, 40, 130, 300])
@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_float_activations(q, m, t):
    """Rows quantized inside the call: bitwise the quantizer, then the product."""
    import torch
    rng, _, _, cw, sw = _operands(m, 400, 1120, "float", t)
    wide, _ = _typed(rng.normal(size=(m, 1120 + 64)), t)
    x = wide[:, 32:32 + 1120]
    w, s = to_gpu(cw), to_gpu(sw)
    ws = q.i8_workspace(m, 1120, "cuda")
    ws.fill_(255)
    c, sx = q.i8_quantize_rows(x)
    assert torch.equal(q.i8_matmul(x, w, s, ws=ws), q.i8_matmul(c, w, s, x_scale=sx))
    assert torch.equal(q.i8_up_gate_swiglu(x, w, s, ws=ws),
                       q.i8_up_gate_swiglu(c, w, s, x_scale=sx))
    with pytest.raises(q.Q8Error, match="WORKSPACE"):
        q.i8_matmul(x, w, s)
    with pytest.raises(q.Q8Error, match="WORKSPACE"):
        q.i8_matmul(x, w, s, ws=ws[:m * 1120])


@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_rows_do_not_depend_on_the_batch(q, t):
    """Bit for bit the same output for a token alone and among others."""
    import torch
    rng, cx, sx, cw, sw = _operands(600, 330, 1376, "batch")
    bias = to_gpu(rng.normal(size=330).astype(np.float32))
    x, s, w, ws = to_gpu(cx), to_gpu(sx), to_gpu(cw), to_gpu(sw)
    tt = i8_ref.torch_type(t)
    full = q.i8_matmul(x, w, ws, x_scale=s, bias=bias, dtype=tt)
    gated = q.i8_up_gate_swiglu(x, w, ws, x_scale=s, dtype=tt)
    for a, b in ((0, 1), (599, 600), (7, 10), (20, 36), (100, 140), (300, 400), (5, 205)):
        assert torch.equal(q.i8_matmul(x[a:b], w, ws, x_scale=s[a:b], bias=bias, dtype=tt), full[a:b])
        assert torch.equal(q.i8_up_gate_swiglu(x[a:b], w, ws, x_scale=s[a:b], dtype=tt), gated[a:b])


@pytest.mark.parametrize("m", [1, 2, 11, 16, 50, 128, 300])
@pytest.mark.parametrize("t", i8_ref.TYPES)
def test_strides_and_surroundings(q, m, t):
    """Operands inside wider buffers, an output inside one: nothing beside it
    is written."""
    import torch
    n, k = 213, 480
    rng, cx, sx, cw, sw = _operands(m, 2 * n, k, "strides")
    tt = i8_ref.torch_type(t)
    x = torch.full((m + 2, k + 80), 99, dtype=torch.int8, device="cuda")
    w = torch.full((2 * n + 2, k + 48), -99, dtype=torch.int8, device="cuda")
    x[1:m + 1, 16:16 + k] = to_gpu(cx)
    w[1:2 * n + 1, 32:32 + k] = to_gpu(cw)
    xv, wv = x[1:m + 1, 16:16 + k], w[1:2 * n + 1, 32:32 + k]
    for fn, cols, ref in ((q.i8_matmul, 2 * n, i8_ref.product), (q.i8_up_gate_swiglu, n, i8_ref.gated)):
        buf = torch.full((m + 2, cols + 9), 5.5, dtype=tt, device="cuda")
        out = buf[1:m + 1, 3:3 + cols]
        fn(xv, wv, to_gpu(sw), to_gpu(sx), **{"y" if fn is q.i8_matmul else "h": out})
        val, bound = ref(cx, sx, cw, sw)
        i8_ref.assert_close(out.double().cpu().numpy(), val, bound, t)
        out.fill_(5.5)
        assert bool((buf == 5.5).all())


@pytest.mark.parametrize("m", [1, 9, 40, 200])
def test_extreme_codes(q, m):
    """The largest sums int32 holds (-128 everywhere, k = 131040)."""
    k, n = 131040, 5
    cx = np.full((m, k), -128, np.int8)
    cw = np.full((n, k), -128, np.int8)
    cw[1] = 127
    cw[2, ::2] = 127
    one = np.ones(max(m, n), np.float32)
    y = q.i8_matmul(to_gpu(cx), to_gpu(cw), to_gpu(one[:n]), x_scale=to_gpu(one[:m]))
    ref = i8_ref.sums(cx, cw).astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), ref)


@pytest.mark.parametrize("m", [3, 20, 70, 200])
def test_special_scales(q, m):
    """A NaN row stays NaN and alone so, zero rows give the bias, scales at the
    ends of fp32 give infinities and zeros as IEEE products do."""
    rng, cx, sx, cw, sw = _operands(m, 96, 256, "special")
    sx[0], sx[1], sx[2] = np.nan, 0.0, 3e37
    sw[5], sw[6] = 0.0, np.nan
    bias = rng.normal(size=96).astype(np.float32)
    y = q.i8_matmul(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(sx), bias=to_gpu(bias)).cpu().numpy()
    s = i8_ref.sums(cx, cw).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = ((s * sx[:, None]).astype(np.float64) * sw + bias).astype(np.float32)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    assert np.array_equal(np.isinf(y), np.isinf(ref))
    assert np.array_equal(y[1, :5], bias[:5]) and np.array_equal(y[3:, 5], np.broadcast_to(bias[5], m - 3))
    h = q.i8_up_gate_swiglu(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(sx)).cpu().numpy()
    assert np.isnan(h[0]).all() and np.isnan(h[:, 6]).all() and (h[1, :5] == 0).all()


def test_silu_range(q):
    """Gates from -120 to 120: products of one code, scales placed so."""
    import torch
    g = np.linspace(-120, 120, 481).astype(np.float32)
    n = g.size
    cw = np.zeros((2 * n, 32), np.int8)
    cw[:, 0] = 1
    cx = np.zeros((1, 32), np.int8)
    cx[0, 0] = 1
    sw = np.concatenate([g, np.ones(n, np.float32)])
    h = q.i8_up_gate_swiglu(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(np.ones(1, np.float32)))
    ref, bound = i8_ref.gated(cx, np.ones(1, np.float32), cw, sw)
    i8_ref.assert_close(h.double().cpu().numpy(), ref, bound, "fp32")
    sw[0], sw[1] = np.inf, 3e38
    h = q.i8_up_gate_swiglu(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(np.ones(1, np.float32)))
    assert torch.isinf(h[0, 0]) and h[0, 1] > 2.9e38
    assert q.i8_matmul(to_gpu(cx)[:0], to_gpu(cw), to_gpu(sw), x_scale=to_gpu(np.ones(0, np.float32))).shape == (0, 2 * n)
