"""The tile kernels of the 8-bit products with token and channel scales: which
sizes run on them (checked without a GPU), then those sizes against the 64-bit
references of tests/i8_ref.py -- every number of k steps and rest, ragged and
whole tiles, both output stores, bias, the ends of the ranges -- and bit for bit
against the streaming kernels."""
import numpy as np
import pytest

import i8_ref
import synth
from gpu_cases import to_gpu

INLINE, STREAM, T128, T256, SOME_HALVES, HALVES = range(6)

# 1 to 13 steps of 128 bytes of k, whole and not (the kernels take six at a
# time, then up to five)
KS = (32, 128, 160, 352, 384, 512, 544, 640, 736, 768, 896, 1024, 1120, 1280, 1376, 1536, 1632)
# (m, outputs plain, outputs gated, form): outputs that end inside a tile and an
# element, outputs in whole tiles, tokens either way
SIZES = [(130, 8301, 5003, T128), (65, 8257, 4163, T128), (256, 8320, 4160, T128), (333, 6001, 3003, T128),
         (300, 15009, 7505, HALVES), (512, 14336, 7168, HALVES),
         (1100, 8449, 4225, T256), (1280, 8192, 4096, T256),
         (1100, 16643, 8323, SOME_HALVES), (1100, 16640, 8320, SOME_HALVES), (1800, 9985, 4993, SOME_HALVES)]


def _form(n, k, m, gated):
    import moe_expert_ffn_q8_amd as q
    return q.raw.q8v_i8_form(n, k, m, gated)


@pytest.mark.parametrize("m,n,n_ff,form", SIZES)
def test_forms(m, n, n_ff, form):
    """The sizes below run on the kernel they are meant for."""
    for k in KS + (131040,):
        assert _form(n, k, m, 0) == form and _form(n_ff, k, m, 1) == form


def test_forms_of_the_other_sizes():
    """The listed kinds: few values, few rows, small matrices; refusals."""
    assert _form(768, 768, 1, 0) == INLINE and _form(768, 2048, 4, 1) == INLINE
    assert _form(768, 8192, 2, 0) == INLINE and _form(262144, 8192, 2, 0) == STREAM
    assert _form(262144, 2048, 64, 0) == STREAM and _form(17000, 2048, 64, 1) == STREAM
    assert _form(330, 1376, 600, 0) == STREAM
    assert _form(17000, 2048, 65, 0) == T128
    for bad, status in (((8, 33, 1, 0), -2), ((0, 32, 1, 0), -2), ((8, 32, 0, 0), -2),
                        ((8, 131072, 1, 0), -4), ((1 << 28, 32, 1, 0), -4), ((1 << 20, 32, 1 << 20, 0), -4)):
        assert _form(*bad) == status
    # every size that the calls take has a kernel
    for m in (1, 64, 65, 1 << 9, 1 << 18, 1 << 27):
        for n in (1, 512, (1 << 36) // m):
            if n <= 1 << 27:
                for gated in (0, 1):
                    assert 0 <= _form(n, 32, m, gated) <= HALVES


@pytest.fixture(scope="module")
def q():
    import torch
    import moe_expert_ffn_q8_amd as q
    yield q
    torch.cuda.empty_cache()


def _operands(m, rows, k, seed):
    """Codes and scales on the GPU: sums are about 5500 sqrt(k), gates of a few
    units."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + k)
    def codes(r):
        return torch.randint(-128, 128, (r, k), dtype=torch.int8, device="cuda", generator=g)
    def scales(n, a):
        return (torch.rand(n, device="cuda", generator=g) + 0.5) * a
    return codes(m), scales(m, 30.0 / (k ** 0.5 * 5500)), codes(rows), scales(rows, 1.0), g


def _reference(x, s, w, ws, bias, gated):
    """(value, bound) in 64 bits on the GPU, as product() and gated() of
    tests/i8_ref.py form them -- but for h where sigmoid(g) is below the smallest
    normal number, 2^-126, and may become 0: that is g < -126 ln 2 = -87.3365, and
    |g| exp(g), falling there, is at most 87.3366 * 2^-126 = 1.0267e-36."""
    import torch
    u = 1.01 * i8_ref.U
    # (the sums are whole numbers below 2^31: exact in any order)
    p = torch.mm(x.double(), w.double().t().contiguous()) * s.double()[:, None] * ws.double()
    if not gated:
        y = p if bias is None else p + bias.double()
        return y, u * ((3 if bias is None else 2) * p.abs() + y.abs()) + 2.0 ** -149
    n = p.shape[1] // 2
    g, up = p[:, :n], p[:, n:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = g * sig * up
    return h, u * h.abs() * (3 * (1 + g.abs() * (1 - sig)) + 13) + 1.03e-36 * up.abs() + 2.0 ** -148


def _close(got, ref, t, what):
    """i8_ref.assert_close on the GPU, for finite values inside t's range."""
    val, bound = ref
    tol = bound + i8_ref.HALF_STEP[t] * (val.abs() + bound) + i8_ref.SUBNORMAL[t]
    err = (got.double() - val).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max()):.2f} of the tolerance"


def _check(q, x, s, w, ws, bias, ref, t, gated, what):
    """Into a tensor of its own and into the middle of a wider one."""
    import torch
    m, cols = ref[0].shape
    tt = i8_ref.torch_type(t)
    fn, name = (q.i8_up_gate_swiglu, "h") if gated else (q.i8_matmul, "y")
    kw = {} if gated else {"bias": bias}
    whole = torch.full((m, cols), 5.5, dtype=tt, device="cuda")
    fn(x, w, ws, x_scale=s, **{name: whole}, **kw)
    _close(whole, ref, t, what)
    buf = torch.full((m + 2, cols + 7), 5.5, dtype=tt, device="cuda")
    out = buf[1:m + 1, 3:3 + cols]
    fn(x, w, ws, x_scale=s, **{name: out}, **kw)
    assert torch.equal(out, whole), what
    out.fill_(5.5)
    assert bool((buf == 5.5).all()), what


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("k", KS)
def test_steps(q, k, gated):
    """Each number of steps of k, on every kind of tile, the types in turn."""
    import torch
    for j, (m, n, n_ff, form) in enumerate(SIZES):
        t = i8_ref.TYPES[(k // 32 + j) % 3]
        cols, rows = (n_ff, 2 * n_ff) if gated else (n, n)
        x, s, w, ws, g = _operands(m, rows, k, j)
        bias = None if gated or j % 2 else torch.randn(rows, device="cuda", generator=g)
        _check(q, x, s, w, ws, bias, _reference(x, s, w, ws, bias, gated), t, gated, f"{m}x{k}x{cols} {t}")


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,n_ff,form", SIZES)
def test_types_and_bias(q, m, n, n_ff, form, gated):
    """Every size in every type, with and without bias."""
    import torch
    k = 416
    cols, rows = (n_ff, 2 * n_ff) if gated else (n, n)
    x, s, w, ws, g = _operands(m, rows, k, 11)
    for bias in (None,) if gated else (None, torch.randn(rows, device="cuda", generator=g)):
        ref = _reference(x, s, w, ws, bias, gated)
        for t in i8_ref.TYPES:
            _check(q, x, s, w, ws, bias, ref, t, gated, f"{m}x{k}x{cols} {t}")


@pytest.mark.gpu
@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n,n_ff,form", [s for s in SIZES if s[0] not in (256, 512, 1280)])
def test_same_bits_as_the_streaming_kernels(q, m, n, n_ff, form, t):
    """A token's outputs alone, among few and among many; tokens quantized
    inside the call and before it."""
    import torch
    k = 1376
    tt = i8_ref.torch_type(t)
    x, s, codes, scales, g = _operands(m, max(n, 2 * n_ff), k, 12)
    f = torch.randn((m, k), device="cuda", generator=g).to(tt)
    fc, fs = q.i8_quantize_rows(f)
    bias = torch.randn(n, device="cuda", generator=g)
    work = q.i8_workspace(m, k, "cuda")
    for fn, cols, rows, kw in ((q.i8_matmul, n, n, {"bias": bias}),
                               (q.i8_up_gate_swiglu, n_ff, 2 * n_ff, {})):
        gated = int(fn is q.i8_up_gate_swiglu)
        w, ws = codes[:rows], scales[:rows]
        full = fn(x, w, ws, x_scale=s, dtype=tt, **kw)
        for a, b in ((0, 1), (m - 1, m), (7, 10), (20, 36), (m - 64, m)):
            assert _form(cols, k, b - a, gated) in (INLINE, STREAM)
            assert torch.equal(fn(x[a:b], w, ws, x_scale=s[a:b], dtype=tt, **kw), full[a:b]), (fn, a, b)
        full = fn(f, w, ws, ws=work, dtype=tt, **kw)
        assert torch.equal(full, fn(fc, w, ws, x_scale=fs, dtype=tt, **kw))
        for a, b in ((0, 1), (m - 3, m), (30, 71 if m > 71 else 65)):
            assert torch.equal(fn(f[a:b], w, ws, ws=work, dtype=tt, **kw), full[a:b]), (fn, a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,form", [(300, 8301, T128), (512, 14336, HALVES), (1100, 8449, T256)])
def test_widest_rows(q, m, n, form):
    """Tokens, then weights, whose rows lie 4 MiB apart: offsets of a tile up to
    2^30 bytes."""
    import torch
    k = 160
    assert _form(n, k, m, 0) == form
    if torch.cuda.mem_get_info()[0] < (n << 22) + (8 << 30):
        pytest.skip("needs 70 GB of free GPU memory")
    x, s, w, ws, _ = _operands(m, n, k, 13)
    y = q.i8_matmul(x, w, ws, x_scale=s)
    _close(y, _reference(x, s, w, ws, None, False), "fp32", "close")
    for far in ("tokens", "weights"):
        wide = torch.empty((m if far == "tokens" else n, 1 << 22), dtype=torch.int8, device="cuda")
        wide[:, :k] = x if far == "tokens" else w
        a, b = (wide[:, :k], w) if far == "tokens" else (x, wide[:, :k])
        assert torch.equal(q.i8_matmul(a, b, ws, x_scale=s), y), far
        if n % 2 == 0:
            h = q.i8_up_gate_swiglu(x, w, ws, x_scale=s)
            assert torch.equal(q.i8_up_gate_swiglu(a, b, ws, x_scale=s), h), far
        del wide, a, b


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,form", [(65, 8301, T128), (512, 14336, HALVES)])
def test_extreme_codes(q, m, n, form):
    """The largest sums int32 holds (-128 everywhere, k = 131040)."""
    import torch
    k = 131040
    assert _form(n, k, m, 0) == form
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1::3] = 127
    w[2::3, ::2] = 127
    sums = np.array([16384 * k, -128 * 127 * k, (16384 - 128 * 127) * (k // 2)], np.float64)
    y = q.i8_matmul(x, w, torch.ones(n, device="cuda"), x_scale=torch.ones(m, device="cuda"))
    want = to_gpu(np.resize(sums, n).astype(np.float32))
    assert bool((y == want).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,n_ff,form", [SIZES[0], SIZES[4], SIZES[6]])
def test_special_scales(q, m, n, n_ff, form):
    """A NaN row stays NaN and alone so, zero rows give the bias, scales at the
    ends of fp32 give infinities and zeros as IEEE products do."""
    x, s, w, ws, g = _operands(m, n, 256, 14)
    cx, sx, cw, sw = (v.cpu().numpy() for v in (x, s, w, ws))
    sx[0], sx[1], sx[2] = np.nan, 0.0, 3e37
    sw[5], sw[6] = 0.0, np.nan
    bias = synth.rng("i8tiles", str(n)).normal(size=n).astype(np.float32)
    y = q.i8_matmul(x, w, to_gpu(sw), x_scale=to_gpu(sx), bias=to_gpu(bias)).cpu().numpy()
    s = i8_ref.sums(cx, cw).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = ((s * sx[:, None]).astype(np.float64) * sw + bias).astype(np.float32)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    assert np.array_equal(np.isinf(y), np.isinf(ref))
    assert np.array_equal(y[1, :5], bias[:5]) and np.array_equal(y[3:, 5], np.broadcast_to(bias[5], m - 3))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n_ff,form", [(130, 5003, T128), (512, 7168, HALVES), (1100, 4225, T256)])
def test_silu_range(q, m, n_ff, form):
    """Gates from -120 to 120: products of one code, scales placed so."""
    assert _form(n_ff, 32, m, 1) == form
    g = np.linspace(-120, 120, n_ff).astype(np.float32)
    cw = np.zeros((2 * n_ff, 32), np.int8)
    cw[:, 0] = 1
    cx = np.zeros((m, 32), np.int8)
    cx[:, 0] = 1
    one = np.ones(m, np.float32)
    sw = np.concatenate([g, np.ones(n_ff, np.float32)])
    h = q.i8_up_gate_swiglu(to_gpu(cx), to_gpu(cw), to_gpu(sw), x_scale=to_gpu(one))
    ref = _reference(to_gpu(cx[:1]), to_gpu(one[:1]), to_gpu(cw), to_gpu(sw), None, True)
    _close(h[0:1], ref, "fp32", f"{m}x{n_ff}")
    assert bool((h == h[0]).all())
