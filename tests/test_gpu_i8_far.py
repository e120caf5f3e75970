"""Operands and outputs past 2^31 and 2^32 bytes and elements, and the most
outputs a product takes, against 64-bit references on sampled rows."""
import numpy as np
import pytest

import i8_ref
import synth
from gpu_cases import to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    import moe_expert_ffn_q8_amd as q
    yield q
    torch.cuda.empty_cache()


def _codes(rows, k, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, (rows, k), dtype=torch.int8, device="cuda", generator=g)


def _scales(n, key):
    return (synth.rng("far", key).random(n) * 1e-3 + 1e-4).astype(np.float32)


def _np(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("m", [1, 5, 80, 300])
def test_far_weights(q, m):
    """Weights of 4.6 GB, in both forms: outputs of rows on both sides of 2^31
    and 2^32 bytes."""
    n, k = 70016, 65536
    w, x = _codes(n, k, 1), _codes(m, k, 2)
    sw, sx = _scales(n, "w"), _scales(m, "x")
    y = q.i8_matmul(x, w, to_gpu(sw), x_scale=to_gpu(sx))
    at = np.array([0, 1, 32767, 32768, 32769, 65535, 65536, 65537, n - 2, n - 1])
    ref, bound = i8_ref.product(_np(x), sx, _np(w[at.tolist()]), sw[at])
    i8_ref.assert_close(_np(y)[:, at], ref, bound, "fp32", "product")
    half = n // 2
    h = q.i8_up_gate_swiglu(x, w, to_gpu(sw), x_scale=to_gpu(sx))
    at = np.array([0, 32760, 32768, half - 1])
    rows = np.concatenate([at, at + half])
    ref, bound = i8_ref.gated(_np(x), sx, _np(w[rows.tolist()]), sw[rows])
    i8_ref.assert_close(_np(h)[:, at], ref, bound, "fp32", "gated")


@pytest.mark.parametrize("t", ["fp32", "bf16"])
def test_far_outputs(q, t):
    """2.15e9 outputs, rows sampled."""
    m, n, k = 131077, 16400, 32
    x, w = _codes(m, k, 3), _codes(n, k, 4)
    sx, sw = _scales(m, "x2"), _scales(n, "w2")
    y = q.i8_matmul(x, w, to_gpu(sw), x_scale=to_gpu(sx), dtype=i8_ref.torch_type(t))
    at = [0, 65000, 130944, m - 2, m - 1]
    ref, bound = i8_ref.product(_np(x[at]), sx[at], _np(w), sw)
    i8_ref.assert_close(_np(y[at].double()), ref, bound, t)


@pytest.mark.parametrize("m", [33, 1100])
def test_widest_rows(q, m):
    """Rows 4 MiB apart, the limit, as tokens and as weights."""
    import torch
    n, k = 300, 64
    wide = torch.zeros((m, 1 << 22), dtype=torch.int8, device="cuda")
    x = wide[:, :k]
    x.copy_(_codes(m, k, 5))
    w = _codes(n, k, 6)
    sx, sw = _scales(m, "x3"), _scales(n, "w3")
    y = q.i8_matmul(x, w, to_gpu(sw), x_scale=to_gpu(sx))
    ref, bound = i8_ref.product(_np(x), sx, _np(w), sw)
    i8_ref.assert_close(_np(y), ref, bound, "fp32", "tokens")
    y = q.i8_matmul(w, x, to_gpu(sx), x_scale=to_gpu(sw))
    i8_ref.assert_close(_np(y), ref.T, bound.T, "fp32", "weights")


def test_most_outputs(q):
    """m * n_ff = 2^36, the limit: 137 GB of binary16."""
    import torch
    m, n_ff, k = 1 << 27, 512, 32
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("needs 170 GiB of free GPU memory")
    x, w = _codes(m, k, 7), _codes(2 * n_ff, k, 8)
    sw = _scales(2 * n_ff, "w4")
    sx = torch.full((m,), 2.0 ** -6, dtype=torch.float32, device="cuda")
    h = q.i8_up_gate_swiglu(x, w, to_gpu(sw), x_scale=sx, dtype=torch.float16)
    at = [0, 255, 256, (1 << 26) - 1, (1 << 26) + 130, m - 257, m - 1]
    ref, bound = i8_ref.gated(_np(x[at]), np.full(len(at), 2.0 ** -6, np.float32), _np(w), sw)
    i8_ref.assert_close(_np(h[at].double()), ref, bound, "fp16")


def test_far_quantize(q):
    """9 GB of fp32 to 2.3 GB of codes."""
    import torch
    n, k = 70001, 32768
    x = torch.empty((n, k), device="cuda").normal_()
    codes, scale = q.i8_quantize_rows(x)
    at = [0, 16383, 16384, 32768, 65535, 65536, n - 1]
    c, s = i8_ref.quantize(_np(x[at]))
    assert np.array_equal(_np(codes[at]), c)
    assert np.array_equal(_np(scale[at]), s)


def test_far_logits(q):
    """Rows 2^31 + 5 logits apart, and one row of 2^28 + 3."""
    import torch
    v, stride = 5000, (1 << 31) + 5
    buf = torch.empty(2 * stride + v, dtype=torch.bfloat16, device="cuda")
    logits = buf.as_strided((3, v), (stride, 1))
    rng = synth.rng("farlp")
    logits.copy_(to_gpu((rng.normal(size=(3, v)) * 3).astype(np.float32)))
    tokens = np.array([[0, v - 1]] * 3, np.int32)
    out = q.logprob_rows(logits, to_gpu(tokens), n_top=7, ws=q.logprob_workspace(3, v, 7, "cuda"))
    i8_ref.assert_logprobs(out, i8_ref.logprobs(_np(logits.double()), tokens, 7))
    del buf, logits
    v = (1 << 28) + 3
    row = torch.empty((1, v), dtype=torch.bfloat16, device="cuda").normal_()
    row[0, v - 1] = 12.5
    row[0, 1 << 27] = 12.0
    tokens = to_gpu(np.array([[v - 1]], np.int32))
    out = q.logprob_rows(row, tokens, n_top=2, ws=q.logprob_workspace(1, v, 2, "cuda"))
    d = row[0].double()
    lse = float(torch.logsumexp(d, 0))
    entropy = lse - float((torch.exp(d - lse) * d).sum())
    assert out.top_ids[0].tolist() == [v - 1, 1 << 27]
    # a lane adds at most v / (64 parts * 1024 lanes) = 4096 terms one by one, the
    # rest in trees: their roundings, twice |d| + 3 = 15 of the terms, and those of
    # values below 32; the entropy takes W / S, |d| = 11.5 on average, from log S:
    # 1 + 2 * 11.5 times the sums' error
    tol = 2.0 ** -24 * (4096 + 32 + 2 * 16) + 2.0 ** -24 * 4 * 32
    assert abs(float(out.lse[0]) - lse) <= tol
    assert abs(float(out.logprob[0, 0]) - (12.5 - lse)) <= 2 * tol
    assert abs(float(out.entropy[0]) - entropy) <= 25 * tol
