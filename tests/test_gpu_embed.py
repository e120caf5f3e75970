"""Embedding rows by token on the GPU: bit for bit against fp32 products in
numpy, from every table format to every output type."""
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


def _rounded(v, t):
    """fp32 values as type t holds them, and back."""
    import torch
    return torch.from_numpy(v).to(i8_ref.torch_type(t)).double().numpy()


def _same(got, want, t):
    got = got.double().cpu().numpy()
    want = _rounded(want, t)
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | np.isnan(want)))[:4]


def _tokens(rng, m, n):
    tok = rng.integers(0, n, m).astype(np.int32)
    tok[:2] = (n - 1, 0)[:m]
    return tok


SIZES = [(1, 1, 32), (2, 9, 64), (5, 100, 256), (33, 1000, 768), (300, 257, 2048), (3, 17, 14336),
         (700, 3000, 96), (1025, 50, 4096)]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("r8", [False, True])
def test_q8_0(q, orc, m, n, k, r8, t):
    rng = synth.rng("emb", str(m), str(n), str(k))
    w = orc.quantize_rows((rng.normal(size=(n, k)) * 0.02).astype(np.float32))
    blocks = w.reshape(n, k // 32, 34)
    d = blocks[:, :, :2].copy().view(np.float16).astype(np.float32)
    rows = (blocks[:, :, 2:].view(np.int8).astype(np.float32) * d).reshape(n, k)
    table = to_gpu(w)
    if r8:
        table = q.q8_0_repack_r8(table, n, k)
    tok = _tokens(rng, m, n)
    scale = np.float32(np.sqrt(k))
    y = q.q8_0_embed_rows(table, to_gpu(tok), n, k, scale=float(scale), r8=r8, dtype=i8_ref.torch_type(t))
    _same(y, rows[tok] * scale, t)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_int8(q, m, n, k, t):
    rng = synth.rng("emb8", str(m), str(n), str(k))
    c = rng.integers(-128, 128, size=(n, k)).astype(np.int8)
    s = (rng.random(n) * 1e-3).astype(np.float32)
    tok = _tokens(rng, m, n)
    y = q.embed_rows(to_gpu(c), to_gpu(tok), scale=0.7, table_scale=to_gpu(s), dtype=i8_ref.torch_type(t))
    _same(y, c[tok].astype(np.float32) * s[tok][:, None] * np.float32(0.7), t)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("table_t", i8_ref.TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 5, 7), (4, 9, 33), (17, 40, 1003), (300, 30, 8), (2, 3, 4099),
                                   (65, 11, 768)])
def test_floats(q, m, n, k, table_t, t):
    """Any row length; rows of the table and of y that start anywhere."""
    import torch
    rng = synth.rng("embf", str(m), str(n), str(k), table_t)
    tt = i8_ref.torch_type(table_t)
    table = torch.full((n, k + 3), 1e4, dtype=tt, device="cuda")[:, 1:k + 1]
    table.copy_(to_gpu(rng.normal(size=(n, k)).astype(np.float32)))
    tok = _tokens(rng, m, n)
    buf = torch.full((m, k + 5), -7.0, dtype=i8_ref.torch_type(t), device="cuda")
    y = q.embed_rows(table, to_gpu(tok), scale=1.5, y=buf[:, 2:k + 2])
    _same(y, table.float().cpu().numpy()[tok] * np.float32(1.5), t)
    assert bool((buf[:, :2] == -7).all()) and bool((buf[:, k + 2:] == -7).all())


def test_tokens_outside(q, orc):
    """A row of NaN, and only that row."""
    import torch
    n, k = 20, 64
    rng = synth.rng("embout")
    f = to_gpu(rng.normal(size=(n, k)).astype(np.float32))
    w = q.q8_0_quantize_rows(f)
    c, s = q.i8_quantize_rows(f)
    tok = torch.tensor([3, -1, 5, n, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    bad = [False, True, False, True, True, True, False]
    for y in (q.embed_rows(f, tok), q.embed_rows(c, tok, table_scale=s), q.q8_0_embed_rows(w, tok, n, k),
              q.q8_0_embed_rows(q.q8_0_repack_r8(w, n, k), tok, n, k, r8=True),
              q.embed_rows(f, tok, dtype=torch.float16)):
        assert torch.isnan(y).all(1).tolist() == bad
        assert torch.isnan(y).any(1).tolist() == bad


def test_no_tokens(q):
    import torch
    y = q.embed_rows(torch.ones((4, 8), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 8)


def test_far_rows(q):
    """Table rows past 2^32 bytes, outputs past 2^32 bytes."""
    import torch
    n, k = 70000, 65536
    table = torch.empty((n, k), dtype=torch.int8, device="cuda")
    s = torch.ones(n, device="cuda")
    at = torch.tensor([n - 1, 0, 65537, 32768, n - 2], dtype=torch.int32, device="cuda")
    for i, r in enumerate(at.tolist()):
        table[r] = i + 1
    y = q.embed_rows(table, at, table_scale=s, dtype=torch.bfloat16)
    assert torch.equal(y, torch.arange(1, 6, device="cuda").bfloat16()[:, None].expand(5, k))
    tok = at.repeat(8000)
    y = q.embed_rows(table, tok, table_scale=s, dtype=torch.bfloat16)
    want = torch.arange(1, 6, device="cuda").bfloat16().repeat(8000)
    assert torch.equal(y[:, 0], want) and torch.equal(y[:, -1], want)
