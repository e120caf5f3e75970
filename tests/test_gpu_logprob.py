"""Log probabilities of logit rows on the GPU against 64-bit references
(tests/i8_ref.py derives the bounds; ids exactly)."""
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


def _run(q, x, t, tokens=None, n_top=0, offset=0, pad=0):
    """x: fp32 [m][v]; rows of v + pad elements starting `offset` elements into
    the buffer.  Returns the outputs and the values the logits hold."""
    import torch
    m, v = x.shape
    tt = i8_ref.torch_type(t)
    buf = torch.full((m * (v + pad) + offset + 8,), 1e4, dtype=tt, device="cuda")
    logits = buf[offset:offset + m * (v + pad)].view(m, v + pad)[:, :v] if m else buf[:0].view(0, v)
    logits.copy_(to_gpu(x.astype(np.float32)))
    held = logits.double().cpu().numpy()
    out = q.logprob_outputs(m, 0 if tokens is None else tokens.shape[1], n_top, "cuda")
    for o in out:
        if o is not None:
            o.fill_(-7)
    ws = q.logprob_workspace(m, v, n_top, "cuda")
    ws.fill_(255)
    q.logprob_rows(logits, None if tokens is None else to_gpu(tokens), n_top=n_top, ws=ws, out=out)
    return out, held


def _check(q, x, t, tokens=None, n_top=0, **kw):
    out, held = _run(q, x, t, tokens, n_top, **kw)
    i8_ref.assert_logprobs(out, i8_ref.logprobs(held, tokens, n_top))
    return out


def _logits(rng, m, v):
    x = rng.normal(size=(m, v)) * 2.5
    x[np.arange(m), rng.integers(0, v, m)] += 9
    return x


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,v", [(1, 1), (2, 2), (3, 7), (1, 63), (5, 64), (2, 65), (3, 300), (1, 1000),
                                 (33, 1025), (4, 4097), (2, 16384), (1, 32000), (7, 32000),
                                 (1, 50257), (300, 2049), (70, 50257), (2, 131071), (1, 262144),
                                 (9, 262144), (700, 513)])
def test_sizes(q, m, v, t):
    rng = synth.rng("lp", str(m), str(v), t)
    tokens = rng.integers(0, v, size=(m, 2)).astype(np.int32)
    for n_top in sorted({0, 1, min(v, 5), min(v, 20), min(v, 64)}):
        _check(q, _logits(rng, m, v), t, tokens, n_top)


@pytest.mark.parametrize("m,v,tops", [(1, 1300000, (0, 20, 64)), (2, 700001, (1, 64)),
                                      (3, 400000, (5, 20, 40)), (70001, 37, (0, 5))])
def test_many_parts_and_rows(q, m, v, tops):
    """Rows in up to 64 parts, and more rows than one launch takes."""
    rng = synth.rng("lpparts", str(m), str(v))
    x = _logits(rng, m, v)
    tokens = rng.integers(0, v, size=(m, 1)).astype(np.int32)
    for n_top in tops:
        _check(q, x, "bf16" if m == 3 else "fp32", tokens, n_top)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (7, 8), (1, 7), (2, 3)])
def test_row_starts(q, offset, pad, t):
    """Rows that start anywhere; the values beside a row are never taken."""
    rng = synth.rng("lpstart", str(offset), str(pad))
    for m, v in ((3, 5), (4, 1003), (2, 50257), (1, 70001)):
        _check(q, _logits(rng, m, v), t, rng.integers(0, v, size=(m, 1)).astype(np.int32),
               min(v, 20), offset=offset, pad=pad)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [50, 1000, 33000, 262144])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "few", "blocks", "peak", "zeros",
                                  "strided", "lane"])
def test_orders(q, v, kind, t):
    """Orders that defeat a threshold, and ties: the lowest index first."""
    rng = synth.rng("lporder", kind, str(v))
    i = np.arange(v)
    x = {"rising": i * (20.0 / v), "falling": -i * (20.0 / v), "equal": np.full(v, 1.5),
         "few": rng.integers(0, 3, v).astype(float), "blocks": (i // 997) * 0.25,
         "peak": np.where(i == v // 2, 60.0, 0.0), "zeros": np.where(i % 3, 0.0, -0.0),
         "strided": np.where(i % 64 == 17, 5 + i * (5.0 / v), rng.normal(size=v)),
         "lane": np.where(i % 1024 < 16, 3 + rng.normal(size=v), rng.normal(size=v) - 9)}[kind]
    for n_top in (1, 20, 50):
        _check(q, np.stack([x, x[::-1]]), t, np.array([[0], [v - 1]], np.int32), n_top)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [40, 1500, 50257, 262144])
def test_masked_rows(q, v, t):
    """Banned tokens, fewer visible tokens than alternatives, none at all, and
    the type's lowest value as a mask."""
    rng = synth.rng("lpmask", str(v))
    low = {"fp32": -3.4028235e38, "fp16": -65504.0, "bf16": -3.3895314e38}[t]
    x = _logits(rng, 8, v)
    x[0, rng.random(v) < 0.5] = -np.inf
    x[1, :] = -np.inf
    x[2, :] = -np.inf
    x[2, v // 3] = 0.25
    x[3, 5:] = -np.inf
    x[4, :v - 3] = -np.inf
    x[5, rng.random(v) < 0.9] = low
    x[6, :] = low
    x[7, :] = -np.inf
    x[7, v - 1] = low
    tokens = np.array([[0, v - 1]] * 8, np.int32)
    for n_top in (1, 20, 40):
        out = _check(q, x, t, tokens, n_top)
    assert float(out.entropy[1]) == 0 and float(out.lse[1]) == -np.inf


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [1000, 12289, 50257, 262144])
def test_low_logits_on_the_way(q, v, t):
    """-infinity, and values whose product with log2 e overflows, that first come
    up late in a row, in one place of it or everywhere behind it, beside small
    and large references."""
    rng = synth.rng("lplow", str(v))
    x = _logits(rng, 8, v)
    x[0, v - 2] = -np.inf
    x[1, v // 2:] = -np.inf
    x[2, v // 3] = -3.1e38
    x[3, 2 * v // 3:] = -2.5e38
    x[4] = x[4] * 1e29 + 1e30
    x[4, v // 2] = -np.inf
    x[5, :-1] = -2e38                 # a reference far above everything else
    x[6] = -2.2e38                    # nothing above the first reference
    x[6, v // 5] = -np.inf
    x[7, ::7] = -1.5e38
    tokens = np.array([[0, v // 2]] * 8, np.int32)
    for n_top in (0, 3, 20, 25, 64):
        _check(q, x, t, tokens, n_top)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [64, 3000, 50257, 200000])
def test_nan_and_infinity(q, v, t):
    """A row with a NaN or +infinity is NaN throughout, its neighbours are not;
    ids stay in range and distinct: infinity first, NaN last."""
    rng = synth.rng("lpnan", str(v))
    x = _logits(rng, 6, v)
    x[0, v // 2] = np.nan
    x[2, 3] = np.inf
    x[2, v - 1] = np.inf
    x[3, :] = np.nan
    x[4, :] = -np.inf
    x[4, 1] = np.nan
    for n_top in (1, 20, 64):
        out = _check(q, x, t, np.array([[1], [1], [3], [0], [0], [2]], np.int32), n_top)
        assert out.top_ids[2, 0] == 3
        ids = np.sort(out.top_ids.cpu().numpy(), axis=1)
        assert (np.diff(ids, axis=1) > 0).all() and ids.min() >= 0 and ids.max() < v


def test_given_tokens(q):
    """None, many, repeated, out of range (NaN)."""
    rng = synth.rng("lpgiven")
    x = _logits(rng, 5, 1234)
    tokens = rng.integers(0, 1234, size=(5, 300)).astype(np.int32)
    tokens[:, 7] = tokens[:, 8]
    tokens[1, 3], tokens[2, 0], tokens[4, 299], tokens[0, 0] = -1, 1234, 2 ** 31 - 1, -2 ** 31
    _check(q, x, "fp32", tokens, 3)
    out, _ = _run(q, x, "fp32", None, 2)
    assert out.logprob is None
    # one token per row as a vector
    import torch
    g = to_gpu(x.astype(np.float32))
    ws = q.logprob_workspace(5, 1234, 0, "cuda")
    one = q.logprob_rows(g, to_gpu(tokens[:, 5]), ws=ws)
    two = q.logprob_rows(g, to_gpu(tokens[:, 5:6]), ws=ws)
    assert torch.equal(one.logprob, two.logprob) and one.top_ids is None
    assert q.logprob_rows(g[:0], ws=ws).lse.shape == (0,)
    with pytest.raises(q.Q8Error, match="SHAPE"):
        q.logprob_rows(g, n_top=-1, ws=ws)
    with pytest.raises(q.Q8Error, match="WORKSPACE"):
        q.logprob_rows(g)


def test_same_bits_again(q):
    import torch
    rng = synth.rng("lpsame")
    for m, v in ((1, 262144), (3, 50257), (600, 5000)):
        x = _logits(rng, m, v)
        a, _ = _run(q, x, "bf16", np.zeros((m, 1), np.int32), 20)
        b, _ = _run(q, x, "bf16", np.zeros((m, 1), np.int32), 20)
        for r, s in zip(a, b):
            assert torch.equal(r, s)
