"""Sampling from rows of logits on the GPU against the definition by sorting
(tests/ops_ref.py): tokens, sizes of what is kept, log probabilities."""
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


def _settings(m, **kw):
    """Settings of m rows: numbers, or an array of m."""
    full = dict(u=0.5, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    full.update(kw)
    return {k: np.broadcast_to(np.asarray(v, np.int32 if k == "top_k" else np.float32), (m,)).copy()
            for k, v in full.items()}


def _run(q, x, t, offset=0, pad=0, **kw):
    """(outputs, the values that the logits hold, settings)."""
    import torch
    m, v = x.shape
    s = _settings(m, **kw)
    buf = torch.full((m * (v + pad) + offset + 8,), 1e4, dtype=i8_ref.torch_type(t), device="cuda")
    logits = buf[offset:offset + m * (v + pad)].view(m, v + pad)[:, :v]
    logits.copy_(to_gpu(x.astype(np.float32)))
    held = logits.double().cpu().numpy()
    out = q.sample_outputs(m, "cuda")
    for o in out:
        o.fill_(-7)
    ws = q.sample_workspace(m, v, "cuda")
    ws.fill_(255)
    q.sample_rows(logits, ws=ws, out=out, **{k: to_gpu(a) for k, a in s.items()})
    return out, held, s


def _check(q, x, t, most_open=0.02, **kw):
    out, held, s = _run(q, x, t, **kw)
    got = np.stack([o.double().cpu().numpy() for o in out], 1)
    open_rows = 0
    for i in range(len(x)):
        ref = ops_ref.sample_row(held[i], s["u"][i], s["temperature"][i], s["top_k"][i], s["top_p"][i], s["min_p"][i])
        open_rows += ops_ref.assert_sample(got[i], ref, f"row {i} {({k: a[i] for k, a in s.items()})}")
    # a target within the sums' units of a border is rare
    assert open_rows <= max(1, most_open * len(x))
    return out


def _logits(rng, m, v, flat=1.5):
    """Rows from sure to flat."""
    x = rng.normal(size=(m, v)) * flat
    r = np.arange(1, 17)
    for i in range(m):
        at = rng.integers(0, v, 16)
        x[i, at] += (0.3 + 0.9 * rng.random()) * 16 - 1.2 * np.log(r)
    return x


SETTINGS = [dict(), dict(temperature=0.6), dict(top_k=1), dict(top_k=20), dict(top_k=300), dict(top_p=0.9),
            dict(top_p=0.999), dict(min_p=0.05), dict(top_k=50, top_p=0.95, temperature=0.8),
            dict(top_k=40, top_p=0.8, min_p=0.02, temperature=1.4), dict(temperature=0.0)]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,v", [(1, 1), (2, 2), (3, 7), (5, 64), (4, 65), (3, 300), (8, 1000), (33, 1025), (4, 4097),
                                 (6, 16384), (2, 16390), (1, 32000), (7, 32000), (5, 50257), (300, 2049), (3, 131071),
                                 (2, 262144), (9, 262144)])
def test_sizes(q, m, v, t):
    rng = synth.rng("sample", str(m), str(v), t)
    for kw in SETTINGS if v < 100000 else SETTINGS[::3]:
        _check(q, _logits(rng, m, v), t, u=rng.random(m), **kw)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [50, 1000, 33000, 262144])
def test_flat_rows(q, v, t):
    """What is kept is a large part of the vocabulary."""
    rng = synth.rng("sampleflat", str(v), t)
    m = 4
    for flat in (0.02, 0.7):
        for kw in (dict(), dict(top_p=0.95), dict(top_p=0.5, temperature=2.0), dict(top_k=v // 2 + 1),
                   dict(top_k=v // 3 + 1, top_p=0.7, min_p=0.1)):
            _check(q, rng.normal(size=(m, v)) * flat, t, most_open=0.5, u=rng.random(m), **kw)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [5, 64, 1000, 33000, 262144])
def test_equal_logits(q, v, t):
    """Equal weights: every target is a whole number, ties go by index."""
    import torch
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24], np.float32)
    x = np.full((5, v), 1.5)
    out = _check(q, x, t, u=u)
    assert out.ids.tolist() == [min(v - 1, int(np.float64(a) * v)) for a in u]
    assert out.kept.tolist() == [v] * 5
    out = _check(q, x, t, u=u, top_p=0.5)
    assert out.kept.tolist() == [-(-v // 2)] * 5
    out = _check(q, x, t, u=u, top_k=3)
    assert out.kept.tolist() == [min(3, v)] * 5 and int(out.ids.max()) == min(2, v - 1)
    # two levels, all of the higher one behind the lower one
    x = np.zeros((5, v))
    x[:, v // 2:] = 30.0
    out = _check(q, x, t, most_open=1.0, u=u, top_k=max(1, v // 4))
    assert int(out.ids.min()) == v // 2


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("v", [40, 1500, 50257, 262144])
def test_masked_rows(q, v, t):
    """Banned tokens, few tokens left, one, none; the type's lowest value and
    -1e9 as masks; infinities and NaN."""
    rng = synth.rng("samplemask", str(v), t)
    low = {"fp32": -3.4028235e38, "fp16": -65504.0, "bf16": -3.3895314e38}[t]
    x = _logits(rng, 12, v)
    x[0, rng.random(v) < 0.5] = -np.inf
    x[1] = -np.inf
    x[2, :] = -np.inf
    x[2, v // 3] = -5.0
    x[3, rng.random(v) < 0.9] = low
    x[4] = low
    x[5, 3] = np.nan
    x[6, v - 1] = np.inf
    x[7, 10:] = -np.inf
    x[8] = np.where(rng.random(v) < 0.99, -1e9 if t != "fp16" else -6e4, x[8])
    x[9, :] = -np.inf
    x[9, 2] = np.nan
    x[10] = -1e9 if t != "fp16" else -6e4
    for kw in (dict(), dict(top_k=20), dict(top_p=0.9), dict(top_k=v), dict(min_p=0.3), dict(temperature=0.0),
               dict(top_k=30, top_p=0.7, temperature=0.5)):
        out = _check(q, x, t, u=rng.random(12), **kw)
        assert out.ids[1] == -1 and out.kept[1] == 0 and out.logprob[1] == -np.inf
        assert out.ids[2] == v // 3 and out.kept[2] == 1 and out.logprob[2] == 0
        for i in (5, 6, 9):
            assert out.ids[i] == -1 and np.isnan(float(out.logprob[i]))


def test_ends_of_the_settings(q):
    """u, temperatures, top_p and min_p at and beyond their ends."""
    rng = synth.rng("sampleends")
    v = 3000
    x = np.repeat(_logits(rng, 1, v), 24, axis=0)
    kw = _settings(24, u=0.4)
    kw["u"][:6] = (0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, np.nan)
    kw["temperature"][6:13] = (0.0, -1.0, np.nan, 1e-30, 1e-45, 1e30, np.inf)
    kw["top_p"][13:18] = (0.0, -1.0, 1.0, 2.0, np.nan)
    kw["min_p"][18:22] = (1.0, 5.0, -1.0, np.nan)
    kw["top_k"][22:24] = (-5, 2 ** 31 - 1)
    ref = {k: a.copy() for k, a in kw.items()}
    ref["top_p"][17], ref["min_p"][21] = 1.0, 0.0
    for t in i8_ref.TYPES:
        out, held, _ = _run(q, x, t, **kw)
        got = np.stack([o.double().cpu().numpy() for o in out], 1)
        for i in range(24):
            r = ops_ref.sample_row(held[i], ref["u"][i], ref["temperature"][i], ref["top_k"][i], ref["top_p"][i],
                                   ref["min_p"][i])
            ops_ref.assert_sample(got[i], r, f"row {i}")
        assert out.ids[4] == out.ids[0] == out.ids[5]
        assert out.ids[2] == out.ids[3]
        assert out.kept[13] == 1 and out.kept[18] == out.kept[19]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (7, 8), (2, 3)])
def test_row_starts(q, offset, pad, t):
    """Rows that start anywhere; the values beside a row are never drawn."""
    rng = synth.rng("samplestart", str(offset), str(pad))
    for m, v in ((3, 5), (4, 1003), (2, 50257), (2, 70001)):
        for kw in (dict(), dict(top_k=30, top_p=0.9)):
            _check(q, _logits(rng, m, v), t, u=rng.random(m), offset=offset, pad=pad, **kw)


@pytest.mark.parametrize("kind", ["rising", "falling", "few", "blocks", "peak", "strided", "far", "zeros"])
@pytest.mark.parametrize("v", [1000, 33000, 262144])
def test_orders(q, v, kind):
    rng = synth.rng("sampleorder", kind, str(v))
    i = np.arange(v)
    x = {"rising": i * (20.0 / v), "falling": -i * (20.0 / v), "few": rng.integers(0, 3, v).astype(float),
         "blocks": (i // 997) * 0.25, "peak": np.where(i == v // 2, 60.0, 0.0),
         "strided": np.where(i % 64 == 17, 5 + i * (5.0 / v), rng.normal(size=v)),
         "far": 1e8 + rng.integers(0, 64, v) * 8.0, "zeros": np.where(i % 3, 0.0, -0.0)}[kind]
    for t in ("fp32", "bf16"):
        for kw in (dict(), dict(top_k=20), dict(top_k=700), dict(top_p=0.9), dict(min_p=0.5, temperature=3.0)):
            _check(q, np.stack([x, x[::-1], x]), t, most_open=1.0, u=[0.1, 0.6, 0.97], **kw)


def test_each_row_its_settings(q):
    rng = synth.rng("samplemixed")
    m, v = 333, 5003
    kw = dict(u=rng.random(m), temperature=rng.choice([0.0, 0.6, 1.0, 1.3], m), top_k=rng.choice([0, 1, 20, 200], m),
              top_p=rng.choice([1.0, 0.95, 0.5], m), min_p=rng.choice([0.0, 0.05], m))
    _check(q, _logits(rng, m, v), "bf16", **kw)


def test_frequencies(q):
    """Tokens come as often as their probabilities say: u over a fine grid gives
    each kept token its share, and they go by the order."""
    import torch
    rng = synth.rng("samplefreq")
    m, v = 4096, 120
    x = np.repeat(rng.normal(size=(1, v)) * 2, m, axis=0)
    u = (np.arange(m) + 0.5) / m
    out, held, _ = _run(q, x, "fp32", u=u, top_k=30)
    order = np.argsort(-held[0], kind="stable")[:30]
    p = np.exp(held[0][order] - held[0].max())
    p /= p.sum()
    place = np.argsort(order)[np.searchsorted(np.sort(order), out.ids.cpu().numpy())]
    assert (np.diff(place) >= 0).all()
    share = np.bincount(place, minlength=30) / m
    assert np.abs(share - p).max() <= 1.0 / m


@pytest.mark.parametrize("m,v", [(70001, 37), (2, 1300000), (3, 700001)])
def test_many_rows_and_long_ones(q, m, v):
    rng = synth.rng("samplemany", str(m), str(v))
    if m > 1000:
        x = rng.normal(size=(m, v)) * 2
        out, held, s = _run(q, x, "bf16", u=rng.random(m), top_k=9, top_p=0.9)
        got = np.stack([o.double().cpu().numpy() for o in out], 1)
        for i in list(range(0, m, 511)) + [m - 1]:
            ops_ref.assert_sample(got[i], ops_ref.sample_row(held[i], s["u"][i], 1.0, 9, s["top_p"][i], 0.0), f"row {i}")
        return
    for kw in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.97)):
        _check(q, _logits(rng, m, v), "fp32", u=rng.random(m), most_open=0.5, **kw)


def test_far_rows(q):
    """Rows past 2^32 bytes."""
    import torch
    m, v = 20000, 131072
    x = torch.zeros((m, v), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(m, device="cuda") * 6
    x[torch.arange(m, device="cuda"), at] = 60.0
    u = torch.full((m,), 0.5, device="cuda")
    out = q.sample_rows(x, u, top_k=torch.full((m,), 5, dtype=torch.int32, device="cuda"),
                        ws=q.sample_workspace(m, v, "cuda"))
    assert torch.equal(out.ids, at.int()) and bool((out.kept == 5).all())


def test_repeats(q):
    """The same bits at every call, whatever the workspace holds, and for a row
    alone."""
    import torch
    rng = synth.rng("samplerepeat")
    m, v = 40, 50257
    x = to_gpu(_logits(rng, m, v).astype(np.float32)).bfloat16()
    kw = {k: to_gpu(a) for k, a in _settings(m, u=rng.random(m), top_p=0.97).items()}
    ws = q.sample_workspace(m, v, "cuda")
    first = q.sample_rows(x, ws=ws, **kw)
    for fill in (0, 255, 7):
        ws.fill_(fill)
        again = q.sample_rows(x, ws=ws, **kw)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    for i in (0, 17, 39):
        one = q.sample_rows(x[i:i + 1], ws=ws, **{k: a[i:i + 1] for k, a in kw.items()})
        assert all(torch.equal(a[0], b[i]) for a, b in zip(one, first))
