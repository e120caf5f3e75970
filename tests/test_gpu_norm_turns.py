"""Norm rows where a workgroup takes several rows one after another (more rows
than are resident): every row against the same rows in calls of a few, which
give each workgroup one, and some of them against the 64-bit reference."""
import numpy as np
import pytest

import i8_ref
import ops_ref
import synth
from test_gpu_norm import _check_y, _host, _narrow

pytestmark = pytest.mark.gpu

SLICE = 199                # rows of a call in which no workgroup has two


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


def _random(g, m, n, t, size=1.0):
    """Rows that all differ, of different sizes."""
    import torch
    x = torch.randn((m, n), generator=g, device="cuda") * size
    x *= 0.25 + torch.rand((m, 1), generator=g, device="cuda") * 4
    x[:, torch.randint(n, (max(1, n // 300),), generator=g, device="cuda")] *= 12
    return x.to(i8_ref.torch_type(t))


# (n, rows): rows of one wave (four to a workgroup), of four and of eight waves, of 1 to
# 16 pieces a thread.  256 CUs hold at most 2048 workgroups of 256 threads, 1024 of 512; no
# count of rows divides by what is resident.
SIZES = [(96, 20011), (800, 9001), (2048, 5003), (4096, 5003), (8192, 2503), (14336, 1301), (32768, 1301), (65536, 1301)]
CASES = [dict(), dict(layer=True, gate="channel", bias=True), dict(post=True, gate="row"),
         dict(post=True, post_bias=True, layer=True, gate="row", alpha=0.5)]


@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("fp16", "fp16", "i8"), ("fp32", "fp32", "fp32"),
                                   ("bf16", "fp32", "fp16"), ("fp32", "fp16", "i8")], ids="-".join)
@pytest.mark.parametrize("n,m", SIZES)
def test_stream_over_many_rows(q, n, m, types):
    import torch
    xt, rt, yt = types
    g = torch.Generator(device="cuda")
    g.manual_seed(int(synth.rng("normturns", str(n), str(types)).integers(1 << 31)))
    yd = torch.int8 if yt == "i8" else i8_ref.torch_type(yt)
    x, r = _random(g, m, n, xt), _random(g, m, n, rt, 3.0)
    vec = lambda size, middle: middle + size * torch.randn(n, generator=g, device="cuda")
    rows = _random(g, m, n, xt, 0.3)
    rng = synth.rng("normturnrows", str(n))
    some = torch.from_numpy(np.unique(np.concatenate([[0, 1, 2, 3, m - 1], rng.integers(0, m, 12)]))).cuda()
    for case in CASES if n < 30000 else CASES[1:3]:
        layer, alpha = case.get("layer", False), case.get("alpha", 1.0)
        kw = dict(bias=vec(0.1, 0.0) if case.get("bias") else None, post_weight=vec(0.2, 1.0) if case.get("post") else None,
                  post_bias=vec(0.1, 0.0) if case.get("post_bias") else None, residual_scale=alpha, eps=1e-6, layer=layer,
                  dtype=yd)
        w = vec(0.2, 1.0)
        by_row = case.get("gate") == "row"
        gate = rows if by_row else vec(0.1, 0.5) if case.get("gate") else None
        out = q.residual_norm_rows(x, r, w, gate=gate, **kw)
        for i in range(0, m, SLICE):
            at = slice(i, i + SLICE)
            one = q.residual_norm_rows(x[at], r[at], w, gate=gate[at] if by_row else gate, **kw)
            assert torch.equal(one.residual, out.residual[at]) and torch.equal(one.y, out.y[at]), (case, i)
            assert yt != "i8" or torch.equal(one.y_scale, out.y_scale[at]), (case, i)
        # in place, the next rows' residual being read while these are written
        stream = r.clone()
        again = q.residual_norm_rows(x, stream, w, gate=gate, residual_out=stream, **kw)
        assert torch.equal(stream, out.residual) and torch.equal(again.y, out.y), case
        narrow = _narrow(yt, x, r, gate if by_row else None)
        gh = _host(gate[some] if by_row else gate)
        value, bound = ops_ref.residual(_host(x[some]), _host(r[some]), _host(kw["post_weight"]), _host(kw["post_bias"]), gh,
                                        alpha, 1e-6, layer, narrow)
        ops_ref.assert_rounded(_host(out.residual[some]), value, bound, rt, (case, "residual"))
        part = q.NormOut(out.y[some], None if out.y_scale is None else out.y_scale[some], None)
        _check_y(q, out.residual[some], w, kw["bias"], 1e-6, layer, part, yt, (case, "y"), narrow)


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "i8"), ("fp32", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("n,m", [(96, 20011), (800, 9001), (4096, 5003), (14336, 1301)])
def test_plain_norms_over_many_rows(q, n, m, xt, yt):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(int(synth.rng("normturnsplain", str(n), xt, yt).integers(1 << 31)))
    x = _random(g, m, n, xt)
    x[m // 2] = 0                                              # (a row of its own way among the others)
    w = 1 + 0.2 * torch.randn(n, generator=g, device="cuda")
    b = 0.1 * torch.randn(n, generator=g, device="cuda")
    yd = torch.int8 if yt == "i8" else i8_ref.torch_type(yt)
    some = torch.tensor([0, 1, 5, m // 2, m // 2 + 1, m - 2, m - 1], device="cuda")
    for layer in (False, True):
        out = q.norm_rows(x, w, bias=b, layer=layer, dtype=yd)
        for i in range(0, m, SLICE):
            at = slice(i, i + SLICE)
            one = q.norm_rows(x[at], w, bias=b, layer=layer, dtype=yd)
            assert torch.equal(one.y, out.y[at]), (layer, i)
            assert yt != "i8" or torch.equal(one.y_scale, out.y_scale[at]), (layer, i)
        part = q.NormOut(out.y[some], None if out.y_scale is None else out.y_scale[some], None)
        _check_y(q, x[some], w, b, 1e-5, layer, part, yt, layer)


def test_far_rows_among_others(q):
    """Rows at bfloat16's ends before and after ordinary ones of the same
    workgroup."""
    import torch
    for n, m in ((96, 20011), (4096, 5003), (14336, 1301)):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        x = torch.randn((m, n), generator=g, device="cuda")
        x[::3] *= 2e-40
        x[1::7] *= 5e37
        x = x.clamp(-3.38e38, 3.38e38).bfloat16()
        w = 1 + 0.2 * torch.randn(n, generator=g, device="cuda")
        for layer in (False, True):
            out = q.norm_rows(x, w, eps=0.0, layer=layer, dtype=torch.bfloat16)
            assert bool(torch.isfinite(out.y).all())
            for i in range(0, m, SLICE):
                assert torch.equal(q.norm_rows(x[i:i + SLICE], w, eps=0.0, layer=layer, dtype=torch.bfloat16).y,
                                   out.y[i:i + SLICE]), (n, layer, i)
