"""8-bit products with an activation and a residual: streams in place and rows
that start anywhere on every kernel that tiles both operands, the one of halves
of k among them."""
import pytest

import i8_ref
from gpu_cases import to_gpu
from test_gpu_i8_act import Case, _check

pytestmark = pytest.mark.gpu

K_HALVES = 6


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


# halves of k (whole and ragged tiles, the second half ending inside a step), tiles of 128 x 128,
# of 256 x 256 whole and in part
SIZES = [(300, 1024, 4100), (97, 1312, 8200), (70, 4128, 515), (512, 2048, 4096), (257, 512, 4100), (2050, 64, 8200),
         (2048, 128, 8192), (4500, 96, 5000)]


def _form(q, m, k, n):
    return q.raw.q8v_i8_act_form(n, k, m)


def test_sizes_reach_the_kernels(q):
    forms = [_form(q, *s) for s in SIZES]
    assert forms[0] == forms[1] == forms[3] == K_HALVES and 2 in forms and {3, 4} & set(forms), forms


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m,k,n", SIZES)
def test_in_place(q, m, k, n, t):
    """The stream updated in place is the one written elsewhere."""
    import torch
    c = Case(m, k, n, "place")
    cx, sx, cw, sw, b, r = c.gpu(t)
    for act in ("none", "gelu"):
        want = _check(q, c, t, act)
        y = r.clone()
        out = q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act=act, residual=y, y=y)
        assert out is y and torch.equal(y, want)


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (5, 8), (64, 64)])
@pytest.mark.parametrize("m,k,n", SIZES[:2] + SIZES[4:5])
def test_row_starts(q, m, k, n, offset, pad, t):
    """Residual and output rows of different strides; what lies beside a row
    stays, in place too."""
    import torch
    tt = i8_ref.torch_type(t)
    c = Case(m, k, n, "starts")
    rb = torch.full((m * (n + pad + 1) + offset,), 1e4, dtype=tt, device="cuda")
    r = rb[offset:].view(m, n + pad + 1)[:, :n]
    r.copy_(to_gpu(c.res))
    yb = torch.full((m * (n + pad) + offset + 9,), -7.0, dtype=tt, device="cuda")
    y = yb[offset:offset + m * (n + pad)].view(m, n + pad)[:, :n]
    _check(q, c, t, "silu", y=y, r=r)

    def beside(buf, rows, width, value):
        body = buf[offset:offset + rows * width].view(rows, width)
        return bool((body[:, n:] == value).all()) and bool((buf[:offset] == value).all()) and \
            bool((buf[offset + rows * width:] == value).all())
    assert beside(yb, m, n + pad, -7) and beside(rb, m, n + pad + 1, 1e4)
    cx, sx, cw, sw, b, _ = c.gpu(t)
    q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act="silu", residual=r, y=r)
    assert torch.equal(r, y) and beside(rb, m, n + pad + 1, 1e4)


@pytest.mark.parametrize("m,k,n", SIZES[:4])
def test_alone_and_captured(q, m, k, n):
    """Halves of k: a row does not depend on the others or on their number, and
    a graph's replays are the eager call."""
    import torch
    c = Case(m, k, n, "alone")
    cx, sx, cw, sw, b, r = c.gpu("bf16")
    want = q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act="relu2", residual=r)
    for i in (0, m // 2, m - 1):
        one = q.i8_matmul_act(cx[i:i + 1], cw, sw, x_scale=sx[i:i + 1], bias=b, act="relu2", residual=r[i:i + 1])
        assert torch.equal(one[0], want[i])
    y = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.i8_matmul_act(cx, cw, sw, x_scale=sx, bias=b, act="relu2", residual=r, y=y)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
