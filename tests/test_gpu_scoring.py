"""Scoring a prompt with 8-bit weights: the gated FFN, the down product with a
bias, the vocabulary product and the log probabilities, run together as a user
runs them -- eagerly, on another stream and in a captured graph that is
replayed on new inputs."""
import numpy as np
import pytest

import i8_ref
import synth
from gpu_cases import to_gpu

pytestmark = pytest.mark.gpu

K, N_FF, VOCAB, TOP = 256, 352, 2500, 7


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


class Model:
    def __init__(self, q, m, t, tag):
        import torch
        rng = synth.rng("scoring", tag)
        self.q, self.m, self.t = q, m, t
        tt = i8_ref.torch_type(t)
        def weights(n, k, sigma):
            return q.i8_quantize_rows(to_gpu((rng.normal(size=(n, k)) * sigma).astype(np.float32)))
        self.ug, self.ugs = weights(2 * N_FF, K, 0.1)
        self.dn, self.dns = weights(K, N_FF, 0.1)
        self.head, self.heads = weights(VOCAB, K, 0.2)
        self.bias = to_gpu(rng.normal(size=K).astype(np.float32))
        dev = "cuda"
        self.x = torch.zeros((m, K), dtype=tt, device=dev)
        self.tok = torch.zeros((m, 1), dtype=torch.int32, device=dev)
        self.h = torch.empty((m, N_FF), dtype=tt, device=dev)
        self.y = torch.empty((m, K), dtype=tt, device=dev)
        self.logits = torch.empty((m, VOCAB), dtype=torch.float32, device=dev)
        self.ws = q.i8_workspace(m, max(K, N_FF), dev)
        self.lws = q.logprob_workspace(m, VOCAB, TOP, dev)
        self.out = q.logprob_outputs(m, 1, TOP, dev)

    def load(self, seed):
        rng = synth.rng("scoring-in", str(seed), self.t)
        self.x.copy_(to_gpu(rng.normal(size=(self.m, K)).astype(np.float32)))
        self.tok.copy_(to_gpu(rng.integers(0, VOCAB, size=(self.m, 1)).astype(np.int32)))

    def run(self):
        q = self.q
        q.i8_up_gate_swiglu(self.x, self.ug, self.ugs, h=self.h, ws=self.ws)
        q.i8_matmul(self.h, self.dn, self.dns, bias=self.bias, y=self.y, ws=self.ws)
        q.i8_matmul(self.y, self.head, self.heads, y=self.logits, ws=self.ws)
        q.logprob_rows(self.logits, self.tok, n_top=TOP, ws=self.lws, out=self.out)

    def outputs(self):
        return [t.clone() for t in (self.h, self.y, self.logits, *self.out)]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m", [1, 14, 60, 150])
def test_chain(q, m, t):
    """Each stage against the reference on the stage's own input."""
    md = Model(q, m, t, "chain")
    md.load(1)
    md.run()
    n = lambda a: a.cpu().numpy()
    f = lambda a: a.float().cpu().numpy()
    cx, sx = i8_ref.quantize(f(md.x))
    i8_ref.assert_close(md.h.double().cpu().numpy(), *i8_ref.gated(cx, sx, n(md.ug), n(md.ugs)), t, "h")
    cx, sx = i8_ref.quantize(f(md.h))
    i8_ref.assert_close(md.y.double().cpu().numpy(),
                        *i8_ref.product(cx, sx, n(md.dn), n(md.dns), n(md.bias)), t, "y")
    cx, sx = i8_ref.quantize(f(md.y))
    i8_ref.assert_close(md.logits.double().cpu().numpy(),
                        *i8_ref.product(cx, sx, n(md.head), n(md.heads)), "fp32", "logits")
    i8_ref.assert_logprobs(md.out, i8_ref.logprobs(n(md.logits).astype(np.float64), n(md.tok), TOP))


@pytest.mark.parametrize("m", [1, 14, 60, 150])
def test_other_stream_and_graph(q, m):
    import torch
    md = Model(q, m, "bf16", "graph")
    want = {}
    for seed in (1, 2, 3):
        md.load(seed)
        md.run()
        want[seed] = md.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        md.load(2)
        md.run()
        got = md.outputs()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        md.run()
    for seed in (3, 1, 2, 2, 1):
        md.load(seed)
        md.ws.fill_(255)
        md.lws.fill_(255)
        graph.replay()
        got = md.outputs()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[seed])), seed
        md.load(seed)
        md.run()                                   # eager work between the replays
        assert all(torch.equal(a, b) for a, b in zip(md.outputs(), want[seed])), seed


def test_two_graphs_share_a_workspace(q):
    """Two captured calls of different sizes with one workspace, replayed in
    turn on one stream."""
    import torch
    a, b = Model(q, 40, "bf16", "share"), Model(q, 9, "bf16", "share")
    b.ws, b.lws = a.ws, (a.lws if a.lws.numel() >= b.lws.numel() else b.lws)
    a.lws = b.lws if b.lws.numel() > a.lws.numel() else a.lws
    graphs, want = [], []
    for i, md in enumerate((a, b)):
        md.load(10 + i)
        md.run()
        want.append(md.outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            md.run()
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
        assert all(torch.equal(x, y) for x, y in zip((a, b)[i].outputs(), want[i]))


def test_logits_of_the_q8_0_vocabulary_product(q):
    """Log probabilities of the rows that the Q8_0 product writes."""
    rng = synth.rng("scoring-q8")
    w = q.q8_0_quantize_rows(to_gpu((rng.normal(size=(VOCAB, K)) * 0.2).astype(np.float32)))
    x = q.q8_0_quantize_rows(to_gpu(rng.normal(size=(3, K)).astype(np.float32)))
    logits = q.q8_0_matmul(w, x, VOCAB, K, 3)
    tok = np.array([[5], [VOCAB - 1], [0]], np.int32)
    out = q.logprob_rows(logits, to_gpu(tok), n_top=TOP, ws=q.logprob_workspace(3, VOCAB, TOP, "cuda"))
    i8_ref.assert_logprobs(out, i8_ref.logprobs(logits.cpu().numpy().astype(np.float64), tok, TOP))
