"""A token's way round, as a user runs it: embedding rows, the norm before a
block with codes for its products, the gated FFN, the down product into the
residual stream, the next norm, logits, and the next token -- eagerly, on
another stream and in a captured graph that is replayed on new tokens, and
other calls of the operators in graphs that share a workspace."""
import numpy as np
import pytest

import i8_ref
import ops_ref
import synth
from gpu_cases import to_gpu

pytestmark = pytest.mark.gpu

K, N_FF, VOCAB, LAYERS = 256, 352, 5000, 2


@pytest.fixture(scope="module")
def q():
    import moe_expert_ffn_q8_amd as q
    return q


class Model:
    def __init__(self, q, m, t, tag):
        import torch
        rng = synth.rng("loop", tag)
        self.q, self.m, self.t = q, m, t
        tt = i8_ref.torch_type(t)

        def weights(n, k, sigma):
            return q.i8_quantize_rows(to_gpu((rng.normal(size=(n, k)) * sigma).astype(np.float32)))

        def vec(n, middle=1.0):
            return to_gpu((middle + 0.2 * rng.normal(size=n)).astype(np.float32))
        self.head = weights(VOCAB, K, 0.3)             # tied: the embedding table too
        self.layers = [dict(up=weights(2 * N_FF, K, 0.1), down=weights(K, N_FF, 0.1), bias=vec(K, 0.0),
                            norm=vec(K), post=vec(K), gate=vec(K, 0.5)) for _ in range(LAYERS)]
        self.last = vec(K)
        dev = "cuda"
        self.tokens = torch.zeros(m, dtype=torch.int32, device=dev)
        self.u = torch.zeros(m, device=dev)
        self.x, self.r = (torch.empty((m, K), dtype=tt, device=dev) for _ in range(2))
        self.codes = torch.empty((m, K), dtype=torch.int8, device=dev)
        self.scale = torch.empty(m, device=dev)
        self.h = torch.empty((m, N_FF), dtype=tt, device=dev)
        self.y = torch.empty((m, K), dtype=tt, device=dev)
        self.logits = torch.empty((m, VOCAB), device=dev)
        self.ws = q.i8_workspace(m, N_FF, dev)
        self.sws = q.sample_workspace(m, VOCAB, dev)
        self.out = q.sample_outputs(m, dev)
        self.set = dict(temperature=torch.full((m,), 0.9, device=dev), top_p=torch.full((m,), 0.95, device=dev),
                        top_k=torch.full((m,), 60, dtype=torch.int32, device=dev))

    def load(self, seed):
        rng = synth.rng("loop-in", str(seed))
        self.tokens.copy_(to_gpu(rng.integers(0, VOCAB, self.m).astype(np.int32)))
        self.u.copy_(to_gpu(rng.random(self.m).astype(np.float32)))

    def step(self):
        q = self.q
        q.embed_rows(self.head[0], self.tokens, scale=16.0, table_scale=self.head[1], y=self.x)
        r = self.x
        q.norm_rows(r, self.layers[0]["norm"], y=self.codes, y_scale=self.scale)
        for i, l in enumerate(self.layers):
            q.i8_up_gate_swiglu(self.codes, *l["up"], x_scale=self.scale, h=self.h)
            after = self.layers[i + 1]["norm"] if i + 1 < LAYERS else self.last
            if i == 0:                                 # the down product into the stream, in place
                q.i8_matmul_act(self.h, *l["down"], bias=l["bias"], residual=r, y=r, ws=self.ws)
                q.norm_rows(r, after, y=self.codes, y_scale=self.scale)
            else:                                      # a norm after the block, gated
                q.i8_matmul_act(self.h, *l["down"], bias=l["bias"], act="gelu_tanh", y=self.y, ws=self.ws)
                q.residual_norm_rows(self.y, r, after, post_weight=l["post"], gate=l["gate"], residual_scale=0.8,
                                     residual_out=r, y=self.codes, y_scale=self.scale)
        q.i8_matmul(self.codes, *self.head, x_scale=self.scale, y=self.logits)
        q.sample_rows(self.logits, self.u, ws=self.sws, out=self.out, **self.set)
        self.tokens.copy_(self.out.ids)

    def state(self):
        return [t.clone() for t in (self.x, self.codes, self.scale, self.h, self.y, self.logits, *self.out, self.tokens)]


@pytest.mark.parametrize("t", i8_ref.TYPES)
@pytest.mark.parametrize("m", [1, 14, 150])
def test_last_stages(q, m, t):
    """Logits and tokens against the references on the stages' own inputs."""
    md = Model(q, m, t, "stages")
    md.load(1)
    md.step()
    n = lambda a: a.cpu().numpy()
    y, _ = ops_ref.norm(md.x.double().cpu().numpy(), n(md.last).astype(np.float64), None, 1e-5, False)
    codes, scale = i8_ref.quantize(y.astype(np.float32))
    assert np.array_equal(n(md.codes), codes) and np.array_equal(n(md.scale), scale)
    i8_ref.assert_close(n(md.logits).astype(np.float64), *i8_ref.product(codes, scale, n(md.head[0]), n(md.head[1])),
                        "fp32", "logits")
    got = np.stack([o.double().cpu().numpy() for o in md.out], 1)
    for i in range(m):
        ref = ops_ref.sample_row(n(md.logits)[i].astype(np.float64), n(md.u)[i], np.float32(0.9), 60, np.float32(0.95), 0.0)
        ops_ref.assert_sample(got[i], ref, f"row {i}")


@pytest.mark.parametrize("m", [1, 14, 150])
def test_other_stream_and_graph(q, m):
    import torch
    md = Model(q, m, "bf16", "graph")
    want = {}
    for seed in (1, 2, 3):
        md.load(seed)
        for _ in range(3):                             # three tokens, one after another
            md.step()
        want[seed] = md.state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        md.load(2)
        for _ in range(3):
            md.step()
        got = md.state()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        md.step()
    for seed in (3, 1, 2, 2):
        md.ws.fill_(255)
        md.sws.fill_(255)
        md.load(seed)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(md.state(), want[seed])), seed
        md.load(seed)
        for _ in range(3):                             # eager work between the replays
            md.step()
        assert all(torch.equal(a, b) for a, b in zip(md.state(), want[seed])), seed


def test_two_graphs_share_a_workspace(q):
    """Sampling of two sizes, one with rows that are read again, captured with
    one workspace and replayed in turn."""
    import torch
    rng = synth.rng("loopshare")
    sizes = [(40, 30000, 0.05), (6, 120000, 1.5)]
    ws = max((q.sample_workspace(m, v, "cuda") for m, v, _ in sizes), key=lambda w: w.numel())
    runs = []
    for m, v, flat in sizes:
        x = to_gpu((rng.normal(size=(m, v)) * flat).astype(np.float32)).bfloat16()
        u = to_gpu(rng.random(m).astype(np.float32))
        p = torch.full((m,), 0.97, device="cuda")
        out = q.sample_outputs(m, "cuda")
        call = lambda x=x, u=u, p=p, out=out: q.sample_rows(x, u, top_p=p, ws=ws, out=out)
        call()
        want = [t.clone() for t in out]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, out, want, call))              # (the call keeps its inputs)
    for i in (0, 1, 1, 0, 0, 1):
        g, out, want, _ = runs[i]
        for t in out:
            t.fill_(-9)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
