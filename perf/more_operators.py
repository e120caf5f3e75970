"""The cases on which the operators around the products of a token step are
measured: embedding rows, residual and norm rows, products with an activation
and a residual in their epilogue, and sampling.  `run` with `own` true makes
the library's calls, with `own` false it computes the same in plain torch
operations."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# The cases.  op: "embed" (rows of a table in one of the library's formats,
# scaled), "norm" (residual stream update and the next norm, to floats or to
# int8 codes with a scale per row), "act" (product of 8-bit codes with bias,
# activation and residual), "sample" (a token per row of logits from a given
# random number, after temperature, top-k, top-p and min-p).

def _em(name, m, n, k, table, y_type, scale):
    return {"name": name, "op": "embed", "m": m, "n": n, "k": k, "table": table,
            "y_type": y_type, "scale": scale}


def _no(name, m, n, x_type, y_type, layer=False, block=True, post=False, gate="none",
        residual_scale=1.0):
    """block: x is a block's output, added to a residual stream of its type;
    gate: "none", "channel" (fp32 [n]) or "row" (of x's type, [m][n])."""
    return {"name": name, "op": "norm", "m": m, "n": n, "x_type": x_type, "y_type": y_type,
            "layer": layer, "block": block, "post": post, "gate": gate,
            "residual_scale": residual_scale}


def _ac(name, m, k, n, x_type, y_type, act, bias, residual, codes=False):
    return {"name": name, "op": "act", "m": m, "k": k, "n": n, "x_type": x_type, "y_type": y_type,
            "act": act, "bias": bias, "residual": residual, "codes": codes}


def _sa(name, m, vocab, x_type, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, banned=False,
        mixed=False):
    """mixed: every row has settings of its own."""
    return {"name": name, "op": "sample", "m": m, "vocab": vocab, "x_type": x_type,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "banned": banned, "mixed": mixed}


def listed():
    return [
        # the embedding row of one decoded token, tied 262144-row vocabulary: latency
        _em("embed_1x2048_q8_0", 1, 262144, 2048, "q8_0", "fp32", 45.254834),
        # a packed prompt of 16384 tokens from an int8 table
        _em("embed_16384x4096_i8", 16384, 32000, 4096, "i8", "bf16", 1.0),
        # the norm before a block of the Llama-110M-shaped step, one token: latency
        _no("norm_1x768", 1, 768, "fp32", "fp32", block=False),
        # a ragged batch: norm after a block, its gate, the residual, the next block's codes
        _no("norm_257x4096_gated", 257, 4096, "bf16", "i8", post=True, gate="row"),
        # a packed prompt: residual and the next norm, with mean and bias
        _no("norm_16384x4096", 16384, 4096, "bf16", "bf16", layer=True, gate="channel"),
        # an FFN's first product for one token: latency
        _ac("act_1x768x2048", 1, 768, 2048, "fp32", "fp32", "gelu_tanh", True, False),
        # the down projection of 13 sequences decoded together, into the residual stream
        _ac("act_13x14336x4096", 13, 14336, 4096, "bf16", "bf16", "none", True, True),
        # the down projection of a 512-token prompt
        _ac("act_512x14336x4096", 512, 14336, 4096, "bf16", "bf16", "none", False, True, codes=True),
        # one decoded token: latency
        _sa("sample_1x32000", 1, 32000, "fp32", 0.8, 40, 0.95),
        # a decode batch over the largest vocabulary, some tokens banned by a grammar
        _sa("sample_8x262144", 8, 262144, "fp32", 0.7, 0, 0.9, banned=True),
        # requests with settings of their own, decoded together, odd vocabulary
        _sa("sample_333x50257_mixed", 333, 50257, "bf16", mixed=True),
        # a large batch of rollouts over the largest vocabulary
        _sa("sample_512x262144", 512, 262144, "bf16", 1.0, 0, 0.95),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "act", "sample", "sample"])
    t = ["fp32", "fp16", "bf16"]
    if op == "embed":
        k = 32 * _logint(rng, 8, 256)
        m = _logint(rng, 1, (1 << 26) // k)
        n = _logint(rng, 1000, min(262144, (1 << 29) // k))
        c = _em("", m, n, k, rng.choice(t + ["i8", "q8_0", "r8"]), rng.choice(t),
                rng.choice([1.0, 16.0, math.sqrt(k)]))
    elif op == "norm":
        y = rng.choice(t + ["i8"])
        n = 32 * _logint(rng, 8, 448) if y == "i8" else _logint(rng, 100, 14336)
        m = _logint(rng, 1, (1 << 25) // n)
        block = rng.random() < 0.8
        c = _no("", m, n, rng.choice(t), y, rng.random() < 0.4, block,
                block and rng.random() < 0.5,
                rng.choice(["none", "channel", "row"]) if block else "none",
                rng.choice([1.0, 0.5]) if block else 1.0)
    elif op == "act":
        k = 32 * _logint(rng, 8, 448)
        n = _logint(rng, 64, 16384)
        m = _logint(rng, 1, max(1, min(2048, 512 * 14336 * 4096 // (n * k))))
        c = _ac("", m, k, n, rng.choice(t), rng.choice(t),
                rng.choice(["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]),
                rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.4)
    else:
        x = rng.choice(t)
        vocab = _logint(rng, 1000, 262144)
        m = _logint(rng, 1, max(1, min(2048, (1 << 28) // (SIZES[x] * vocab))))
        c = _sa("", m, vocab, x, rng.choice([0.0, 0.6, 1.0, 1.3]),
                rng.choice([0, 0, 1, 20, 50, 500]), rng.choice([1.0, 0.8, 0.95]),
                rng.choice([0.0, 0.0, 0.02]), rng.random() < 0.3, rng.random() < 0.4)
    del c["name"]
    return c


def _row_bytes(table, k):
    """Bytes of one table row."""
    if table == "i8":
        return k + 4
    return 34 * (k // 32) if table in ("q8_0", "r8") else k * SIZES[table]


def work(case):
    m = case["m"]
    if case["op"] == "embed":
        k = case["k"]
        # a row that several tokens name is read once
        rows = case["n"] * (1.0 - (1.0 - 1.0 / case["n"]) ** m)
        return {"bytes": rows * _row_bytes(case["table"], k) + 4 * m + m * k * SIZES[case["y_type"]],
                "flops": 2 * m * k}
    if case["op"] == "norm":
        n, xs = case["n"], SIZES[case["x_type"]]
        rows = 1 + 2 * case["block"] + (case["gate"] == "row")     # x, residual in and out, gate
        y = m * n + 4 * m if case["y_type"] == "i8" else m * n * SIZES[case["y_type"]]
        vectors = 1 + case["layer"] + case["post"] + (case["gate"] == "channel")
        # squares and products of each norm, gate and residual
        ops = 4 + 4 * case["post"] + 3 * case["block"] + 2 * case["layer"]
        return {"bytes": rows * m * n * xs + y + 4 * n * vectors, "flops": ops * m * n}
    if case["op"] == "act":
        k, n, ys = case["k"], case["n"], SIZES[case["y_type"]]
        x = m * k + 4 * m if case["codes"] else m * k * SIZES[case["x_type"]]
        return {"bytes": x + n * k + 4 * n * (1 + case["bias"]) + m * n * ys * (1 + case["residual"]),
                "flops": 2 * m * n * k}
    v = case["vocab"]
    # per logit: scale, subtract, exp, sum, compare
    return {"bytes": m * v * SIZES[case["x_type"]] + 4 * m * 8, "flops": 5 * m * v}


# ---------------------------------------------------------------------------
# Inputs, on the GPU, from the seed alone.

def _quantize(x):
    """Codes and scales of each row of fp32 values: s = max|x| / 127 in fp32,
    code = sign(x) * floor(|x| / s + 1/2), the quotient in 64 bits."""
    x = x.float()
    a = x.abs().amax(1)
    s = a / torch.full_like(a, 127.0)
    d = torch.where(s > 0, s, torch.ones_like(s)).double()
    c = torch.floor(x.abs().double() / d[:, None] + 0.5).clamp_(max=127.0)
    c = torch.where(s[:, None] > 0, c, torch.zeros_like(c)) * torch.sign(x)
    return c.to(torch.int8), s


def _weights(n, k, g):
    """[n][k] codes and [n] scales of N(0, 0.02) rows, a slice at a time."""
    w = torch.empty((n, k), dtype=torch.int8, device="cuda")
    s = torch.empty(n, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // k)
    for i in range(0, n, step):
        r = torch.randn((min(step, n - i), k), generator=g, device="cuda") * 0.02
        w[i:i + step], s[i:i + step] = _quantize(r)
    return w, s


def _table(case, g):
    """A table of n rows of k values of size about 0.02, and the row scales of
    an int8 one."""
    n, k, kind = case["n"], case["k"], case["table"]
    if kind in DTYPES:
        return (torch.randn((n, k), generator=g, device="cuda") * 0.02).to(DTYPES[kind]), None
    nb = k // 32

    def scales(*shape):
        return torch.rand(shape, generator=g, device="cuda") * 3e-4 + 3e-4

    def codes(*shape):
        return torch.randint(1, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

    if kind == "i8":
        return codes(n, k).view(torch.int8), scales(n)
    if kind == "q8_0":
        t = codes(n, nb, 34)
        t[:, :, :2] = scales(n, nb, 1).half().view(torch.uint8)
        return t.view(n, nb * 34), None
    groups = (n + 7) // 8                   # r8: eight rows together, scales then codes
    t = codes(groups, nb * 272)
    t[:, :16 * nb] = scales(groups, 8 * nb).half().view(torch.uint8)
    return t.view(-1), None


def _hidden(m, k, g):
    x = torch.randn((m, k), generator=g, device="cuda")
    # a few channels of hidden states are far larger than the rest
    x[:, torch.randint(k, (max(1, k // 512),), generator=g, device="cuda")] *= 12.0
    return x


def _sample_inputs(case, g):
    m, v = case["m"], case["vocab"]

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    x = torch.randn((m, v), generator=g, device="cuda") * 1.5
    # likely continuations by rank; most rows are sure, a few rows' tails weigh as much
    likely = torch.randint(v, (m, 64), generator=g, device="cuda")
    rank = torch.arange(1, 65, device="cuda").float()
    x.scatter_(1, likely, (0.85 + 0.35 * rand(m, 1)) * 18.0 - 1.2 * torch.log(rank) + 0.5 * rand(m, 64))
    if case["banned"]:
        x.masked_fill_(rand(m, v) < 0.1, -math.inf)

    def each(value, dtype=torch.float32):
        return torch.full((m,), value, dtype=dtype, device="cuda")

    d = {"logits": x.to(DTYPES[case["x_type"]]), "u": rand(m),
         "temperature": each(case["temperature"]), "top_k": each(case["top_k"], torch.int32),
         "top_p": each(case["top_p"]), "min_p": each(case["min_p"])}
    if case["mixed"]:
        def some(key, values):
            at = torch.randint(len(values), (m,), generator=g, device="cuda")
            d[key] = torch.tensor(values, dtype=d[key].dtype, device="cuda")[at]
        some("temperature", [0.0, 0.6, 0.8, 1.0, 1.0, 1.3])
        some("top_k", [0, 0, 0, 1, 20, 50, 200])
        some("top_p", [1.0, 0.95, 0.9, 0.5])
        some("min_p", [0.0, 0.0, 0.05, 0.1])
    return d


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m = case["m"]
    if case["op"] == "sample":
        return _sample_inputs(case, g)
    if case["op"] == "embed":
        table, s = _table(case, g)
        tok = torch.randint(case["n"], (m,), generator=g, device="cuda")
        return {"table": table, "table_scale": s, "tokens": tok.to(torch.int32)}
    if case["op"] == "norm":
        n, t = case["n"], DTYPES[case["x_type"]]

        def vector(size, middle):
            return middle + size * torch.randn(n, generator=g, device="cuda")

        d = {"x": _hidden(m, n, g).to(t), "weight": vector(0.2, 1.0), "bias": None, "residual": None,
             "post_weight": None, "gate": None}
        if case["layer"]:
            d["bias"] = vector(0.1, 0.0)
        if case["block"]:
            d["residual"] = (3.0 * _hidden(m, n, g)).to(t)
        if case["post"]:
            d["post_weight"] = vector(0.2, 1.0)
        if case["gate"] == "channel":
            d["gate"] = vector(0.1, 0.5)
        elif case["gate"] == "row":
            d["gate"] = torch.rand((m, n), generator=g, device="cuda").to(t)
        return d
    k, n = case["k"], case["n"]
    w, ws = _weights(n, k, g)
    d = {"x": _hidden(m, k, g).to(DTYPES[case["x_type"]]), "x_scale": None, "w": w, "w_scale": ws,
         "bias": None, "residual": None}
    if case["codes"]:
        d["x"], d["x_scale"] = _quantize(d["x"])
    if case["bias"]:
        d["bias"] = torch.randn(n, generator=g, device="cuda") * 0.5
    if case["residual"]:
        d["residual"] = (3.0 * _hidden(m, n, g)).to(DTYPES[case["y_type"]])
    return d


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import moe_expert_ffn_q8_amd as q
        st["q"] = q
        m = case["m"]
        if case["op"] == "sample":
            st["ws"] = q.sample_workspace(m, case["vocab"], "cuda")
            st["out"] = q.sample_outputs(m, "cuda")
        elif case["op"] == "embed":
            st["y"] = torch.empty((m, case["k"]), dtype=DTYPES[case["y_type"]], device="cuda")
        elif case["op"] == "norm":
            codes = case["y_type"] == "i8"
            st["y"] = torch.empty((m, case["n"]), device="cuda",
                                  dtype=torch.int8 if codes else DTYPES[case["y_type"]])
            st["y_scale"] = torch.empty(m, device="cuda") if codes else None
            st["residual_out"] = torch.empty_like(st["x"]) if case["block"] else None
        else:
            st["y"] = torch.empty((m, case["n"]), dtype=DTYPES[case["y_type"]], device="cuda")
            st["ws"] = q.i8_workspace(m, case["k"], "cuda")
    return st


# ---------------------------------------------------------------------------
# One pass.

EPS = 1e-5


def _plain_embed(st):
    case, tok = st["case"], st["tokens"].long()
    m, k, nb, kind = case["m"], case["k"], case["k"] // 32, case["table"]
    if kind in DTYPES:
        y = st["table"][tok].float()
    elif kind == "i8":
        y = st["table"][tok].float() * st["table_scale"][tok][:, None]
    elif kind == "q8_0":
        r = st["table"][tok].view(m, nb, 34)
        d = r[:, :, :2].contiguous().view(torch.float16)
        y = (r[:, :, 2:].contiguous().view(torch.int8).float() * d.float()).view(m, k)
    else:
        r = st["table"].view(-1, nb * 272)[tok // 8]
        row, at = torch.arange(m, device=tok.device), tok % 8
        d = r[:, :16 * nb].contiguous().view(torch.float16).view(m, nb, 8)[row, :, at]
        c = r[:, 16 * nb:].contiguous().view(torch.int8).view(m, nb, 8, 32)[row, :, at]
        y = (c.float() * d.float()[:, :, None]).view(m, k)
    return (y * case["scale"]).to(DTYPES[case["y_type"]])


def _normed(x, weight, bias, layer):
    """In 64 bits: a code of the row rule turns at a border."""
    if layer:
        x = x - x.mean(1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * weight.double()
    return y if bias is None else y + bias.double()


def _plain_norm(st):
    case = st["case"]
    t = DTYPES[case["x_type"]]
    x, out = st["x"].double(), {}
    if case["block"]:
        if case["post"]:
            x = _normed(x, st["post_weight"], None, case["layer"])
        if st["gate"] is not None:
            x = x * st["gate"].double()
        out["residual"] = (x + case["residual_scale"] * st["residual"].double()).to(t)
        x = out["residual"].double()                   # the next norm reads the stream as stored
    y = _normed(x, st["weight"], st["bias"], case["layer"])
    if case["y_type"] == "i8":
        codes, s = _quantize(y)
        out["y"] = codes * s[:, None]
    else:
        out["y"] = y.to(DTYPES[case["y_type"]])
    return out


def _activation(v, act):
    if act == "relu":
        return torch.clamp(v, min=0.0)
    if act == "relu2":
        return torch.clamp(v, min=0.0) ** 2
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v / (1.0 + torch.exp(-v)) if act == "silu" else v


def _plain_act(st):
    case = st["case"]
    c, s = (st["x"], st["x_scale"]) if case["codes"] else _quantize(st["x"])
    # sums of code products pass 2^24: in 64 bits
    y = (c.double() @ st["w"].double().t()).float() * s[:, None] * st["w_scale"][None, :]
    if st["bias"] is not None:
        y = y + st["bias"]
    y = _activation(y, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DTYPES[case["y_type"]])


def _plain_sample(st):
    """In 64 bits: sums over a vocabulary meet the borders of top-p and of the
    random number."""
    x, at = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)
    v = x.shape[1]
    temp = st["temperature"].double()
    greedy = temp <= 0
    temp = torch.where(greedy, torch.ones_like(temp), temp)[:, None]
    z = (x.double() - x[:, :1].double()) / temp
    w = torch.exp(z)
    c = torch.cumsum(w, 1)
    k = st["top_k"].long()
    kept = torch.minimum(torch.where(k > 0, k, torch.full_like(k, v)), (x > -math.inf).sum(1))
    mass = c.gather(1, kept[:, None] - 1)
    p = st["top_p"].double()[:, None]
    nucleus = (c < p * mass).sum(1) + 1
    kept = torch.where(p[:, 0] < 1, torch.minimum(kept, nucleus), kept)
    kept = torch.minimum(kept, (w >= st["min_p"].double()[:, None]).sum(1))
    kept = torch.where(greedy, torch.ones_like(kept), kept)
    mass = c.gather(1, kept[:, None] - 1)
    pos = torch.minimum((c <= st["u"].double()[:, None] * mass).sum(1), kept - 1)[:, None]
    return {"ids": at.gather(1, pos)[:, 0].to(torch.int32), "kept": kept.to(torch.int32),
            "logprob": (z.gather(1, pos) - torch.log(mass))[:, 0].float()}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        q = state["q"]
        if op == "embed":
            if case["table"] in ("q8_0", "r8"):
                return q.q8_0_embed_rows(state["table"], state["tokens"], case["n"], case["k"],
                                         scale=case["scale"], r8=case["table"] == "r8", y=state["y"])
            return q.embed_rows(state["table"], state["tokens"], scale=case["scale"],
                                table_scale=state["table_scale"], y=state["y"])
        if op == "norm":
            if case["block"]:
                o = q.residual_norm_rows(state["x"], state["residual"], state["weight"],
                                         bias=state["bias"], post_weight=state["post_weight"],
                                         gate=state["gate"], residual_scale=case["residual_scale"],
                                         eps=EPS, layer=case["layer"],
                                         residual_out=state["residual_out"], y=state["y"],
                                         y_scale=state["y_scale"])
            else:
                o = q.norm_rows(state["x"], state["weight"], bias=state["bias"], eps=EPS,
                                layer=case["layer"], y=state["y"], y_scale=state["y_scale"])
            y = o.y * o.y_scale[:, None] if case["y_type"] == "i8" else o.y
            return {"residual": o.residual, "y": y} if case["block"] else {"y": y}
        if op == "act":
            return q.i8_matmul_act(state["x"], state["w"], state["w_scale"],
                                   x_scale=state["x_scale"], bias=state["bias"], act=case["act"],
                                   residual=state["residual"], y=state["y"], ws=state["ws"])
        o = q.sample_rows(state["logits"], state["u"], temperature=state["temperature"],
                          top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"],
                          ws=state["ws"], out=state["out"])
        return {"ids": o.ids, "kept": o.kept, "logprob": o.logprob}
    if op == "embed":
        return _plain_embed(state)
    if op == "norm":
        return _plain_norm(state)
    if op == "act":
        return _plain_act(state)
    return _plain_sample(state)


# ---------------------------------------------------------------------------
# The same outputs from the definition, in 64 bits.

def _exact_embed(case, d):
    k, nb, kind = case["k"], case["k"] // 32, case["table"]
    rows = []
    for i in range(0, case["m"], 4096):
        tok = d["tokens"][i:i + 4096].long()
        if kind in ("q8_0", "r8"):
            # byte addresses of each block's scale and codes
            b = torch.arange(nb, device="cuda")[None, :]
            t = tok[:, None]
            if kind == "q8_0":
                s_at = (t * nb + b) * 34
                c_at = s_at + 2
            else:
                base = t // 8 * (272 * nb)
                s_at = base + 2 * (8 * b + t % 8)
                c_at = base + 16 * nb + 32 * (8 * b + t % 8)
            flat = d["table"].reshape(-1)
            s = torch.stack((flat[s_at], flat[s_at + 1]), 2).view(torch.float16)[:, :, 0].double()
            c = flat[c_at[:, :, None] + torch.arange(32, device="cuda")].view(torch.int8).double()
            y = (c * s[:, :, None]).reshape(-1, k)
        else:
            y = torch.index_select(d["table"], 0, tok).double()
            if kind == "i8":
                y *= torch.index_select(d["table_scale"], 0, tok).double()[:, None]
        rows.append(y * case["scale"])
    return torch.cat(rows)


def _exact_codes(y):
    """The values that the codes of rows y stand for."""
    y = y.float().double()
    s = (y.abs().max(dim=1).values / torch.tensor(127.0, dtype=torch.float64,
                                                  device=y.device)).float().double()[:, None]
    v = y / torch.where(s == 0, torch.ones_like(s), s)
    return torch.where(v < 0, torch.ceil(v - 0.5), torch.floor(v + 0.5)).clamp(-127, 127) * s


def _exact_norm(case, d):
    def norm(x, w, b):
        mean = x.sum(1, keepdim=True) / case["n"] if case["layer"] else 0.0
        var = torch.linalg.vector_norm(x - mean, dim=1, keepdim=True) ** 2 / case["n"]
        y = (x - mean) * torch.rsqrt(var + EPS) * w.double()
        return y + b.double() if b is not None else y

    parts = []
    for i in range(0, case["m"], 1024):
        x = d["x"][i:i + 1024].double()
        r = {}
        if case["block"]:
            if case["post"]:
                x = norm(x, d["post_weight"], None)
            if case["gate"] == "channel":
                x = d["gate"].double() * x
            elif case["gate"] == "row":
                x = d["gate"][i:i + 1024].double() * x
            r["residual"] = d["residual"][i:i + 1024].double() * case["residual_scale"] + x
            x = r["residual"].to(DTYPES[case["x_type"]]).double()
        y = norm(x, d["weight"], d["bias"])
        r["y"] = _exact_codes(y) if case["y_type"] == "i8" else y
        parts.append(r)
    return {name: torch.cat([r[name] for r in parts]) for name in parts[0]}


def _exact_act(case, d):
    if case["codes"]:
        c, s = d["x"].double(), d["x_scale"].double()
    else:
        x = d["x"].double()
        s = (x.abs().max(dim=1).values / torch.tensor(127.0, dtype=torch.float64,
                                                      device=x.device)).float().double()
        v = x / torch.where(s == 0, torch.ones_like(s), s)[:, None]
        c = torch.where(v < 0, torch.ceil(v - 0.5), torch.floor(v + 0.5)).clamp(-127, 127)
    y = []
    step = max(1, (1 << 27) // case["k"])
    for j in range(0, d["w"].shape[0], step):      # the weights' rows a slice at a time
        part = torch.mm(c, d["w"][j:j + step].double().t().contiguous())
        y.append(part * s[:, None] * d["w_scale"][j:j + step].double())
    y = torch.cat(y, 1)
    if d["bias"] is not None:
        y = y + d["bias"].double()
    if case["act"] in ("relu", "relu2"):
        y = torch.where(y > 0, y, torch.zeros_like(y))
        y = y * y if case["act"] == "relu2" else y
    elif case["act"] == "gelu":
        y = 0.5 * y * torch.erfc(-y / math.sqrt(2.0))
    elif case["act"] == "gelu_tanh":
        y = y * torch.sigmoid(math.sqrt(8.0 / math.pi) * y * (1.0 + 0.044715 * y * y))
    elif case["act"] == "silu":
        y = y * torch.sigmoid(y)
    if d["residual"] is not None:
        y = y + d["residual"].double()
    return y


def _exact_sample(case, d):
    """Log probabilities alone: the tokens are whole numbers, and the rows are
    the plain form's.  The token and the size of the set come from a table of
    the row's distinct logits, how often each occurs and their mass."""
    lp = torch.empty(case["m"], dtype=torch.float64, device="cuda")
    x = d["logits"].double()
    host = {key: d[key].double().cpu().tolist() for key in ("u", "temperature", "top_k", "top_p", "min_p")}
    for i in range(case["m"]):
        t = host["temperature"][i]
        if t <= 0:
            lp[i] = 0.0
            continue
        row = x[i]
        val, times = torch.unique(row[row > -math.inf], return_counts=True)
        val, times = val.flip(0), times.flip(0)
        z = (val - val[0]) / t
        one = torch.exp(z)
        count, mass = times.cumsum(0), (one * times).cumsum(0)

        def top(n):                                # the mass of the n first tokens
            j = int(torch.searchsorted(count, n))
            before = (int(count[j - 1]), float(mass[j - 1])) if j else (0, 0.0)
            return before[1] + (n - before[0]) * float(one[j])

        def reach(target, strict):                 # how many tokens reach (pass) a mass
            j = int(torch.searchsorted(mass, target, right=strict))
            if j >= len(mass):
                return int(count[-1])
            before = (int(count[j - 1]), float(mass[j - 1])) if j else (0, 0.0)
            q = (target - before[1]) / float(one[j])
            return before[0] + min(int(times[j]), max(1, math.floor(q) + 1 if strict else math.ceil(q)))

        n = int(count[-1])
        if host["top_k"][i] > 0:
            n = min(n, int(host["top_k"][i]))
        least = int(times[one >= host["min_p"][i]].sum())
        if host["top_p"][i] < 1:
            n = min(n, reach(host["top_p"][i] * top(n), False))
        n = max(1, min(n, least))
        total = top(n)
        pos = min(n, reach(host["u"][i] * total, True))
        lp[i] = z[int(torch.searchsorted(count, pos))] - math.log(total)
    return {"ids": None, "kept": None, "logprob": lp}


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "embed":
        return _exact_embed(case, d)
    if case["op"] == "norm":
        return _exact_norm(case, d)
    if case["op"] == "act":
        return _exact_act(case, d)
    return _exact_sample(case, d) if case["m"] <= 700 else None
