"""The cases on which the 8-bit products with token and channel scales and the
log probabilities are measured: `run` with `own` true makes the library's
calls, with `own` false it computes the same in plain torch operations."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# The cases.  op: "matmul" (activations quantized per token, product, optional
# bias), "up_gate" (the same with both projections of a gated FFN and SwiGLU),
# "logprob" (log probabilities, entropy and top alternatives of logit rows).
# codes: the activations are codes and scales already (one quantization shared
# by several products); else they are x_type rows that the call quantizes.

def _mm(name, m, k, n, x_type, y_type, codes=False, bias=False):
    return {"name": name, "op": "matmul", "m": m, "k": k, "n": n, "x_type": x_type,
            "y_type": y_type, "codes": codes, "bias": bias}


def _ug(name, m, k, n_ff, x_type, y_type, codes=False):
    return {"name": name, "op": "up_gate", "m": m, "k": k, "n_ff": n_ff, "x_type": x_type,
            "y_type": y_type, "codes": codes}


def _lp(name, m, vocab, x_type, n_top, given, banned=False):
    return {"name": name, "op": "logprob", "m": m, "vocab": vocab, "x_type": x_type,
            "n_top": n_top, "given": given, "banned": banned}


def listed():
    return [
        # a q/k/v/o projection of the Llama-110M-shaped step, one token: latency
        _mm("matmul_1x768x768", 1, 768, 768, "fp32", "fp32"),
        # the 262144-token vocabulary projection of one decoded token: HBM
        _mm("matmul_1x2048x262144", 1, 2048, 262144, "bf16", "fp32"),
        # a batch of 13 sequences decoded together
        _mm("matmul_13x4096x14336", 13, 4096, 14336, "bf16", "bf16", bias=True),
        # logits of a ragged prompt over the GPT-2 vocabulary, hidden states quantized before
        _mm("matmul_333x768x50257", 333, 768, 50257, "fp16", "fp16", codes=True),
        # the 512-token prefill product
        _mm("matmul_512x4096x14336", 512, 4096, 14336, "bf16", "bf16"),
        # the FFN of the Llama-110M-shaped step, one token
        _ug("up_gate_1x768x2048", 1, 768, 2048, "fp32", "fp32"),
        # 48 sequences decoded together
        _ug("up_gate_48x2048x5632", 48, 2048, 5632, "fp16", "fp16"),
        # a long prompt through a wide FFN, activations quantized before
        _ug("up_gate_2048x4096x14336", 2048, 4096, 14336, "bf16", "bf16", codes=True),
        # one decoded token, five alternatives: latency
        _lp("logprob_1x32000", 1, 32000, "fp32", 5, 1),
        # a decode batch over the largest vocabulary, some tokens banned by a grammar
        _lp("logprob_8x262144", 8, 262144, "fp32", 20, 1, banned=True),
        # a scored prompt over an odd vocabulary, twenty alternatives (ties are common in bf16)
        _lp("logprob_1021x50257", 1021, 50257, "bf16", 20, 1),
        # perplexity of a prompt: no alternatives
        _lp("logprob_512x262144", 512, 262144, "bf16", 0, 1),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "up_gate", "logprob"])
    t = ["fp32", "fp16", "bf16"]
    if op == "logprob":
        x_type = rng.choice(t)
        vocab = _logint(rng, 1000, 262144)
        # at most the elements of the largest listed case of the type's size
        m = _logint(rng, 1, max(1, min(2048, (1 << 28) // (SIZES[x_type] * vocab))))
        c = _lp("", m, vocab, x_type, rng.choice([0, 1, 5, 20]), rng.choice([1, 1, 3]),
                rng.random() < 0.3)
    else:
        k = 32 * _logint(rng, 8, 256)
        n = _logint(rng, 64, 28672)
        top = 2 * 2048 * 4096 * 28672                       # operations of the largest listed case
        m = _logint(rng, 1, max(1, min(2048, top // (2 * n * k))))
        if op == "matmul":
            c = _mm("", m, k, n, rng.choice(t), rng.choice(t), rng.random() < 0.4,
                    rng.random() < 0.3)
        else:
            c = _ug("", m, k, max(1, n // 2), rng.choice(t), rng.choice(t), rng.random() < 0.4)
    del c["name"]
    return c


def work(case):
    m = case["m"]
    if case["op"] == "logprob":
        v = case["vocab"]
        out = 4 * m * (case["given"] + 2) + 8 * m * case["n_top"]
        # subtract, exp, two sums with a product, a comparison per logit
        return {"bytes": m * v * SIZES[case["x_type"]] + 4 * m * case["given"] + out,
                "flops": 6 * m * v}
    k = case["k"]
    rows, cols = ((2 * case["n_ff"], case["n_ff"]) if case["op"] == "up_gate"
                  else (case["n"], case["n"]))
    x = m * k + 4 * m if case["codes"] else m * k * SIZES[case["x_type"]]
    bias = 4 * rows if case.get("bias") else 0
    return {"bytes": x + rows * k + 4 * rows + bias + m * cols * SIZES[case["y_type"]],
            "flops": 2 * m * rows * k}


# ---------------------------------------------------------------------------
# Inputs, on the GPU, from the seed alone.

def _quantize(x):
    """Codes and scales of each row: s = max|x| / 127 in fp32, code =
    sign(x) * floor(|x| / s + 1/2), the quotient in 64 bits."""
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


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m = case["m"]
    t = DTYPES[case["x_type"]]
    if case["op"] == "logprob":
        v = case["vocab"]
        x = torch.randn((m, v), generator=g, device="cuda") * 2.5
        # a few likely continuations per row, as a model's logits have
        likely = torch.randint(v, (m, 8), generator=g, device="cuda")
        x.scatter_add_(1, likely, 4.0 * torch.rand((m, 8), generator=g, device="cuda") + 6.0)
        given = torch.randint(v, (m, case["given"]), generator=g, device="cuda")
        given[:, 0] = likely[:, 0]
        if case["banned"]:
            x.masked_fill_(torch.rand((m, v), generator=g, device="cuda") < 0.1, -math.inf)
        return {"logits": x.to(t), "tokens": given.to(torch.int32)}
    k = case["k"]
    rows = 2 * case["n_ff"] if case["op"] == "up_gate" else case["n"]
    x = torch.randn((m, k), generator=g, device="cuda")
    # a few channels of hidden states are far larger than the rest
    x[:, torch.randint(k, (max(1, k // 512),), generator=g, device="cuda")] *= 12.0
    w, ws = _weights(rows, k, g)
    d = {"x": x.to(t), "w": w, "w_scale": ws, "bias": None}
    if case["codes"]:
        d["x"], d["x_scale"] = _quantize(d["x"])
    if case.get("bias"):
        d["bias"] = torch.randn(rows, generator=g, device="cuda") * 0.5
    return d


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import moe_expert_ffn_q8_amd as q
        st["q"] = q
        m = case["m"]
        if case["op"] == "logprob":
            st["ws"] = q.logprob_workspace(m, case["vocab"], case["n_top"], "cuda")
            st["out"] = q.logprob_outputs(m, case["given"], case["n_top"], "cuda")
        else:
            cols = case["n_ff"] if case["op"] == "up_gate" else case["n"]
            st["y"] = torch.empty((m, cols), dtype=DTYPES[case["y_type"]], device="cuda")
            st["ws"] = None if case["codes"] else q.i8_workspace(m, case["k"], "cuda")
    return st


# ---------------------------------------------------------------------------
# One pass.

def _plain_product(st):
    if st["case"]["codes"]:
        c, s = st["x"], st["x_scale"]
    else:
        c, s = _quantize(st["x"])
    # sums of code products pass 2^24: in 64 bits
    acc = (c.double() @ st["w"].double().t()).float()
    y = acc * s[:, None] * st["w_scale"][None, :]
    return y if st["bias"] is None else y + st["bias"]


def _plain_logprob(st):
    case, tok = st["case"], st["tokens"].long()
    x = st["logits"].float()
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    mean = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / s
    lse = top + torch.log(s)
    out = {"logprob": x.gather(1, tok) - lse, "lse": lse[:, 0],
           "entropy": (torch.log(s) - mean)[:, 0]}
    if case["n_top"]:
        v = x.shape[1]
        index = torch.arange(v, dtype=torch.int32, device=x.device)[None, :]
        last = torch.full_like(index, v)
        cur = x.clone()
        ids = torch.empty((case["m"], case["n_top"]), dtype=torch.int32, device=x.device)
        val = torch.empty((case["m"], case["n_top"]), dtype=torch.float32, device=x.device)
        for i in range(case["n_top"]):
            best = cur.amax(1, keepdim=True)
            at = torch.where(cur == best, index, last).amin(1, keepdim=True)
            ids[:, i], val[:, i] = at[:, 0], best[:, 0]
            cur.scatter_(1, at.long(), -math.inf)
        out["top_ids"], out["top_logprobs"] = ids, val - lse
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        q = state["q"]
        if op == "matmul":
            return q.i8_matmul(state["x"], state["w"], state["w_scale"],
                               x_scale=state.get("x_scale"), bias=state["bias"], y=state["y"],
                               ws=state["ws"])
        if op == "up_gate":
            return q.i8_up_gate_swiglu(state["x"], state["w"], state["w_scale"],
                                       x_scale=state.get("x_scale"), h=state["y"],
                                       ws=state["ws"])
        o = q.logprob_rows(state["logits"], state["tokens"], n_top=case["n_top"],
                           ws=state["ws"], out=state["out"])
        r = {"logprob": o.logprob, "lse": o.lse, "entropy": o.entropy}
        if case["n_top"]:
            r["top_ids"], r["top_logprobs"] = o.top_ids, o.top_logprobs
        return r
    if op == "logprob":
        return _plain_logprob(state)
    y = _plain_product(state)
    if op == "up_gate":
        g, u = y.split(case["n_ff"], dim=1)
        y = g / (1.0 + torch.exp(-g)) * u
    return y.to(DTYPES[case["y_type"]])


# ---------------------------------------------------------------------------
# The same outputs from the definition, in 64 bits.

def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "logprob":
        n_top = case["n_top"]
        rows = []
        for i in range(0, case["m"], 64):          # 64 rows at a time
            x = d["logits"][i:i + 64].double()
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            r = {"logprob": torch.gather(x, 1, d["tokens"][i:i + 64].long()) - lse[:, None],
                 "lse": lse,
                 "entropy": -torch.where(p > 0, p * (x - lse[:, None]), 0.0).sum(1)}
            if n_top:
                s, at = torch.sort(x, dim=1, descending=True, stable=True)
                r["top_ids"] = at[:, :n_top].to(torch.int32)
                r["top_logprobs"] = s[:, :n_top] - lse[:, None]
            rows.append(r)
        return {name: torch.cat([r[name] for r in rows]) for name in rows[0]}
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
    if case["op"] == "up_gate":
        gate, up = y[:, :case["n_ff"]], y[:, case["n_ff"]:]
        y = gate * torch.sigmoid(gate) * up
    return y
