"""64-bit references and error bounds of the operators around the products of a
token step: products with an activation and a residual, norms, sampling.
(Embedding rows are checked bit for bit.)  u = 2^-24, as in i8_ref."""
import math

import numpy as np

import i8_ref
from i8_ref import HALF_STEP, SUBNORMAL, U

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(act, v, b):
    """(act(v), bound) for fp32 values within b of v.  The derivatives of gelu,
    its tanh form and silu are below 1.13.
    gelu: z = -v / sqrt 2 carries 2 u, which moves erfc(z) by 2 / sqrt(pi)
    exp(-z^2) |z| 2 u; erfc itself is good to 16 units in the last place (32 u),
    and three products and roundings add 3 u.
    tanh form: s carries 6 u (two constants, two products, a fused sum, a
    product) and sigmoid's slope turns it into |v| |s| sigma (1 - sigma) 6 u; the
    exponential, the sum, the reciprocal and the products make 13 u, as in
    silu (i8_ref.gated).  Below s = -87 the true value is under 1e-36 |v|."""
    if act == "none":
        return v, b
    if act == "relu":
        return np.maximum(v, 0), b
    if act == "relu2":
        r = np.maximum(v, 0)
        return r * r, (2 * r + b) * b + 1.01 * U * r * r
    if act == "gelu":
        z = -v / math.sqrt(2)
        h = 0.5 * v * _erfc(z)
        own = np.abs(v) * np.exp(-z * z) * np.abs(z) * 2 * U * (2 / math.sqrt(math.pi)) / 2
        return h, 1.13 * b + 1.01 * (own + 35 * U * np.abs(h)) + 1e-36 * np.abs(v) + 2.0 ** -148
    s = v if act == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-s))
    h = v * sig
    own = np.abs(v * s) * sig * (1 - sig) * (0 if act == "silu" else 6 * U)
    return h, 1.13 * b + 1.01 * (own + 13 * U * np.abs(h)) + 1e-36 * np.abs(v) + 2.0 ** -148


def product_act(cx, sx, cw, sw, bias, act, residual):
    v, b = i8_ref.product(cx, sx, cw, sw, bias)
    y, b = activation(act, v, b)
    if residual is not None:
        y = y + residual
        b = b + 1.01 * U * (np.abs(y) + b)
    return y, b


# ---------------------------------------------------------------------------
# Norms.  The 64-bit arithmetic of either side is off by a few n 2^-53 of the
# sums' terms, below 2^-36 for n <= 65536; a mean taken off a row far from 0
# multiplies that by the terms' size.
#
# Rows that are all of 16-bit types are computed in 32 bits (`narrow`), by
# differences from a value p of the row, c = (x - p) - (mean - p): two differences
# and one rounding of mean - p, of terms below |c| + cmax and cmax, are off by
# u (2 |c| + 3 cmax).  The squares' sums of up to 128 terms a thread carry 130 u,
# their inverse root 65 u and 2 u of the instruction; three products and sums
# 3 u of the value before the bias and u of the value.

REL64 = 2.0 ** -36


def norm(x, weight, bias, eps, layer, narrow=False):
    """(value, bound of the arithmetic) of rows x (fp64)."""
    mean = x.mean(axis=1, keepdims=True) if layer else 0.0
    d = x - mean
    r = 1 / np.sqrt((d * d).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    y = d * r * weight
    size = (np.abs(x) + np.abs(mean)) * r * np.abs(weight)
    bound = REL64 * size
    if narrow:
        far = np.abs(d).max(axis=1, keepdims=True) if layer else 0.0
        bound = bound + 1.01 * U * (r * np.abs(weight) * (2 * np.abs(d) + 3 * far) + 71 * np.abs(y))
    if bias is not None:
        y = y + bias
        bound = bound + REL64 * np.abs(bias) + (U * np.abs(y) if narrow else 0)
    return y, bound


def residual(x, r, post_weight, post_bias, gate, residual_scale, eps, layer, narrow=False):
    a, b = norm(x, post_weight, post_bias, eps, layer, narrow) if post_weight is not None else (x, 0.0)
    g = 1.0 if gate is None else gate
    y = g * a + float(np.float32(residual_scale)) * r
    rel = (3 * U if narrow else 0) + REL64            # the gate's product and the fused sum
    return y, np.abs(g) * b + rel * (np.abs(g * a) + np.abs(residual_scale * r))


def assert_rounded(got, value, bound, t, what):
    """fp64 values rounded to fp32 and then to type t."""
    i8_ref.assert_close(got, value, bound + U * (np.abs(value) + bound), t, what)


# ---------------------------------------------------------------------------
# Sampling.

def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row (fp64 values of the logits) by sorting it: a dict with the order,
    the range of sizes of what is kept, the range of places of the drawn token,
    and the log probability of a place.  The library sums whole units of
    2^-52, or of 2^-60 of the sum (of n where no sum is taken): targets are met within n of them, and where that much
    decides, either side may come out."""
    if np.isnan(x).any() or np.isposinf(x).any():
        return {"id": -1, "kept": 0, "logprob": np.nan}
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    n = len(order)
    if n == 0:
        return {"id": -1, "kept": 0, "logprob": -np.inf}
    if not temperature > 0:
        return {"id": int(order[0]), "kept": 1, "logprob": 0.0}
    z = (x[order] - x[order[0]]) / float(np.float32(temperature))
    w = np.exp(z.astype(np.longdouble))
    c = np.cumsum(w)
    most = n if top_k > 0 or (min_p > 0 and not top_p < 1) else float(c[-1])
    slack = n * max(2.0 ** -52, most * 2.0 ** -60)
    whole = bool(np.all(w == 1))          # whole numbers of units: targets are met exactly

    def reach(target, strict):
        """Range of how many tokens it takes to reach (pass) a mass."""
        side, off = "right" if strict else "left", 0.0 if whole else slack + 1e-12 * float(target)
        return tuple(max(1, int(np.searchsorted(c, target + d, side)) + 1) for d in (-off, off))

    k = min(n, top_k) if top_k > 0 else n
    lo = hi = k
    if top_p < 1:
        a, b = reach(np.longdouble(np.float32(max(top_p, 0.0))) * c[k - 1], False)
        lo, hi = min(lo, a), min(hi, b)
    if min_p > 0:
        p = min(float(np.float32(min_p)), 1.0)
        lo = min(lo, max(1, int((w >= p * (1 + (1e-12 if p < 1 else 0))).sum())))
        hi = min(hi, max(1, int((w >= p * (1 - (1e-12 if p < 1 else 0))).sum())))
    u = float(np.float32(u))
    u = 0.0 if not u > 0 else u
    first = min(reach(np.longdouble(u) * c[lo - 1], True)[0], lo) if u < 1 else 1
    last = min(reach(np.longdouble(u) * c[hi - 1], True)[1], hi) if u < 1 else hi
    return {"order": order, "kept": (lo, hi), "place": (first, last), "z": z, "mass": c, "slack": slack / float(c[0]) + 1e-12}


def assert_sample(got, ref, what=""):
    """got: (id, logprob, kept) of a row."""
    i, lp, kept = int(got[0]), float(got[1]), int(got[2])
    if "id" in ref:
        assert (i, kept) == (ref["id"], ref["kept"]), (what, got, ref)
        assert lp == ref["logprob"] or (np.isnan(lp) and np.isnan(ref["logprob"])), (what, got, ref)
        return 0
    lo, hi = ref["kept"]
    assert lo <= kept <= hi, f"{what}: kept {kept}, expected {lo} to {hi}"
    first, last = ref["place"]
    places = ref["order"][first - 1:last]
    at = np.flatnonzero(places == i)
    assert len(at) == 1, f"{what}: id {i}, expected one of {places[:4]} (places {first} to {last})"
    z = ref["z"][first - 1 + at[0]]
    want = float(z - np.log(ref["mass"][kept - 1]))
    tol = 1.01 * (U * abs(want) + 2 * ref["slack"] + 2.0 ** -48 * (1 + abs(z))) + 2.0 ** -149
    assert abs(lp - min(want, 0.0)) <= tol, f"{what}: logprob {lp!r}, expected {want!r}"
    return int(lo != hi or first != last)
