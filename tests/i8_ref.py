"""64-bit references and error bounds of the 8-bit products with token and
channel scales and of the log probabilities, in numpy.

u = 2^-24 is half a step of fp32.  A value y of a type t with step eps (relative
to a power of two) is stored within eps/2 * |y|, or within half its smallest
subnormal."""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -24, "bf16": 2.0 ** -133}
TYPES = ("fp32", "fp16", "bf16")


def torch_type(t):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[t]


def quantize(x):
    """fp32 [rows][k] -> (codes int8, scales fp32).  The 64-bit quotient of two
    fp32 values decides every rounding: |x| - (q + 1/2) s is a multiple of the
    last place of a 32-bit product, far above 2^-53 of it."""
    x = np.asarray(x, dtype=np.float32)
    ok = np.isfinite(x).all(axis=1)
    a = np.where(ok, np.abs(np.where(np.isfinite(x), x, 0)).max(axis=1), 0).astype(np.float32)
    s = (a / np.float32(127.0)).astype(np.float32)
    live = s > 0
    d = np.where(live, s, 1).astype(np.float64)
    v = np.abs(np.where(ok[:, None], x, 0).astype(np.float64)) / d[:, None]
    c = np.minimum(np.floor(v + 0.5), 127) * np.sign(np.where(ok[:, None], x, 0))
    c = np.where(live[:, None], c, 0).astype(np.int8)
    return c, np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def sums(cx, cw):
    """Exact sums of code products (|sum| < 2^31 fits a double)."""
    return cx.astype(np.float64) @ cw.astype(np.float64).T


def product(cx, sx, cw, sw, bias=None):
    """(value, bound of the fp32 arithmetic): the sum's conversion and the two
    scale products, or the product and the fused multiply-add, are 3 roundings
    of at most u each."""
    p = sums(cx, cw) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    b = np.zeros(cw.shape[0]) if bias is None else bias.astype(np.float64)
    y = p + b
    return y, 1.01 * U * (2 * np.abs(p) + np.abs(y) + (np.abs(p) if bias is None else 0)) + 2.0 ** -149


def gated(cx, sx, cw, sw):
    """silu(g) * u and the bound of its fp32 arithmetic: g and u carry 3 u
    each, and silu turns a relative error of g into 1 + |g| (1 - sigmoid(g))
    times that; the exponential (2 u of the instruction, 2 u of the argument's
    rest, 1 u of the correction), the sum, the reciprocal (2 u) and two
    products make 10 u.  exp(-g) overflows below g = -88: there the true value
    is under 1e-36 * |u|."""
    y, _ = product(cx, sx, cw, sw)
    n = y.shape[1] // 2
    g, up = y[:, :n], y[:, n:]
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-g))
    h = g * sig * up
    return h, 1.01 * U * np.abs(h) * (3 * (1 + np.abs(g) * (1 - sig)) + 3 + 10) + 1e-36 * np.abs(up) + 2.0 ** -148


def assert_close(got, ref, bound, t, what=""):
    """|got - ref| <= bound + the rounding to type t (NaN where ref is NaN)."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    tol = bound + HALF_STEP[t] * (np.abs(ref) + bound) + SUBNORMAL[t]
    big = {"fp32": 3.4028234e38, "fp16": 65504.0, "bf16": 3.3895314e38}[t]
    over = ~nan & (np.abs(ref) * (1 + 2 * HALF_STEP[t]) + bound > big)  # may round to infinity
    fine = nan | over | (np.abs(got - np.where(nan, 0, ref)) <= tol)
    if not fine.all():
        i = tuple(np.argwhere(~fine)[0])
        raise AssertionError(f"{what}: {(~fine).sum()} of {fine.size} off, first at {i}: got "
                             f"{got[i]!r}, expected {ref[i]!r} +- {tol[i]:.3e}")


def logprobs(x, tokens, n_top):
    """The outputs for rows x (fp64) and their bounds, as a dict of (value,
    bound).  With d = x - M, E = sum p |d| (finite d), and c = V / 64 + 32, no
    chain of additions being longer: exp(d) is off by (|d| + 3) 2u (argument
    and instruction), so S by (E + 3) 2u + c u relative, and so are W's terms
    with 1 u more."""
    m, v = x.shape
    out = {}
    nan = np.isnan(x).any(axis=1) | np.isposinf(x).any(axis=1)
    safe = np.where(nan[:, None], 0.0, x)
    top = safe.max(axis=1, keepdims=True)
    empty = np.isneginf(top[:, 0])
    top = np.where(empty[:, None], 0.0, top)
    d = safe - top
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.exp(d)
        s = e.sum(axis=1)
        ls = np.log(s)
        lse = top[:, 0] + ls
        p = e / s[:, None]
        pd = np.where(e > 0, p * d, 0.0)
        ent = np.where(empty, 0.0, ls - pd.sum(axis=1))
        aver = np.where(empty, 0.0, np.abs(pd).sum(axis=1))
    rel = U * (2 * (aver + 3) + v / 64 + 32)
    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0.0)
    b_lse = 1.01 * (rel + 3 * U * fin(ls) + U * fin(lse))
    b_ent = 1.01 * (rel * (1 + aver) * 2 + U * np.abs(pd * np.where(e > 0, d, 0.0)).sum(axis=1) * 2
                    + 4 * U * (fin(ls) + aver))
    def mask(a):
        return np.where(nan.reshape((-1,) + (1,) * (a.ndim - 1)), np.nan, a)
    out["lse"] = (mask(lse), b_lse)
    out["entropy"] = (mask(ent), b_ent)
    def lp(vals):
        with np.errstate(invalid="ignore"):
            r = np.where(empty[:, None], -np.inf, vals - lse[:, None])
        return mask(r), b_lse[:, None] + 1.01 * U * fin(r)
    if tokens is not None:
        ok = (tokens >= 0) & (tokens < v)
        val, b = lp(np.take_along_axis(safe, np.where(ok, tokens, 0).astype(np.int64), axis=1))
        out["logprob"] = (np.where(ok, val, np.nan), b)
    if n_top:
        key = np.where(np.isnan(x), -np.inf, x)
        # -infinity before NaN: stable sort on (NaN, -value)
        order = np.lexsort((np.broadcast_to(np.arange(v), x.shape), -key, np.isnan(x)), axis=1)
        ids = order[:, :n_top].astype(np.int32)
        out["top_ids"] = ids
        out["top_logprobs"] = lp(np.take_along_axis(safe, ids.astype(np.int64), axis=1))
    return out


def assert_logprobs(got, ref):
    """got: a LogprobOut on the host side (numpy); ref: logprobs(...)."""
    for name, r in ref.items():
        g = getattr(got, name).cpu().numpy()
        if name == "top_ids":
            assert np.array_equal(g, r), f"top_ids differ in rows {np.argwhere((g != r).any(1))[:4].ravel()}"
            continue
        val, bound = r
        g = g.astype(np.float64).reshape(val.shape)
        assert np.array_equal(np.isnan(g), np.isnan(val)), f"{name}: NaN in other places"
        assert np.array_equal(np.isneginf(g), np.isneginf(val)), f"{name}: -infinity in other places"
        fin = np.isfinite(val)
        err = np.abs(np.where(fin, g - np.where(fin, val, 0), 0))
        tol = np.broadcast_to(bound, val.shape) + 2.0 ** -149
        assert (err <= tol).all(), (f"{name}: worst {np.max(err / tol):.2f} of the bound at "
                                    f"{np.unravel_index(np.argmax(err / tol), val.shape)}")
