"""The training operators in fp64 numpy, written from their definitions, and
the bounds the GPU results are held to.

Every bound counts roundings: u = 2^-24 is an fp32 rounding, half an eps of the
result's type its last one.  Hardware exp2, rcp and sqrt are within 1 ulp
(2u).  A sum of m fp32 terms added one after another is within m u times the
sum of their magnitudes.
"""
import math

import numpy as np

BLOCK = 128
LEAST = 2.0 ** -100
U = 2.0 ** -24
HALF_EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
# half the spacing of the smallest values (fp16 has only 2^-24 below 2^-14)
HALF_LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def rounding(value, dtype):
    """The result's own rounding."""
    return HALF_EPS[dtype] * np.abs(value) + HALF_LEAST[dtype]


# ---- 8-bit blocks --------------------------------------------------------------

def blocks(d):
    return -(-d // BLOCK)


def encode(x, positive=False):
    """(codes, scales, quotients) of x [..., d] (values exact in fp64)."""
    d = x.shape[-1]
    nb = blocks(d)
    pad = np.zeros(x.shape[:-1] + (nb * BLOCK,))
    pad[..., :d] = x
    pad = pad.reshape(x.shape[:-1] + (nb, BLOCK))
    with np.errstate(invalid="ignore"):
        top = np.abs(pad).max(-1, keepdims=True)          # NaN stays
        bad = ~(top < 2.0 ** 126)
        top = np.where(bad, 1.0, np.maximum(top, LEAST))
        quotient = np.where(bad, 0.0, 127.0 * np.where(bad, 0.0, pad) / top)
    codes = np.rint(quotient)                             # ties to even
    if positive:
        codes = np.where((pad > 0) & ~bad, np.maximum(codes, 1.0), codes)
    scales = np.where(bad, np.nan, top / 127.0)[..., 0]
    shape = x.shape[:-1] + (nb * BLOCK,)
    return codes.reshape(shape)[..., :d].astype(np.int8), scales, quotient.reshape(shape)[..., :d]


def decode(codes, scales):
    """What fp32 scales and int8 codes stand for, exactly."""
    d = codes.shape[-1]
    wide = np.repeat(scales.astype(np.float64), BLOCK, axis=-1)[..., :d]
    return codes.astype(np.float64) * wide


# ---- activations: value, slope and their bounds ---------------------------------

def sigmoid(w):
    return np.where(w >= 0, 1.0 / (1.0 + np.exp(-np.abs(w))), np.exp(-np.abs(w)) / (1.0 + np.exp(-np.abs(w))))


_erf = np.vectorize(math.erf, otypes=[float])


def activation(act, x):
    """f(x), f'(x) and bounds of their fp32 errors."""
    if act == "squared_relu":
        r = np.maximum(x, 0.0)
        return r * r, 2.0 * r, 2 * U * r * r, 2 * U * r
    if act == "gelu":
        # the erf approximation's 1.5e-7 in erf is 7.5e-8 in Phi; the hardware functions and the
        # polynomial add a few roundings of values up to 1/2 each (16 u in all)
        cdf = 0.5 * (1.0 + _erf(x * math.sqrt(0.5)))
        phi = np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
        off = 7.5e-8 + 16 * U
        arg = 0.5 * x * x * math.log2(math.e)             # the exponent's own rounding, 2 u of it, times ln 2
        return x * cdf, cdf + x * phi, np.abs(x) * off, off + np.abs(x) * phi * (4 * arg + 8) * U
    # x p with p = 1 / (1 + 2^-w): w is rounded three times, so 2^-w is off by 3 u |w| ln 2 <= 3 u |w|
    # relative, and exp2, the sum, rcp and the product add 2 + 1 + 2 + 1
    if act == "silu":
        w, slope_of_w = x, np.ones_like(x)
    else:
        a, b = 2.0 * math.sqrt(2.0 / math.pi), 2.0 * math.sqrt(2.0 / math.pi) * 0.044715
        w, slope_of_w = x * (a + b * x * x), a + 3.0 * b * x * x
    p = sigmoid(w)
    rel = (3.0 * 1.45 * np.abs(w) + 6.0) * U
    f = x * p
    df = p + f * (1.0 - p) * slope_of_w
    # 1 - p is off by rel p (1 - p) (through 2^-w) and a rounding; f and the products by rel + 3 u
    bound_df = p * rel + np.abs(f) * slope_of_w * (2.0 * rel + 4.0 * U)
    tiny = 2.0 ** -120                                    # 2^-w past fp32's range
    return f, df, np.abs(f) * (rel + 2 * U) + np.abs(x) * tiny, bound_df + tiny


def halves(act):
    return 1 if act == "squared_relu" else 2


def forward(act, x, dtype, z=None):
    """(out, bound) of x [rows, halves * d]."""
    if act == "squared_relu":
        f, _, bf, _ = activation(act, x)
        return f, bf + rounding(f, dtype)
    d = x.shape[1] // 2
    gate, up = x[:, :d], x[:, d:]
    if act == "gelu_sparse":
        t = over_cutoff(gate, z)[0]
        f, df, bf, _ = activation("gelu_tanh", np.maximum(t, 0.0))
        bf = bf + np.abs(df) * U * np.abs(t)              # t's rounding to fp32
    else:
        f, _, bf, _ = activation(act, gate)
    out = f * up
    return out, (bf + 2 * U * np.abs(f)) * np.abs(up) + rounding(out, dtype)


def backward(act, dout, parts, dtype):
    """(dx, bound) at the exact values of parts: (x,) or (gate, up)."""
    f, df, bf, bdf = activation(act, parts[0])
    if act == "squared_relu":
        dx = dout * df
        return dx, np.abs(dout) * (bdf + 2 * U * np.abs(df)) + rounding(dx, dtype)
    up = parts[1]
    dg, du = dout * up * df, dout * f
    bg = np.abs(dout * up) * (bdf + 3 * U * np.abs(df))
    bu = np.abs(dout) * (bf + 2 * U * np.abs(f))
    return np.concatenate([dg, du], 1), np.concatenate([bg + rounding(dg, dtype), bu + rounding(du, dtype)], 1)


def over_cutoff(gate, z):
    """gate - cutoff, cutoff and std by row (population statistics)."""
    mean = gate.mean(1, keepdims=True)
    std = np.sqrt(np.square(gate - mean).mean(1, keepdims=True))
    std = np.where((gate == gate[:, :1]).all(1, keepdims=True), 0.0, std)  # a constant row has none
    mean = np.where(std == 0.0, gate[:, :1], mean)
    cutoff = mean + z * std
    return gate - cutoff, cutoff, std


def sparse_backward(dout, t, std, up, z, dtype):
    """(dx, bound) of the sparse GELU at the given t = gate - cutoff."""
    d = t.shape[1]
    s = np.maximum(t, 0.0)
    f, df, bf, bdf = activation("gelu_tanh", s)
    on = t > 0
    q = np.where(on, dout * up * df, 0.0)
    bq = np.where(on, np.abs(dout * up) * (bdf + 3 * U * np.abs(df) + 2 * U * np.abs(t)), 0.0)
    total = q.sum(1, keepdims=True)
    # G: at most 64 values a lane one after another, then 6 + 16 partial sums
    btotal = bq.sum(1, keepdims=True) + 90 * U * np.abs(q).sum(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        a = np.where(std > 0, 1.0 + z * z, 1.0)
        b = np.where(std > 0, z / std, 0.0)
    bracket = a + b * t
    size = np.abs(a) + np.abs(b * t)
    dg = q - total / d * bracket
    bg = bq + btotal / d * np.abs(bracket) + np.abs(total) / d * size * 8 * U + 2 * U * np.abs(q)
    du = dout * f
    bu = np.abs(dout) * (bf + 2 * U * np.abs(f) + 2 * U * np.abs(df * t) * on)
    return np.concatenate([dg, du], 1), np.concatenate([bg + rounding(dg, dtype), bu + rounding(du, dtype)], 1)


# ---- layer norm -----------------------------------------------------------------

def layer_norm(x, w, b, eps, dtype):
    """(y, bound, mean, rstd)."""
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(np.square(x - mean).mean(1, keepdims=True) + eps)
    n = (x - mean) * rstd
    y = n * w + b
    # x - mean, rstd and their product are rounded once each, the last fma once
    return y, 4 * U * (np.abs(n * w) + np.abs(b)) + rounding(y, dtype), mean, rstd


def layer_norm_backward(dy, n, rstd, w, dtype, wdtype, sequential):
    """((dx, dw, db), bounds) at exact n; `sequential`: the most terms a lane adds in a row's sums."""
    d = n.shape[1]
    v = dy * w
    m1, m2 = v.mean(1, keepdims=True), (v * n).mean(1, keepdims=True)
    dx = rstd * (v - m1 - n * m2)
    k = (sequential + 40) * U
    bdx = np.abs(rstd) * (8 * U * (np.abs(v) + np.abs(m1) + np.abs(n * m2))
                          + k * (np.abs(v).mean(1, keepdims=True) + np.abs(n) * np.abs(v * n).mean(1, keepdims=True)))
    dw, db = (dy * n).sum(0), dy.sum(0)
    rows = dy.shape[0]
    bw = (rows + 40) * U * np.abs(dy * n).sum(0) + rounding(dw, wdtype)
    bb = (rows + 40) * U * np.abs(dy).sum(0) + rounding(db, wdtype)
    del d
    return (dx, dw, db), (bdx + rounding(dx, dtype), bw, bb)


# ---- balance loss ---------------------------------------------------------------

def softmax(logits):
    with np.errstate(invalid="ignore"):
        top = logits.max(1, keepdims=True)
        p = np.exp(logits - np.where(np.isneginf(top), 0.0, top))
        s = p.sum(1, keepdims=True)
        return np.where(s == 0.0, 0.0, p / np.where(s == 0.0, 1.0, s))


def balance(logits, index, coefficient, use):
    """(loss, bound, counts, offsets, n) over the rows where use is true."""
    rows, e = logits.shape
    k = index.shape[1]
    chosen = index[use].reshape(-1)
    counts = np.bincount(chosen[(chosen >= 0) & (chosen < e)], minlength=e)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    n = int(use.sum())
    if n == 0:
        return 0.0, 0.0, counts, offsets, 0
    p = softmax(logits[use])
    loss = coefficient * e / (k * n * n) * (counts * p.sum(0)).sum()
    return loss, abs(loss) * (relative_softmax(logits[use]) + (n + 1200) * U), counts, offsets, n


def relative_softmax(logits):
    """p's relative error: the exponent (l - max) log2(e) rounded twice, at most 3 u of it in base e; exp2,
    the sum of up to 1024 terms in lanes of 16, the division and the product."""
    finite = np.where(np.isfinite(logits), logits, 0.0)
    spread = (finite.max(1) - finite.min(1)).max() if logits.size else 0.0
    return 2 * (3 * spread + 40) * U


def balance_backward(logits, counts, k, coefficient, n, use, dloss, dtype):
    rows, e = logits.shape
    if n == 0:
        return np.zeros_like(logits), np.full_like(logits, HALF_LEAST[dtype])
    p = softmax(logits)
    factor = dloss * coefficient * e / (k * n * n)
    off = counts - counts.mean()
    dot = (p * off).sum(1, keepdims=True)
    live = p.sum(1, keepdims=True) > 0
    g = np.where(use[:, None] & live, factor * p * (off - dot), 0.0)
    rel = relative_softmax(logits)
    # the kernel takes the counts from floor(mean), so off carries up to 1 more
    size = np.abs(off) + 1.0 + (p * (np.abs(off) + 1.0)).sum(1, keepdims=True)
    bound = np.where(use[:, None] & live, abs(factor) * p * size * (2 * rel + 40 * U), 0.0)
    return g, bound + rounding(g, dtype)
