"""The feed-forward layer and microscaled 4-bit arrays in fp64 numpy, written
from their definitions, and the bounds the GPU results are held to.

u = 2^-24 is an fp32 rounding.  A sum of n fp32 products on the matrix cores is
counted as n + 8 additions that are each off by at most 2 u (they may truncate)
of the sum of magnitudes.  A rounding to 16 bits is half an eps of the type.
Element by element every bound adds magnitudes, so it holds whatever the signs.
Over many outputs the roundings of the terms are independent and each at most
half an eps, so the errors' 2-norm stays below half an eps of the 2-norm of the
root of the terms' squares: `spread` holds that, and it is the sharper check of
long sums.
"""
import numpy as np

import train_ref as ref
from train_ref import HALF_EPS, U, rounding

GROUP = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def product(a, b):
    """a b^T of fp64 [m, k], [n, k]: (value, bound of the fp32 sum)."""
    return a @ b.T, 2 * (a.shape[1] + 8) * U * (np.abs(a) @ np.abs(b).T)


def through(error, b):
    """What errors of a's elements do to a b^T."""
    return error @ np.abs(b).T


def spread(a, b):
    return np.sqrt(np.square(a) @ np.square(b).T)


def value_and_slopes(act, z):
    """h, its derivatives by gate and up (None: not gated), and h's fp32 bound."""
    if act == "squared_relu":
        f, df, bf, _ = ref.activation(act, z)
        return f, df, None, bf
    d = z.shape[1] // 2
    f, df, bf, _ = ref.activation(act, z[:, :d])
    up = z[:, d:]
    return f * up, df * up, f, (bf + 2 * U * np.abs(f)) * np.abs(up)


def hidden(act, x, w_in):
    """(z, bound of z, h, bound of h) in fp32, before any rounding to 16 bits."""
    z, bz = product(x, w_in)
    h, by_gate, by_up, bh = value_and_slopes(act, z)
    d = h.shape[1]
    if by_up is None:
        # the slope may change by twice the step within it
        return z, bz, h, bh + (np.abs(by_gate) + 2 * bz) * bz
    bg, bu = bz[:, :d], bz[:, d:]
    # |f''| < 2 for all of them
    return z, bz, h, bh + (np.abs(by_gate) + 2 * bg * np.abs(z[:, d:])) * bg + (np.abs(by_up) + 2 * bg) * bu


def forward(act, x, w_in, w_down, dtype):
    """(y, bound, its spread, z, bound of the kept z)."""
    z, bz, h, bh = hidden(act, x, w_in)
    bh = bh + rounding(h, dtype)
    y, by = product(h, w_down)
    return y, by + through(bh, w_down) + rounding(y, dtype), spread(h, w_down), z, bz + rounding(z, dtype)


def backward(act, dy, x, z, w_in, w_down, dtype):
    """[(gradient, bound, spread)] of dx, dw_in, dw_down at the kept z."""
    dh, bdh = product(dy, w_down.T)
    d = dh.shape[1]
    f, df, bf, bdf = ref.activation(act, z[:, :d])
    if act == "squared_relu":
        h, bh = f, bf
        dz = dh * df
        bdz = np.abs(df) * bdh + np.abs(dh) * bdf + 2 * U * np.abs(dz)
    else:
        up = z[:, d:]
        h, bh = f * up, (bf + 2 * U * np.abs(f)) * np.abs(up)
        dg, du = dh * up * df, dh * f
        bg = np.abs(up * df) * bdh + np.abs(dh * up) * bdf + 3 * U * np.abs(dg)
        bu = np.abs(f) * bdh + np.abs(dh) * bf + 2 * U * np.abs(du)
        dz, bdz = np.concatenate([dg, du], 1), np.concatenate([bg, bu], 1)
    bdz, bh = bdz + rounding(dz, dtype), bh + rounding(h, dtype)
    out = []
    for a, ba, b in ((dz, bdz, w_in.T), (dz.T, bdz.T, x.T), (dy.T, None, h.T)):
        v, bv = product(a, b)
        bv = bv + (through(ba, b) if ba is not None else np.abs(a) @ bh)
        out.append((v, bv + rounding(v, dtype), spread(a, b)))
    return out


def norm_bound(value, spread_of, dtype):
    """Of the 2-norm of the errors: the terms' roundings and the result's own, and half as much again for
    what a finite number of outputs strays."""
    return 1.5 * HALF_EPS[dtype] * (np.linalg.norm(spread_of) + np.linalg.norm(value)) + 1e-30


# ---- microscaled 4 bits -----------------------------------------------------------

def groups(d):
    return -(-d // GROUP)


def _blocks(x):
    rows, d = x.shape
    whole = np.zeros((rows, groups(d) * GROUP))
    whole[:, :d] = x
    return whole.reshape(rows, groups(d), GROUP)


def scale_bytes(x):
    """uint8 [rows, blocks] of x [rows, d]."""
    b = _blocks(x)
    with np.errstate(invalid="ignore"):
        top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1          # floor(log2)
    return np.where(bad, 255, np.where(top == 0, 0, np.maximum(e - 2 + 127, 0))).astype(np.uint8)


def codes_of(x, scales):
    """uint8 [rows, 32 blocks], one code a value, by the nearest level (ties to the even one)."""
    b = _blocks(x)
    bad = (scales == 255)[..., None]
    with np.errstate(invalid="ignore"):
        y = np.abs(np.where(bad, 0.0, b)) / np.exp2(np.where(bad, 0.0, scales[..., None].astype(np.float64) - 127.0))
    k = np.zeros(y.shape, np.uint8)
    for i in range(1, 8):
        border = (LEVELS[i - 1] + LEVELS[i]) / 2
        k += (y >= border) if i % 2 == 0 else (y > border)
    k = np.where(np.signbit(b) & ~bad, k | 8, k)
    return k.reshape(x.shape[0], groups(x.shape[1]) * GROUP).astype(np.uint8)


def pack(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def unpack(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def quantize(x):
    s = scale_bytes(x)
    return pack(codes_of(x, s)), s


def values(packed, scales, d):
    """fp64 [rows, d], exactly."""
    c = unpack(packed)
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return (v.reshape(len(c), groups(d), GROUP) * s[..., None]).reshape(c.shape)[:, :d]


def quantized(x):
    return values(*quantize(x), x.shape[1])


def quantized_within(h, error):
    """What 4 bits keep of h, and how far the kept value of a number within `error` of h may be from that:
    nothing where its code is certain; else two codes of the same number in two blocks' scales, each within
    its largest step (2, and 2 past the largest level) of the number."""
    q = quantized(h)
    low, high = np.maximum(np.abs(h) - error, 0.0), np.abs(h) + error
    s = scale_bytes(h)
    # a block's scale is certain if its largest value crosses no power of two either way
    certain = (scale_bytes(low) == s) & (scale_bytes(high) == s)
    # (a number that may have either sign and a code of 0 is worth 0 in both)
    same = codes_of(low, s) == codes_of(high, s)
    sure = same & np.repeat(certain, GROUP, axis=1)
    step = np.repeat(np.exp2(s.astype(np.float64) - 127.0), GROUP, axis=1)
    return q, np.where(sure, 0.0, 6.0 * step)[:, :h.shape[1]]


def product4(a, b, dtype):
    v, bound = product(a, b)
    return v, bound + rounding(v, dtype)


def layer4(act, x, w_in, w_down, dtype):
    """(y, bound) at the exact values of w_in, w_down and the quantised x."""
    _, _, h, bh = hidden(act, quantized(x), w_in)
    q, off = quantized_within(h, bh)
    y, by = product(q, w_down)
    return y, by + through(off, w_down) + rounding(y, dtype)
