"""The fp64 reference of the training operators against differences of its own
forward passes, and the 8-bit code against exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

import train_ref as ref

H = 1e-6


def _difference(f, x, dout):
    """d sum(dout f(x)) / dx by central differences, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        g[i] = ((f(a) - f(b)) * dout).sum() / (2 * H)
    return g


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu", "squared_relu"])
def test_activation_gradient(act):
    rng = np.random.default_rng(1)
    h = ref.halves(act)
    x = rng.normal(0, 2, (3, h * 9))
    dout = rng.normal(0, 1, (3, 9))
    parts = (x,) if h == 1 else (x[:, :9], x[:, 9:])
    dx, _ = ref.backward(act, dout, parts, "fp32")
    np.testing.assert_allclose(dx, _difference(lambda v: ref.forward(act, v, "fp32")[0], x, dout), atol=1e-7, rtol=1e-6)


@pytest.mark.parametrize("z", [1.6448536, -0.5, 0.0])
def test_sparse_gradient_through_the_statistics(z):
    rng = np.random.default_rng(2)
    x = rng.normal(0.4, 2, (4, 2 * 24))
    dout = rng.normal(0, 1, (4, 24))
    t, _, std = ref.over_cutoff(x[:, :24], z)
    assert np.abs(t).min() > 1e3 * H            # no value within a difference of its cutoff
    dx, _ = ref.sparse_backward(dout, t, std, x[:, 24:], z, "fp32")
    np.testing.assert_allclose(dx, _difference(lambda v: ref.forward("gelu_sparse", v, "fp32", z)[0], x, dout),
                               atol=1e-7, rtol=1e-6)


def test_layer_norm_gradient():
    rng = np.random.default_rng(3)
    x, dy = rng.normal(1, 2, (3, 17)), rng.normal(0, 1, (3, 17))
    w, b = rng.normal(1, 0.3, 17), rng.normal(0, 0.3, 17)
    _, _, mean, rstd = ref.layer_norm(x, w, b, 1e-5, "fp32")
    (dx, dw, db), _ = ref.layer_norm_backward(dy, (x - mean) * rstd, rstd, w, "fp32", "fp32", 8)
    for got, at, f in ((dx, x, lambda v: ref.layer_norm(v, w, b, 1e-5, "fp32")[0]),
                       (dw, w, lambda v: ref.layer_norm(x, v, b, 1e-5, "fp32")[0]),
                       (db, b, lambda v: ref.layer_norm(x, w, v, 1e-5, "fp32")[0])):
        np.testing.assert_allclose(got, _difference(f, at, dy), atol=1e-7, rtol=1e-6)


def test_balance_gradient():
    rng = np.random.default_rng(4)
    logits = rng.normal(0, 1, (7, 5))
    index = rng.integers(-1, 6, (7, 2))
    use = np.array([1, 1, 0, 1, 1, 1, 0], bool)
    _, _, counts, offsets, n = ref.balance(logits, index, 0.7, use)
    assert n == 5 and offsets[-1] == counts.sum() == ((index[use] >= 0) & (index[use] < 5)).sum()
    g, _ = ref.balance_backward(logits, counts, 2, 0.7, n, use, 1.5, "fp32")
    fd = _difference(lambda v: np.asarray(ref.balance(v, index, 0.7, use)[0]), logits, np.asarray(1.5))
    np.testing.assert_allclose(g, fd, atol=1e-8, rtol=1e-6)


def test_code_is_the_exact_quotient_rounded():
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (6, 300)).astype(np.float32)
    x[1] = (rng.integers(-254, 255, 300) * 0.5).astype(np.float32)   # halves: ties where the largest is 127
    x[1, :2], x[1, 128], x[1, 256] = (127.0, 0.5), 127.0, 127.0
    codes, scales, _ = ref.encode(x.astype(np.float64))
    for r in range(6):
        for c in range(300):
            top = max(Fraction(float(abs(v))) for v in x[r, c // 128 * 128:c // 128 * 128 + 128])
            assert codes[r, c] == round(127 * Fraction(float(x[r, c])) / top)     # Python rounds halves to even
    back = ref.decode(codes, scales)
    top = np.repeat(scales * 127, 128, axis=1)[:, :300]
    assert np.all(np.abs(back - x) <= top / 254 * (1 + 1e-12))


def test_code_of_unusual_blocks():
    x = np.zeros((4, 130))
    x[1, 5] = np.inf
    x[2, 129] = np.nan
    x[3, 0] = 2.0 ** -120
    codes, scales, _ = ref.encode(x)
    assert (codes == 0).all()
    assert np.isnan(scales[1, 0]) and scales[1, 1] == ref.LEAST / 127 and np.isnan(scales[2, 1])
    positive, _, _ = ref.encode(x, positive=True)
    assert positive[3, 0] == 1 and (np.delete(positive.reshape(-1), 3 * 130) == 0).all()
