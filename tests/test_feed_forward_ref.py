"""The fp64 reference of the feed-forward layer and the 4-bit arrays, on the CPU:
against another way to say the same, and mistakes planted in it."""
import numpy as np
import pytest

import feed_forward_ref as ff
import train_ref as ref

ACTS = ["silu", "gelu_tanh", "gelu", "squared_relu"]


def _layer(act, rng, rows=5, H=8, d=6):
    h = ref.halves(act)
    return rng.normal(0, 1, (rows, H)), rng.normal(0, H ** -0.5, (h * d, H)), rng.normal(0, d ** -0.5, (H, d))


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    x, w_in, w_down = _layer(act, rng)
    dy = rng.normal(0, 1, x.shape)
    z = x @ w_in.T
    grads = [g for g, _, _ in ff.backward(act, dy, x, z, w_in, w_down, "fp32")]
    for i, g in enumerate(grads):
        for _ in range(3):
            v = rng.normal(0, 1, g.shape)
            at = []
            for s in (1e-5, -1e-5):
                a = [x, w_in, w_down]
                a[i] = a[i] + s * v
                at.append((ff.forward(act, *a, "fp32")[0] * dy).sum())
            assert abs((at[0] - at[1]) / 2e-5 - (g * v).sum()) < 1e-7 * (1 + np.abs(g * v).sum())


def test_levels_are_the_nearest():
    """Every code by brute force over the sixteen values, ties to the even code."""
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, (40, 64)), np.arange(-64, 64).reshape(2, 64) / 16.0, np.zeros((1, 64))])
    s = ff.scale_bytes(x)
    codes = ff.codes_of(x, s)
    unit = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    off = np.abs(np.abs(x / unit)[..., None] - ff.LEVELS)
    best = off.min(-1)
    for i, j in np.ndindex(x.shape):
        ties = np.flatnonzero(off[i, j] == best[i, j])
        want = ties[0] if len(ties) == 1 else [t for t in ties if t % 2 == 0][0]
        assert codes[i, j] & 7 == want and bool(codes[i, j] & 8) == bool(np.signbit(x[i, j]))
    top = np.abs(x.reshape(-1, 2, 32)).max(-1)
    lead = top / np.exp2(s.astype(float) - 127)
    assert np.all((lead >= 4) & (lead < 8) | (top == 0))


def test_pack_and_values_invert():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (7, 96)).astype(np.uint8)
    assert np.array_equal(ff.unpack(ff.pack(codes)), codes)
    x = rng.normal(0, 3, (7, 70))
    q = ff.quantized(x)
    assert np.array_equal(ff.quantized(q), q) or np.all(np.abs(ff.quantized(q) - q) <= 0)
    bad = x.copy()
    bad[2, 33], bad[4, 5] = np.nan, np.inf
    q = ff.quantized(bad)
    assert np.isnan(q[2, 32:64]).all() and np.isnan(q[4, :32]).all() and np.isfinite(q[3]).all()


def test_uncertain_codes_are_found():
    rng = np.random.default_rng(2)
    h = rng.normal(0, 1, (20, 64))
    e = np.full_like(h, 1e-3)
    q, off = ff.quantized_within(h, e)
    seen = 0
    for _ in range(30):
        moved = ff.quantized(h + rng.uniform(-1, 1, h.shape) * e)
        assert np.all(np.abs(moved - q) <= off)
        seen += int((moved != q).sum())
    assert seen > 0 and (off > 0).mean() < 0.05


@pytest.mark.parametrize("mistake", ["halves", "tail", "rounding", "transposed"])
def test_a_planted_mistake_is_outside_the_bounds(mistake):
    rng = np.random.default_rng(5)
    x, w_in, w_down = _layer("silu", rng, 16, 64, 40)
    y, bound, spread, _, _ = ff.forward("silu", x, w_in, w_down, "bf16")
    if mistake == "halves":
        wrong = ff.forward("silu", x, np.concatenate([w_in[40:], w_in[:40]]), w_down, "bf16")[0]
    elif mistake == "tail":
        wrong = ff.forward("silu", x[:, :56], w_in[:, :56], w_down, "bf16")[0]
    elif mistake == "rounding":
        h = ff.hidden("silu", x, w_in)[2]
        wrong = (np.round(h * 32) / 32) @ w_down.T
    else:
        wrong = ff.forward("silu", x, w_in, w_down[:, ::-1], "bf16")[0]
    assert np.linalg.norm(wrong - y) > ff.norm_bound(y, spread, "bf16")
