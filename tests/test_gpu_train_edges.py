"""Training operators at the edges of what their formats hold: blocks without a
finite scale, values next to the cutoff, means far above the spread, multipliers
and spreads far out, probabilities next to one (needs an MI355X)."""
import math

import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import TYPES, close, values

pytestmark = pytest.mark.gpu
Z = float(np.float32(1.6448536))


# ---- blocks without a finite scale ------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [300, 2048, 9000])
def test_a_gate_block_past_the_codes_reaches_the_rows_sum(d, dtype):
    """One finite gate value of 1e38: gate - cutoff is past 2^126, so its block has no finite scale, while the
    row's statistics do.  That value's share of the row's sum is in every dgate: all of them are NaN."""
    x = torch.randn(3, 2 * d, generator=torch.Generator().manual_seed(8)).to(TYPES[dtype])
    x[1, 130] = 1e38
    dout = torch.ones(3, d, dtype=TYPES[dtype])
    t, _, std = ref.over_cutoff(x[:, :d].double().numpy(), Z)
    assert t[1, 130] > 2.0 ** 126 and np.isfinite(std).all() and (t[1] > 0).sum() == 1
    _, c = ga.activation_checkpoint(x.cuda(), "gelu_sparse", z=Z)
    dx = ga.activation_backward(dout.cuda(), c, "gelu_sparse", z=Z).float().cpu().numpy().reshape(3, 2, d)
    assert torch.isfinite(c.stats).all() and int(torch.isnan(c.scales).sum()) == 1
    nan = np.isnan(dx)
    assert nan[1, 0].all() and not nan[[0, 2]].any()
    assert nan[1, 1, 128:256].all() and nan[1, 1].sum() == 128


def test_an_up_block_past_the_codes_counts_where_the_gate_passes():
    """An up block without a finite scale: NaN through the row's sum where one of its gates is above the cutoff;
    nothing where none is (a value at or below the cutoff has no gradient, whatever its up is)."""
    d = 300
    x = torch.randn(2, 2 * d, generator=torch.Generator().manual_seed(9))
    x[:, 128:256] = -3.0
    x[1, 200] = 6.0
    x[:, d + 130] = float("inf")
    _, c = ga.activation_checkpoint(x.cuda(), "gelu_sparse", z=Z)
    dx = ga.activation_backward(torch.ones(2, d, device="cuda"), c, "gelu_sparse", z=Z).cpu().numpy().reshape(2, 2, d)
    assert np.isfinite(dx[0]).all() and (dx[0, 0] != 0).any()
    assert np.isnan(dx[1, 0]).all() and np.isfinite(dx[1, 1]).all()


# ---- the cutoff's side -------------------------------------------------------------

@pytest.mark.parametrize("above", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [400, 4096, 16384])
def test_the_cutoffs_side_where_the_sampled_values_are_far_out(d, dtype, above):
    """First, middle and last value 60000, the others 0.00146, four values of 100 and a multiplier that puts the
    cutoff 7e-4 past them or short of them: differences to 60000 in fp32 would move the mean by 1.4e-3."""
    x = torch.full((1, 2 * d), 1.0)
    x[0, :d] = 0.00146
    at = [9, 77, d // 2 + 30, d - 20]
    x[0, at] = 100.0
    x[0, [0, d // 2, d - 1]] = 60000.0
    x = x.to(TYPES[dtype])
    g = x[0, :d].double().numpy()
    mean = math.fsum(g) / d
    std = math.sqrt(math.fsum((g - mean) ** 2) / d)
    z = float(np.float32((g[9] + (-7e-4 if above else 7e-4) - mean) / std))
    # an fp32 multiplier puts the cutoff within 2^-24 |z| s <= 2.1e-5 of that
    assert 6.7e-4 < abs(g[9] - (mean + z * std)) < 7.3e-4 and (g[9] > mean + z * std) == above
    xg, dg = x.cuda(), torch.ones(1, d, dtype=TYPES[dtype], device="cuda")
    out, c = ga.activation_checkpoint(xg, "gelu_sparse", z=z)
    dx = ga.activation_backward(dg, c, "gelu_sparse", z=z)
    wx = ga.activation_backward(dg, xg, "gelu_sparse", z=z)
    torch.cuda.synchronize()
    on = np.zeros(d, bool)
    on[[0, d // 2, d - 1] + (at if above else [])] = True
    assert np.array_equal((c.codes[0, 0] > 0).cpu().numpy(), on)
    assert np.array_equal((out[0] > 0).cpu().numpy(), on)
    for v in (dx, wx):   # dup = gelu(max(t, 0))
        assert np.array_equal((v[0, d:] > 0).cpu().numpy(), on)
    y, st = ga.layer_norm(xg[:, :d].contiguous(), torch.ones(d, device="cuda"))
    torch.cuda.synchronize()
    assert abs(float(st[0, 0]) - mean) <= 2 * ref.U * mean


# ---- layer norm: a mean far above the spread ------------------------------------------

def _offset_rows(rng, rows, d, dtype, mean, spread):
    if spread is not None:
        return values(rng, (rows, d), dtype, mean=mean, std=spread)
    x = torch.ones(rows, d, dtype=TYPES[dtype])            # one step of the type in one place of each row
    x[torch.arange(rows), torch.from_numpy(rng.integers(0, d, rows))] += 2 * ref.HALF_EPS[dtype]
    return x, x.double().numpy()


@pytest.mark.parametrize("dtype,mean,spread", [("fp32", 65536.3, 1.0), ("fp32", -4096.1, 0.5), ("fp32", 300.7, 1.0),
                                               ("fp16", 1.0, None), ("bf16", 1.0, None)])
@pytest.mark.parametrize("rows,d", [(64, 5), (70, 100), (40, 500), (64, 1000), (33, 2000), (20, 4000), (12, 8192),
                                    (9, 20000)])
def test_backward_from_x_where_the_mean_is_far_above_the_spread(rows, d, dtype, mean, spread):
    """n is taken from the row's own mean, not from its rounding to fp32 in stats, which would add the same amount
    (up to 2^-25 of the mean, in spreads) to every n of a row: 3.75e-3 at mean 65536.3 and spread 1."""
    rng = np.random.default_rng(rows + d)
    x, xe = _offset_rows(rng, rows, d, dtype, mean, spread)
    dy, de = values(rng, (rows, d), dtype, mean=0.5)
    if dtype == "fp16":                                    # r is up to 3e4: dx fits the type
        dy = dy * 2.0 ** -4
        de = dy.double().numpy()
    w, we = values(rng, (d,), "fp32", mean=1.0, std=0.3)
    xg, wg = x.cuda(), w.cuda()
    _, st = ga.layer_norm(xg, wg, eps=1e-12)
    dx, dw, db = ga.layer_norm_backward(dy.cuda(), xg, wg, stats=st)
    torch.cuda.synchronize()
    r = st[:, 1:].double().cpu().numpy()
    t = xe - xe.mean(1, keepdims=True)
    assert (np.abs(xe.mean(1, keepdims=True) * r) > 16).all()
    (wx, ww, wb), bounds = ref.layer_norm_backward(de, t * r, r, we, dtype, "fp32", 32)
    # x - mean is exact or rounded by u of itself; the mean of those differences to the fp32 mean is the sum of d
    # terms of at most |t| + the mean's rounding (2 u of it), added 32 one after another and then by pairs
    off = 72 * ref.U * (np.abs(t) + 2 * ref.U * np.abs(xe)).mean(1, keepdims=True) * r + 2 * ref.U * np.abs(t) * r
    v = np.abs(de * we)
    extra = r * (off * (v * np.abs(t * r)).mean(1, keepdims=True) + np.abs(t * r) * (v * off).mean(1, keepdims=True))
    close(dx, wx, bounds[0] + extra, "dx")
    close(dw, ww, bounds[1] + (np.abs(de) * off).sum(0), "dw")
    close(db, wb, bounds[2], "db")


# ---- sparse GELU: multipliers and spreads far out -----------------------------------------

def _sparse_from_x(gate, up, dout, z, dtype):
    """dx from x with the statistics' term from gate - mean, and bounds that do not grow with z^2."""
    d = gate.shape[1]
    t, _, std = ref.over_cutoff(gate, z)
    f, df, bf, bdf = ref.activation("gelu_tanh", np.maximum(t, 0.0))
    on = t > 0
    # past 10 the sigmoid is 1 to 2^-120: f = t, f' = 1 but for the roundings of the products
    bf, bdf = np.where(t > 10, 4 * ref.U * np.abs(f), bf), np.where(t > 10, 4 * ref.U, bdf)
    moved = np.where(t > 10, 0.0, 2 * ref.U * np.abs(t))  # what t's own rounding does to f'
    q = np.where(on, dout * up * df, 0.0)
    bq = np.where(on, np.abs(dout * up) * (bdf + 3 * ref.U * np.abs(df) + moved), 0.0)
    total = q.sum(1, keepdims=True)
    btotal = bq.sum(1, keepdims=True) + 90 * ref.U * np.abs(q).sum(1, keepdims=True)
    n = (gate - gate.mean(1, keepdims=True)) / std
    size = 1.0 + np.abs(z * n)
    dg = q - total / d * (1.0 + z * n)
    bg = bq + (btotal / d + np.abs(total) / d * 8 * ref.U) * size + 2 * ref.U * np.abs(q)
    du = dout * f
    bu = np.abs(dout) * (bf + 2 * ref.U * np.abs(f) + 2 * ref.U * np.abs(df * t) * on)
    return (np.concatenate([dg, du], 1),
            np.concatenate([bg + ref.rounding(dg, dtype), bu + ref.rounding(du, dtype)], 1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("z", [-1e4, -60.0, -3.0, 0.0])
@pytest.mark.parametrize("d", [5, 900, 6000, 16400])
def test_sparse_from_x_with_every_value_past_the_cutoff(d, z, dtype):
    """The term of the row's std is z times a normalised gate: its error grows with z, not with z^2 as where it is
    formed from gate - cutoff."""
    rng = np.random.default_rng(d)
    x, xe = values(rng, (3, 2 * d), dtype)
    dout, de = values(rng, (3, d), dtype, mean=0.5)
    z32 = float(np.float32(z))
    if dtype == "fp16" and z < -100.0:
        dout = dout * 2.0 ** -6                           # dup is dout times 1e4
        de = dout.double().numpy()
    wx = ga.activation_backward(dout.cuda(), x.cuda(), "gelu_sparse", z=z)
    torch.cuda.synchronize()
    want, bound = _sparse_from_x(xe[:, :d], xe[:, d:], de, z32, dtype)
    close(wx, want, bound, "dx from x")


@pytest.mark.parametrize("dtype,spread", [("fp32", 1e-37), ("fp32", 2.0 ** -133), ("bf16", 1e-37)])
def test_sparse_from_x_with_next_to_no_spread(dtype, spread):
    """z / std alone is past fp32's range times the row's sum; z n is not."""
    d = 700
    rng = np.random.default_rng(3)
    x, _ = values(rng, (3, 2 * d), "fp32")
    x[:, :d] *= spread
    x = x.to(TYPES[dtype])
    xe = x.double().numpy()
    dout, de = values(rng, (3, d), dtype, mean=900.0, std=9000.0)
    wx = ga.activation_backward(dout.cuda(), x.cuda(), "gelu_sparse", z=Z)
    torch.cuda.synchronize()
    want, bound = _sparse_from_x(xe[:, :d], xe[:, d:], de, Z, dtype)
    assert np.abs(want).max() < 1e7 and np.abs(want[:, :d]).max() > 1.0
    # gate - mean and gate - cutoff of subnormal numbers are rounded to a whole 2^-149
    low = 2.0 ** -148
    extra = np.abs(want).max() * 4 * Z * low / np.abs(xe[:, :d]).mean() + np.abs(np.tile(de, (1, 2))) * low
    close(wx, want, bound + extra, "dx from x")


@pytest.mark.parametrize("z", [-3.0, -1.0, 0.0, 0.5, 2.5])
@pytest.mark.parametrize("d", [900, 6000])
def test_sparse_from_codes_at_other_multipliers(d, z):
    """As at the usual multiplier: the formulas at the values that the codes stand for."""
    rng = np.random.default_rng(18)
    x, xe = values(rng, (4, 2 * d), "fp32")
    dout, de = values(rng, (4, d), "fp32", mean=0.3)
    z32 = float(np.float32(z))
    _, c = ga.activation_checkpoint(x.cuda(), "gelu_sparse", z=z)
    dx = ga.activation_backward(dout.cuda(), c, "gelu_sparse", z=z)
    torch.cuda.synchronize()
    v = ref.decode(c.codes.cpu().numpy(), c.scales.cpu().numpy())
    s32 = c.stats[:, 1:].double().cpu().numpy()
    want, bound = ref.sparse_backward(de, v[:, 0], s32, v[:, 1], z32, "fp32")
    # a restored value is rounded once in fp32: its slope may move by that much
    extra = 4 * ref.U * np.tile(np.abs(de), (1, 2)) * (1 + np.abs(v[:, 0]).max()) * (2 + np.abs(v[:, 1]).max())
    close(dx, want, bound + extra, "dx from codes")
    q = np.where(v[:, 0] > 0, de * v[:, 1] * ref.activation("gelu_tanh", np.maximum(v[:, 0], 0.0))[1], 0.0)
    assert (np.abs(q.sum(1)) / d * (1 + z * z) > 100 * bound[:, :d].mean(1)).any()   # the statistics' term shows


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [6, 700])
def test_sparse_from_x_with_a_cutoff_past_fp32(d, dtype):
    """Nothing is above it: no output and no gradient."""
    x = torch.randn(2, 2 * d, generator=torch.Generator().manual_seed(4)) * 50
    xg, z = x.to(TYPES[dtype]).cuda(), 3e38
    out, _ = ga.activation_checkpoint(xg, "gelu_sparse", z=z)
    wx = ga.activation_backward(torch.ones(2, d, dtype=TYPES[dtype], device="cuda"), xg, "gelu_sparse", z=z)
    torch.cuda.synchronize()
    assert float(out.abs().max()) == 0.0 and float(wx.abs().max()) == 0.0


# ---- balance loss: a probability next to one -------------------------------------------

@pytest.mark.parametrize("experts", [3, 8, 40, 128, 300, 1000])
def test_balance_gradient_where_one_probability_is_next_to_one(experts):
    """The gradient of a token whose router is (almost) sure is p (counts - their mean under p): small numbers, off
    by roundings of themselves and not of the counts."""
    rows, k = 96, 2
    rng = np.random.default_rng(experts)
    logits = rng.normal(0, 1, (rows, experts)).astype(np.float32)
    top = rng.integers(0, experts, rows)
    logits[np.arange(rows), top] = 6.0 + np.linspace(0, 20, rows, dtype=np.float32) + np.float32(math.log(experts))
    index = np.stack([top, np.minimum(rng.integers(0, experts, rows), experts // 3)], 1)
    b = ga.balance_loss(torch.from_numpy(logits).cuda(), torch.from_numpy(index).cuda())
    g = ga.balance_loss_backward(torch.from_numpy(logits).cuda(), b).double().cpu().numpy()
    le = logits.astype(np.float64)
    counts = np.bincount(index.reshape(-1), minlength=experts)
    p = ref.softmax(le)
    factor = experts / (k * rows * rows)
    # counts less their mean under p, without cancellation: sum_j p_j (counts_e - counts_j)
    apart = (counts[:, None] - counts[None, :]).astype(np.float64)
    off, size = p @ apart.T, p @ np.abs(apart)
    rel = ref.relative_softmax(le)
    # p's own errors, those of the p_j in the mean and of a sum of up to 1024 terms, relative to the counts'
    # distances from their mean; a first mean that is off by as much of the largest count counts twice so small
    most = 2 * rel + 64 * ref.U
    bound = factor * (p * (size * most + (counts.max() + 1) * most ** 2)) + 2.0 ** -149
    close(torch.from_numpy(g), factor * p * off, bound, "dlogits")


# ---- what a Checkpoint is of ---------------------------------------------------------------

def test_a_checkpoint_knows_its_activation_and_multiplier():
    """The backward pass takes the forward's z from it, and refuses another z or activation."""
    x = torch.randn(6, 2 * 300, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    dout = torch.ones(6, 300, device="cuda")
    _, c = ga.activation_checkpoint(x, "gelu_sparse", z=0.5)
    assert c.activation == "gelu_sparse" and c.z == 0.5
    codes, scales, stats = c                                                           # a tuple of three
    want = ga.activation_backward(dout, ga.Checkpoint(codes, scales, stats), "gelu_sparse", z=0.5)  # of tensors alone
    moved = c._replace(codes=codes.cpu().cuda())
    assert moved.z == 0.5 and torch.equal(ga.activation_backward(dout, moved, "gelu_sparse"), want)
    for z in (None, 0.5, np.float32(0.5)):
        assert torch.equal(ga.activation_backward(dout, c, "gelu_sparse", z=z), want)
    assert torch.equal(ga.activation_backward(dout, c, "gelu_sparse"), want)
    with pytest.raises(ValueError):
        ga.activation_backward(dout, c, "gelu_sparse", z=ga.Z_SPARSITY_095)
    _, s = ga.activation_checkpoint(x, "silu")
    assert s.activation == "silu" and s.z is None
    for act in ("gelu", "gelu_tanh"):
        with pytest.raises(ValueError):
            ga.activation_backward(dout, s, act)
    assert torch.equal(ga.activation_backward(dout, s, "silu", z=0.1), ga.activation_backward(dout, s, "silu"))
    # written into another's tensors it is its own
    _, again = ga.activation_checkpoint(x, "gelu", checkpoint=s)
    assert again.activation == "gelu" and again.codes is s.codes
    ga.activation_backward(dout, again, "gelu")
    # from x and from tensors alone the default z is activation_checkpoint's
    _, c = ga.activation_checkpoint(x, "gelu_sparse")
    assert torch.equal(ga.activation_backward(dout, ga.Checkpoint(*c), "gelu_sparse"),
                       ga.activation_backward(dout, c, "gelu_sparse"))
    assert torch.equal(ga.activation_backward(dout, x, "gelu_sparse"),
                       ga.activation_backward(dout, x, "gelu_sparse", z=ga.Z_SPARSITY_095))
    # codes stored by themselves are of no activation
    r = torch.randn(4, 40, device="cuda")
    kept = ga.checkpoint_store(r)
    assert kept.activation is None
    ga.activation_backward(torch.ones_like(r), kept, "squared_relu")
    torch.cuda.synchronize()
