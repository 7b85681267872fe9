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
