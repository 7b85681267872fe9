"""Activation checkpoints and the activations' training pair on the GPU against
fp64 (needs an MI355X): codes exactly, values and gradients within the bounds
of train_ref."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import TYPES, check_guard, close, guarded, live_tensor, placed, untouched, values

pytestmark = pytest.mark.gpu
Z = float(np.float32(1.6448536))
ELEMENTWISE = ["silu", "gelu_tanh", "gelu", "squared_relu"]
# rows, d, elements the arrays are shifted by, live rows
SHAPES = [(1, 1, 0, None), (1, 8, 0, None), (3, 127, 1, None), (5, 128, 0, 4), (4, 129, 3, None), (7, 200, 0, 0),
          (33, 768, 0, 20), (2, 2048, 0, 99), (5, 4099, 1, None), (2, 16384, 0, 1)]


def _exact_codes(got, want, label):
    g = got.cpu().numpy()
    assert np.array_equal(g, want), f"{label}: {int((g != want).sum())} codes differ"


def _scales(got, want, label):
    """m / 127 in fp32: m (itself within 2 u where it is a difference), the constant and the product are rounded."""
    close(got, want, 4 * ref.U * np.nan_to_num(np.abs(want)), label)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,d,offset,live", SHAPES)
def test_store_and_restore(dtype, rows, d, offset, live):
    print(f"store {dtype} {rows}x{d}", flush=True)
    rng = np.random.default_rng(rows * 7 + d)
    x, xe = values(rng, (rows, d), dtype, std=3.0)
    n = rows if live is None else min(live, rows)
    codes_buf, codes = guarded((rows, d), torch.int8, offset)
    scales_buf, scales = guarded((rows, ref.blocks(d)), torch.float32)
    c = ga.checkpoint_store(placed(x, offset), live_rows=live_tensor(live), checkpoint=ga.Checkpoint(codes, scales))
    out_buf, out = guarded((rows, d), TYPES[dtype], offset)
    back = ga.checkpoint_restore(c, TYPES[dtype], live_rows=live_tensor(live), out=out)
    torch.cuda.synchronize()
    want, want_scales, _ = ref.encode(xe)
    _exact_codes(c.codes[:n], want[:n], f"store {dtype} {rows}x{d}")
    _scales(c.scales[:n], want_scales[:n], "scales")
    for t in (c.codes, c.scales, back):
        untouched(t, n, "store / restore")
    check_guard(codes_buf, rows * d, offset)
    check_guard(scales_buf, rows * ref.blocks(d))
    check_guard(out_buf, rows * d, offset)
    v = ref.decode(c.codes.cpu().numpy(), c.scales.cpu().numpy())[:n]
    close(back[:n], v, ref.U * np.abs(v) + ref.rounding(v, dtype), "restore")
    # half a code from the input, beside the roundings
    step = np.repeat(want_scales, ref.BLOCK, axis=1)[:n, :d]
    close(back[:n], xe[:n], step * 0.5 + 4 * ref.U * np.abs(v) + ref.rounding(v, dtype), "round trip")


def test_codes_at_ties():
    """Quotients that are half-integers, where a plain fp32 product may fall to either side."""
    rng = np.random.default_rng(3)
    top = np.float32([127.0, 127.0 * 0.75, 254.0 / 3.0, 1.27, 126.99999, 3.1e-5])
    x = np.zeros((6, 1024), np.float32)
    for r in range(6):
        h = rng.integers(-127, 127, 1024) + 0.5
        x[r] = (h * (float(top[r]) / 127.0)).astype(np.float32)
        x[r, ::128] = top[r]
    c = ga.checkpoint_store(torch.from_numpy(x).cuda())
    torch.cuda.synchronize()
    want, _, quotient = ref.encode(x.astype(np.float64))
    assert (np.abs(quotient - np.rint(quotient)) == 0.5).sum() > 900     # rows 0 and more are exact ties
    _exact_codes(c.codes, want, "ties")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unusual_blocks(dtype):
    x = np.ones((5, 400), np.float32)
    x[0] = 0.0
    x[1, 3], x[1, 390] = np.inf, -np.inf
    x[2, 200] = np.nan
    x[3, :128] = 2.0 ** -110
    x[4, 0], x[4, 128], x[4, 256] = 2.0 ** 126, 2.0 ** 125, -2.0 ** 127
    t = torch.from_numpy(x).to(TYPES[dtype])
    c = ga.checkpoint_store(t.cuda())
    back = ga.checkpoint_restore(c, TYPES[dtype])
    torch.cuda.synchronize()
    want, scales, _ = ref.encode(t.double().numpy())
    _exact_codes(c.codes, want, "unusual")
    _scales(c.scales, scales, "unusual scales")
    got = back.float().cpu().numpy()
    nan = np.isnan(got)
    assert nan[1, :128].all() and nan[1, 384:].all() and not nan[1, 128:384].any()
    assert nan[2, 128:256].all() and nan[4, :128].all() and not nan[4, 128:256].any() and nan[4, 256:384].all()
    assert (got[0] == 0).all() and (got[3, :128] == 0).all()


@pytest.mark.parametrize("d", [5, 400])
@pytest.mark.parametrize("bad", [np.inf, np.nan, 2.0 ** 126])
@pytest.mark.parametrize("act", ELEMENTWISE)
def test_backward_of_a_bad_block_is_nan(act, bad, d):
    """The gradients from a gate block whose scale is NaN are NaN, other blocks' are not."""
    h = ref.halves(act)
    x = torch.full((3, h * d), -1.0)
    x[1, min(d - 1, 130)] = float(bad)
    first, last = (0, d) if d <= 128 else (128, 256)
    dout = torch.ones(3, d)
    for dtype in (torch.bfloat16, torch.float32):
        _, c = ga.activation_checkpoint(x.to(dtype).cuda(), act)
        dx = ga.activation_backward(dout.to(dtype).cuda(), c, act).float().cpu().numpy()
        nan = np.isnan(dx).reshape(3, h, d)
        assert nan[1, :, first:last].all() and nan.sum() == h * (last - first), (act, bad, dtype)


@pytest.mark.parametrize("d", [300, 3000])
def test_sparse_backward_of_a_bad_block_is_nan(d):
    """A gate block whose scale is NaN: both halves' gradients of it, though nothing of it is above the cutoff."""
    x = torch.randn(3, 2 * d, generator=torch.Generator().manual_seed(5))
    dout = torch.ones(3, d)
    _, c = ga.activation_checkpoint(x.cuda(), "gelu_sparse", z=Z)
    c.scales[1, 0, 1] = float("nan")
    dx = ga.activation_backward(dout.cuda(), c, "gelu_sparse", z=Z).cpu().numpy().reshape(3, 2, d)
    nan = np.isnan(dx)
    assert nan[1, :, 128:256].all() and not nan[[0, 2]].any() and not nan[1, 1, 256:].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", ELEMENTWISE)
@pytest.mark.parametrize("rows,d,offset,live", SHAPES)
def test_forward_keeps_codes_and_backward(act, dtype, rows, d, offset, live):
    label = f"{act} {dtype} {rows}x{d} live {live}"
    print(label, flush=True)
    h = ref.halves(act)
    rng = np.random.default_rng(rows + 3 * d + len(act))
    x, xe = values(rng, (rows, h * d), dtype, std=1.5)
    dout, de = values(rng, (rows, d), dtype)
    n = rows if live is None else min(live, rows)
    lead = (rows, d) if h == 1 else (rows, 2, d)
    codes_buf, codes = guarded(lead, torch.int8, offset)
    scales_buf, scales = guarded(lead[:-1] + (ref.blocks(d),), torch.float32)
    out_buf, out = guarded((rows, d), TYPES[dtype], offset)
    xg, dg, lv = placed(x, offset), placed(dout, offset), live_tensor(live)
    out, c = ga.activation_checkpoint(xg, act, live_rows=lv, out=out, checkpoint=ga.Checkpoint(codes, scales))
    dx_buf, dx = guarded((rows, h * d), TYPES[dtype], offset)
    ga.activation_backward(dg, c, act, live_rows=lv, out=dx)
    wx_buf, wx = guarded((rows, h * d), TYPES[dtype], offset)
    ga.activation_backward(dg, xg, act, live_rows=lv, out=wx)
    torch.cuda.synchronize()
    for t in (out, codes, scales, dx, wx):
        untouched(t, n, label)
    for buf, t, o in ((codes_buf, codes, offset), (scales_buf, scales, 0), (out_buf, out, offset), (dx_buf, dx, offset),
                      (wx_buf, wx, offset)):
        check_guard(buf, t.numel(), o)
    xe, de = xe[:n], de[:n]
    want, bound = ref.forward(act, xe, dtype)
    close(out[:n], want, bound, label + " out")
    parts = (xe,) if h == 1 else (xe[:, :d], xe[:, d:])
    wc, ws, _ = ref.encode(xe.reshape((n,) + lead[1:]))
    _exact_codes(codes[:n], wc, label)
    _scales(scales[:n], ws, label + " scales")
    want, bound = ref.backward(act, de, parts, dtype)
    close(wx[:n], want, bound, label + " backward from x")
    v = ref.decode(codes[:n].cpu().numpy(), scales[:n].cpu().numpy()).reshape(n, h * d)
    parts = (v,) if h == 1 else (v[:, :d], v[:, d:])
    want, bound = ref.backward(act, de, parts, dtype)
    # a restored value is rounded once in fp32: its slope may move by that much
    extra = 4 * ref.U * np.tile(np.abs(de), (1, h)) * (1 + np.abs(v)) * (2 + np.abs(np.tile(v[:, -d:], (1, h))))
    close(dx[:n], want, bound + extra, label + " backward from codes")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,d,offset,live", [(1, 1, 0, None), (3, 2, 0, None), (4, 8, 0, None), (2, 127, 1, None),
                                                (9, 129, 0, 7), (5, 513, 3, None), (3, 1024, 0, 0), (6, 1025, 1, None),
                                                (2, 2048, 0, 99), (3, 4100, 0, None), (2, 8192, 0, None),
                                                (3, 16384, 0, 2), (2, 16385, 1, None), (2, 32769, 0, None),
                                                (2, 65536, 0, None)])
def test_sparse(dtype, rows, d, offset, live):
    label = f"sparse {dtype} {rows}x{d} live {live}"
    print(label, flush=True)
    rng = np.random.default_rng(rows + 5 * d)
    x, xe = values(rng, (rows, 2 * d), dtype, mean=0.5, std=1.5)
    dout, de = values(rng, (rows, d), dtype)
    n = rows if live is None else min(live, rows)
    codes_buf, codes = guarded((rows, 2, d), torch.int8, offset)
    scales_buf, scales = guarded((rows, 2, ref.blocks(d)), torch.float32)
    stats_buf, stats = guarded((rows, 2), torch.float32)
    out_buf, out = guarded((rows, d), TYPES[dtype], offset)
    xg, dg, lv = placed(x, offset), placed(dout, offset), live_tensor(live)
    out, c = ga.activation_checkpoint(xg, "gelu_sparse", z=Z, live_rows=lv, out=out,
                                      checkpoint=ga.Checkpoint(codes, scales, stats))
    dx_buf, dx = guarded((rows, 2 * d), TYPES[dtype], offset)
    ga.activation_backward(dg, c, "gelu_sparse", z=Z, live_rows=lv, out=dx)
    wx_buf, wx = guarded((rows, 2 * d), TYPES[dtype], offset)
    ga.activation_backward(dg, xg, "gelu_sparse", z=Z, live_rows=lv, out=wx)
    back = ga.checkpoint_restore(c, torch.float32, live_rows=lv)
    torch.cuda.synchronize()
    for t in (out, codes, scales, stats, dx, wx):
        untouched(t, n, label)
    for buf, t, o in ((codes_buf, codes, offset), (scales_buf, scales, 0), (stats_buf, stats, 0), (out_buf, out, offset),
                      (dx_buf, dx, offset), (wx_buf, wx, offset)):
        check_guard(buf, t.numel(), o)
    if n == 0:
        return
    xe, de = xe[:n], de[:n]
    gate, up = xe[:, :d], xe[:, d:]
    t, cutoff, std = ref.over_cutoff(gate, Z)
    want, bound = ref.forward("gelu_sparse", xe, dtype, Z)
    close(out[:n], want, bound, label + " out")
    close(stats[:n], np.concatenate([cutoff, std], 1), 2 * ref.U * np.abs(np.concatenate([cutoff, std], 1)), "stats")
    # t is held in fp32; the two fp64 statistics may differ in their last bits, so a quotient within
    # 1e-6 of a half-integer may fall to either side.  16-bit rows form t in two fp32 roundings and the
    # quotient in fp32: 2 u of t (and of the block's largest) and 2^-22 of the quotient, up to 127
    t32 = t.astype(np.float32).astype(np.float64)
    wt, st, qt = ref.encode(t32, positive=True)
    wu, su, _ = ref.encode(up)
    got = codes[:n].cpu().numpy()
    assert np.array_equal(got[:, 1], wu), label
    near = np.abs(np.abs(qt - np.rint(qt)) - 0.5) < (1e-6 if dtype == "fp32" else 127 * (2 * 2 * ref.U + 2.0 ** -22) + 1e-6)
    assert np.array_equal(got[:, 0][~near], wt[~near]) and (np.abs(got[:, 0].astype(int) - wt) <= 1).all(), label
    assert np.array_equal(got[:, 0] > 0, t32 > 0), label + ": the mask"
    _scales(scales[:n], np.stack([st, su], 1), label + " scales")
    want, bound = ref.sparse_backward(de, t, std, up, Z, dtype)
    close(wx[:n], want, bound, label + " backward from x")
    v = ref.decode(got, scales[:n].cpu().numpy())
    s32 = stats[:n, 1:].double().cpu().numpy()
    want, bound = ref.sparse_backward(de, v[:, 0], s32, v[:, 1], Z, dtype)
    extra = 4 * ref.U * np.tile(np.abs(de), (1, 2)) * (1 + np.abs(v[:, 0]).max()) * (2 + np.abs(v[:, 1]).max())
    close(dx[:n], want, bound + extra, label + " backward from codes")
    c32 = stats[:n, :1].double().cpu().numpy()
    want = np.concatenate([v[:, 0] + c32, v[:, 1]], 1)
    close(back[:n], want, 3 * ref.U * (np.abs(want) + np.abs(v[:, :1]).reshape(n, -1).max() + np.abs(c32)), label + " restore")


def test_sparse_rows_without_spread_or_finite_values():
    d = 300
    rng = np.random.default_rng(9)
    x = rng.normal(0, 1, (5, 2 * d)).astype(np.float32)
    x[0, :d] = 0.7300000190734863          # one repeated value: std 0, nothing above the cutoff
    x[1, :d] = 0.0
    x[2, 17] = np.nan
    x[3, 18] = np.inf
    dout = rng.normal(0, 1, (5, d)).astype(np.float32)
    xg, dg = torch.from_numpy(x).cuda(), torch.from_numpy(dout).cuda()
    out, c = ga.activation_checkpoint(xg, "gelu_sparse", z=Z)
    dx, wx = ga.activation_backward(dg, c, "gelu_sparse", z=Z), ga.activation_backward(dg, xg, "gelu_sparse", z=Z)
    torch.cuda.synchronize()
    stats = c.stats.cpu().numpy()
    assert stats[0, 1] == 0.0 and stats[0, 0] == np.float32(0.73) and stats[1, 1] == 0.0
    for g in (dx, wx):
        g = g.cpu().numpy()
        assert (g[:2] == 0).all()                                      # no value passes: no gradient
        assert np.isnan(g[2, :d]).all() and np.isnan(g[3, :d]).all()   # a row that is not finite shows
        assert np.isfinite(g[4]).all()
    # a negative multiplier with no spread: every value sits at its cutoff
    out, c = ga.activation_checkpoint(xg[:2], "gelu_sparse", z=-1.0)
    assert float(out.abs().max()) == 0.0


@pytest.mark.parametrize("z", [-3.0, 0.0, 8.0, 1e25])
def test_sparse_multipliers(z):
    """Every value past the cutoff, half of them, none (and a multiplier whose square fp32 cannot hold)."""
    rng = np.random.default_rng(17)
    x, xe = values(rng, (4, 2 * 900), "fp32")
    dout, de = values(rng, (4, 900), "fp32")
    z32 = float(np.float32(z))
    out, c = ga.activation_checkpoint(x.cuda(), "gelu_sparse", z=z)
    wx, dx = (ga.activation_backward(dout.cuda(), k, "gelu_sparse", z=z) for k in (x.cuda(), c))
    torch.cuda.synchronize()
    want, bound = ref.forward("gelu_sparse", xe, "fp32", z32)
    close(out, want, bound, "out")
    t, _, std = ref.over_cutoff(xe[:, :900], z32)
    assert z != -3.0 or (t > 0).mean() > 0.99
    want, bound = ref.sparse_backward(de, t, std, xe[:, 900:], z32, "fp32")
    close(wx, want, bound, "dx from x")
    if z >= 8.0:
        assert float(out.abs().max()) == 0.0 and float(wx.abs().max()) == 0.0 and float(dx.abs().max()) == 0.0


@pytest.mark.parametrize("act", ELEMENTWISE)
def test_gradient_against_differences(act):
    """The kernel's own forward pass, differenced along random directions in fp32."""
    rows, d, h, halves = 5, 96, 2.0 ** -6, ref.halves(act)
    rng = np.random.default_rng(21)
    x, xe = values(rng, (rows, halves * d), "fp32")
    dout, de = values(rng, (rows, d), "fp32")
    dx = ga.activation_backward(dout.cuda(), x.cuda(), act).double().cpu().numpy()
    for _ in range(4):
        v = np.sign(rng.normal(0, 1, x.shape)).astype(np.float32)
        plus, minus = (ga.activation_checkpoint(x.cuda() + s * h * torch.from_numpy(v).cuda(), act)[0].double() for s in (1, -1))
        moved = ((plus - minus).cpu().numpy() * de).sum() / (2 * h)
        # along +-1: third derivatives of f(gate) up below 2 + 3 |up| (h^2 / 6 of them; squared ReLU: a second
        # derivative that jumps by 2 where it passes zero within h), forward errors of 32 u of (1 + |x|)^2 over h
        size = (1 + np.abs(xe[:, :d])) * (1 + np.abs(xe[:, -d:]))
        slack = (np.abs(de) * (h * h * (2 + 3 * np.abs(xe[:, -d:])) + 32 * ref.U * size / h)).sum()
        slack += (np.abs(de) * h * 2 * (np.abs(xe) < h)).sum() if act == "squared_relu" else 0.0
        assert abs((dx * v).sum() - moved) <= slack


def test_many_rows_past_one_launch_of_blocks():
    """More blocks of 128 than rows: the numbering of a wide array of many rows, spot rows exactly."""
    rows, d = 70000, 257
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, d, device="cuda", generator=g).to(torch.bfloat16)
    c = ga.checkpoint_store(x)
    back = ga.checkpoint_restore(c, torch.bfloat16)
    pick = torch.tensor([0, 1, 4095, 65535, 65536, rows - 1], device="cuda")
    torch.cuda.synchronize()
    want, _, _ = ref.encode(x[pick].double().cpu().numpy())
    assert np.array_equal(c.codes[pick].cpu().numpy(), want)
    assert float((back.float() - x.float()).abs().max()) < 0.5 * 6.0 / 127 + 0.02
