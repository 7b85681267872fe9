"""Layer norm and its backward pass on the GPU against fp64 (needs an MI355X)."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import PAD, TYPES, check_guard, close, guarded, live_tensor, placed, untouched, values

pytestmark = pytest.mark.gpu
EPS = 1e-5
# every width at which another kernel takes over, and odd ones; rows, d, shift, live
SHAPES = [(1, 1, 0, None), (1, 7, 0, None), (5, 64, 0, None), (67, 128, 0, 50), (3, 129, 1, None), (70, 512, 0, 0),
          (9, 513, 0, None), (300, 777, 1, None), (20, 1024, 0, 19), (18, 1025, 0, None), (2100, 2048, 0, None),
          (5, 2049, 3, None), (9, 4096, 0, 300), (4, 4097, 0, None), (3, 8192, 0, None), (2, 8200, 0, None),
          (1, 16384, 0, None), (3, 16385, 0, 2), (2, 32767, 1, None), (3, 32768, 0, None)]


def _case(rows, d, dtype, wide, seed):
    rng = np.random.default_rng(seed)
    wdtype = "fp32" if wide else dtype
    x, xe = values(rng, (rows, d), dtype, mean=0.7, std=2.0)
    dy, de = values(rng, (rows, d), dtype)
    w, we = values(rng, (d,), wdtype, mean=1.0, std=0.3)
    b, be = values(rng, (d,), wdtype, std=0.3)
    return x, xe, dy, de, w, we, b, be, wdtype


@pytest.mark.parametrize("dtype,wide", [("bf16", False), ("bf16", True), ("fp16", False), ("fp16", True), ("fp32", True)])
@pytest.mark.parametrize("rows,d,offset,live", SHAPES)
def test_forward_and_backward(dtype, wide, rows, d, offset, live):
    label = f"layer norm {dtype} wide {wide} {rows}x{d} live {live}"
    print(label, flush=True)
    x, xe, dy, de, w, we, b, be, wdtype = _case(rows, d, dtype, wide, rows + 11 * d)
    n = rows if live is None else min(live, rows)
    xg, dg, lv = placed(x, offset), placed(dy, offset), live_tensor(live)
    wg, bg = placed(w, offset), placed(b, offset)
    y_buf, y = guarded((rows, d), TYPES[dtype], offset)
    st_buf, st = guarded((rows, 2), torch.float32)
    ga.layer_norm(xg, wg, bg, eps=EPS, live_rows=lv, out=y, stats=st)
    k_buf, k = guarded((rows, d), torch.int8, offset)
    s_buf, s = guarded((rows, ref.blocks(d)), torch.float32)
    st2 = torch.full((rows, 2), PAD, dtype=torch.float32, device="cuda")
    y2, c = ga.layer_norm_checkpoint(xg, wg, None, eps=EPS, live_rows=lv, checkpoint=ga.Checkpoint(k, s, st2))
    dx_buf, dx = guarded((rows, d), TYPES[dtype], offset)
    _, dw, db = ga.layer_norm_backward(dg, xg, wg, stats=st, live_rows=lv, out=dx)
    kx_buf, kx = guarded((rows, d), TYPES[dtype], offset)
    _, kw, kb = ga.layer_norm_backward(dg, c, wg, live_rows=lv, out=kx, bias=rows % 2 == 0)
    torch.cuda.synchronize()
    for t in (y, st, k, s, st2, dx, kx):
        untouched(t, n, label)
    for buf, t, o in ((y_buf, y, offset), (st_buf, st, 0), (k_buf, k, offset), (s_buf, s, 0), (dx_buf, dx, offset),
                      (kx_buf, kx, offset)):
        check_guard(buf, t.numel(), o)
    assert dw.dtype == TYPES[wdtype] and (kb is None) == (rows % 2 == 1)
    if n == 0:
        for g in (dw, db, kw) + ((kb,) if kb is not None else ()):
            assert float(g.abs().max()) == 0.0
        return
    xe, de = xe[:n], de[:n]
    want, bound, mean, rstd = ref.layer_norm(xe, we, be, EPS, dtype)
    close(y[:n], want, bound, label + " y")
    want, bound, _, _ = ref.layer_norm(xe, we, np.zeros(d), EPS, dtype)
    close(y2[:n], want, bound, label + " y without bias")
    both = np.concatenate([mean, rstd], 1)
    # the mean's fp64 sum is exact to 2^-50 of the values, the rest is the rounding to fp32
    close(st[:n], both, 2 * ref.U * np.abs(both) + 1e-14, label + " stats")
    assert torch.equal(st[:n], st2[:n])
    t32 = (xe - mean).astype(np.float32).astype(np.float64)
    wc, ws, q = ref.encode(t32)
    # fp64 means may differ in their last bits; 16-bit rows form x - mean in two fp32 roundings and the
    # quotient in fp32: 2 u of x - mean (and of the block's largest) and 2^-22 of the quotient, up to 127
    near = np.abs(np.abs(q - np.rint(q)) - 0.5) < (1e-6 if dtype == "fp32" else 127 * (2 * 2 * ref.U + 2.0 ** -22) + 1e-6)
    got = k[:n].cpu().numpy()
    assert np.array_equal(got[~near], wc[~near]) and (np.abs(got.astype(int) - wc) <= 1).all(), label
    close(s[:n], ws, 5 * ref.U * ws + 1e-14, label + " scales")
    # terms a lane adds in a row's sums: 8 an octet, at most 4 octets
    st64 = st[:n].double().cpu().numpy()
    grads, bounds = ref.layer_norm_backward(de, (xe - st64[:, :1]) * st64[:, 1:], st64[:, 1:], we, dtype, wdtype, 32)
    for g, wv, bv, what in zip((dx[:n], dw, db), grads, bounds, ("dx", "dw", "db")):
        close(g, wv, bv, f"{label} {what}")
    v = ref.decode(got, s[:n].cpu().numpy())
    grads, bounds = ref.layer_norm_backward(de, v * st64[:, 1:], st64[:, 1:], we, dtype, wdtype, 32)
    close(kx[:n], grads[0], bounds[0], label + " dx from codes")
    close(kw, grads[1], bounds[1], label + " dw from codes")
    if kb is not None:
        close(kb, grads[2], bounds[2], label + " db from codes")


@pytest.mark.parametrize("rows,d", [(5000, 128), (9000, 96), (3000, 512), (2500, 1000), (700, 4096), (600, 8192),
                                    (400, 16384), (300, 20000)])
def test_many_rows_add_up_and_repeat(rows, d):
    """Rows over every workgroup and several turns of it; the same bits every time."""
    print(f"many rows {rows}x{d}", flush=True)
    x, xe, dy, de, w, we, _, _, _ = _case(rows, d, "bf16", True, d)
    xg, dg, wg = x.cuda(), dy.cuda(), w.cuda()
    _, st = ga.layer_norm(xg, wg)
    first = ga.layer_norm_backward(dg, xg, wg, stats=st)
    ws = torch.full((max(1, ga.layer_norm_backward_workspace_bytes(rows, d)),), 255, dtype=torch.uint8, device="cuda")
    again = ga.layer_norm_backward(dg, xg, wg, stats=st, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    s = st.double().cpu().numpy()
    grads, bounds = ref.layer_norm_backward(de, (xe - s[:, :1]) * s[:, 1:], s[:, 1:], we, "bf16", "fp32", 32)
    for g, wv, bv, what in zip(first, grads, bounds, ("dx", "dw", "db")):
        close(g, wv, bv, f"{rows}x{d} {what}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_offset_and_constant_rows(dtype):
    """A mean far above the spread costs nothing beyond the inputs' own rounding; a constant row is exact."""
    d = 1000
    rng = np.random.default_rng(4)
    x = rng.normal(0, 1, (4, d)).astype(np.float32) + np.float32([[0], [4096], [-65536], [0]])
    x[3] = 0.1
    t = torch.from_numpy(x).to(TYPES[dtype])
    xe = t.double().numpy()
    w = torch.ones(d, dtype=TYPES[dtype], device="cuda")
    y, st = ga.layer_norm(t.cuda(), w)
    torch.cuda.synchronize()
    want, bound, _, _ = ref.layer_norm(xe, np.ones(d), np.zeros(d), EPS, dtype)
    assert (y[3] == 0).all() and float(st[3, 0]) == float(t[3, 0])
    close(y[:3], want[:3], bound[:3], "offset rows")


def test_gradient_against_differences():
    """The kernel's own forward pass, differenced along random directions in fp32."""
    rows, d, h = 6, 64, 2.0 ** -6
    x, xe, dy, de, w, we, b, be, _ = _case(rows, d, "fp32", True, 5)
    xg, dg, wg, bg = x.cuda(), dy.cuda(), w.cuda(), b.cuda()
    _, st = ga.layer_norm(xg, wg, bg)
    dx, dw, db = (g.double().cpu().numpy() for g in ga.layer_norm_backward(dg, xg, wg, stats=st))
    rng = np.random.default_rng(6)
    for _ in range(4):
        v = rng.normal(0, 1, (rows, d)).astype(np.float32)
        vg = torch.from_numpy(v).cuda()
        plus, minus = ga.layer_norm(xg + h * vg, wg, bg)[0], ga.layer_norm(xg - h * vg, wg, bg)[0]
        moved = ((plus.double() - minus.double()).cpu().numpy() * de).sum() / (2 * h)
        # the third derivative is O(1 / spread^3): h^2 / 6 of it, and 2 U / h a value for the fp32 differences
        slack = np.abs(de).sum() * (h * h + 16 * ref.U / h)
        assert abs((dx * v).sum() - moved) <= slack
        assert abs((dw * v[0]).sum() - (((ga.layer_norm(xg, wg + h * vg[0], bg)[0].double()
                                          - ga.layer_norm(xg, wg - h * vg[0], bg)[0].double()).cpu().numpy() * de).sum()
                                        / (2 * h))) <= np.abs(de).sum() * 32 * ref.U / h


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_with_one_value_far_out(dtype):
    """A first value 3000 spreads out: the statistics of the rest do not suffer."""
    d = 4096
    rng = np.random.default_rng(11)
    x = rng.normal(0, 1, (3, d)).astype(np.float32)
    x[0, 0], x[1, d // 2], x[2, d - 1] = 3000.0, -3000.0, 3000.0
    t = torch.from_numpy(x).to(TYPES[dtype])
    y, st = ga.layer_norm(t.cuda(), torch.ones(d, device="cuda"))
    torch.cuda.synchronize()
    want, bound, mean, rstd = ref.layer_norm(t.double().numpy(), np.ones(d), np.zeros(d), EPS, dtype)
    # differences to the pivot and their sums of eight: 2^-24 of 3000 in one octet of 512, of 8 elsewhere
    moved = (3000.0 / 512 + 8.0) * 2.0 ** -24
    close(st[:, :1], mean, 2 * ref.U * np.abs(mean) + moved, "mean")
    close(st[:, 1:], rstd, 4 * ref.U * rstd, "rstd")
    close(y, want, bound + rstd * moved, "y")
