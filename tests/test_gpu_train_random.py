"""Seeded random shapes, types, shifts and live counts through every training
operator, against fp64 (needs an MI355X)."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import TYPES, close, live_tensor, placed, untouched, guarded, values

pytestmark = pytest.mark.gpu
Z = float(np.float32(1.6448536))


def _shape(rng, most_d, most):
    d = int(np.exp(rng.uniform(0, np.log(most_d + 1))))
    if rng.random() < 0.5:                      # near a multiple of 128, where blocks and octets end
        d = max(1, d // 128 * 128 + int(rng.integers(-9, 10)))
    d = max(1, min(d, most_d))
    rows = max(1, min(int(np.exp(rng.uniform(0, np.log(600)))), most // d))
    live = None if rng.random() < 0.6 else int(rng.integers(-1, rows + 2))
    return rows, d, live, (rows if live is None else max(0, min(live, rows))), int(rng.integers(0, 4))


@pytest.mark.parametrize("seed", range(60))
def test_activations(seed):
    rng = np.random.default_rng(1000 + seed)
    dtype = ["bf16", "fp16", "fp32"][seed % 3]
    act = ["silu", "gelu_tanh", "gelu", "squared_relu", "gelu_sparse", "gelu_sparse"][seed % 6]
    rows, d, live, n, offset = _shape(rng, 65536 if act == "gelu_sparse" else 9000, 200000)
    print(f"random {act} {dtype} {rows}x{d} live {live} offset {offset}", flush=True)
    h, sparse = ref.halves(act), act == "gelu_sparse"
    x, xe = values(rng, (rows, h * d), dtype, mean=rng.normal(), std=1.2)
    dout, de = values(rng, (rows, d), dtype)
    xg, dg, lv = placed(x, offset), placed(dout, offset), live_tensor(live)
    _, out = guarded((rows, d), TYPES[dtype], offset)
    out, c = ga.activation_checkpoint(xg, act, z=Z, live_rows=lv, out=out)
    _, wx = guarded((rows, h * d), TYPES[dtype], offset)
    ga.activation_backward(dg, xg, act, z=Z, live_rows=lv, out=wx)
    _, dx = guarded((rows, h * d), TYPES[dtype], offset)
    ga.activation_backward(dg, c, act, z=Z, live_rows=lv, out=dx)
    torch.cuda.synchronize()
    for t in (out, wx, dx):
        untouched(t, n, act)
    if n == 0:
        return
    xe, de = xe[:n], de[:n]
    want, bound = ref.forward(act, xe, dtype, Z)
    close(out[:n], want, bound, "out")
    v = ref.decode(c.codes[:n].cpu().numpy(), c.scales[:n].cpu().numpy())
    if sparse:
        t, _, std = ref.over_cutoff(xe[:, :d], Z)
        want, bound = ref.sparse_backward(de, t, std, xe[:, d:], Z, dtype)
        close(wx[:n], want, bound, "dx from x")
        assert np.array_equal(c.codes[:n, 0].cpu().numpy() > 0, t > 0)
        s32 = c.stats[:n, 1:].double().cpu().numpy()
        want, bound = ref.sparse_backward(de, v[:, 0], s32, v[:, 1], Z, dtype)
        slack = 4 * ref.U * np.tile(np.abs(de), (1, 2)) * (1 + np.abs(v[:, 0]).max()) * (2 + np.abs(v[:, 1]).max())
    else:
        want, bound = ref.backward(act, de, (xe,) if h == 1 else (xe[:, :d], xe[:, d:]), dtype)
        close(wx[:n], want, bound, "dx from x")
        v = v.reshape(n, h * d)
        want, bound = ref.backward(act, de, (v,) if h == 1 else (v[:, :d], v[:, d:]), dtype)
        slack = 4 * ref.U * np.tile(np.abs(de), (1, h)) * (1 + np.abs(v)) * (2 + np.abs(np.tile(v[:, -d:], (1, h))))
    close(dx[:n], want, bound + slack, "dx from codes")


@pytest.mark.parametrize("seed", range(60))
def test_layer_norm(seed):
    rng = np.random.default_rng(2000 + seed)
    dtype = ["bf16", "fp16", "fp32"][seed % 3]
    wdtype = "fp32" if seed % 2 else dtype
    rows, d, live, n, offset = _shape(rng, 32768, 300000)
    d = max(d, 2)
    print(f"random layer norm {dtype} {wdtype} {rows}x{d} live {live} offset {offset}", flush=True)
    x, xe = values(rng, (rows, d), dtype, mean=rng.normal(), std=2.0)
    dy, de = values(rng, (rows, d), dtype)
    w, we = values(rng, (d,), wdtype, mean=1.0, std=0.3)
    b, be = values(rng, (d,), wdtype, std=0.3)
    xg, dg, wg, bg, lv = placed(x, offset), placed(dy, offset), placed(w, offset), placed(b, offset), live_tensor(live)
    _, y = guarded((rows, d), TYPES[dtype], offset)
    _, c = ga.layer_norm_checkpoint(xg, wg, bg, live_rows=lv, out=y)
    _, dx = guarded((rows, d), TYPES[dtype], offset)
    _, dw, db = ga.layer_norm_backward(dg, xg, wg, stats=c.stats, live_rows=lv, out=dx)
    _, kx = guarded((rows, d), TYPES[dtype], offset)
    _, kw, kb = ga.layer_norm_backward(dg, c, wg, live_rows=lv, out=kx)
    back = ga.checkpoint_restore(c, torch.float32, live_rows=lv)
    torch.cuda.synchronize()
    for t in (y, dx, kx):
        untouched(t, n, "layer norm")
    if n == 0:
        assert float(dw.abs().max()) == 0 and float(kb.abs().max()) == 0
        return
    xe, de = xe[:n], de[:n]
    want, bound, mean, rstd = ref.layer_norm(xe, we, be, 1e-5, dtype)
    # a row of few values may have next to no spread: its x - mean is rounded against the values themselves
    bound = bound + 4 * ref.U * np.abs(rstd * we) * np.abs(xe).max(1, keepdims=True) * (d < 64)
    close(y[:n], want, bound, "y")
    s = c.stats[:n].double().cpu().numpy()
    v = ref.decode(c.codes[:n].cpu().numpy(), c.scales[:n].cpu().numpy())
    for got, nv, what in (((dx[:n], dw, db), (xe - s[:, :1]) * s[:, 1:], "x"), ((kx[:n], kw, kb), v * s[:, 1:], "codes")):
        grads, bounds = ref.layer_norm_backward(de, nv, s[:, 1:], we, dtype, wdtype, 32)
        # x - mean loses the mean's own rounding where they nearly cancel
        loss = 2 * ref.U * np.abs(s[:, :1]) * s[:, 1:]
        extra = (s[:, 1:] * np.abs(we) * (np.abs(nv) + 1) * (np.abs(de).max() + 1) * loss * 4,
                 (np.abs(de) * loss).sum(0), 0.0)
        for g, wv, bv, ev, name in zip(got, grads, bounds, extra, ("dx", "dw", "db")):
            close(g, wv, bv + (ev if what == "x" else 0.0), f"{name} from {what}")
    want = v + s[:, :1]
    close(back[:n], want, 3 * ref.U * (np.abs(v) + np.abs(s[:, :1]) + np.abs(want)), "restored")
    top = np.repeat(c.scales[:n].double().cpu().numpy(), ref.BLOCK, axis=1)[:, :d]
    close(back[:n], xe, top * (0.5 + 1e-4) + 4 * ref.U * (np.abs(v) + np.abs(s[:, :1])), "restored against x")


@pytest.mark.parametrize("seed", range(40))
def test_balance(seed):
    rng = np.random.default_rng(3000 + seed)
    dtype = ["bf16", "fp16", "fp32"][seed % 3]
    experts = max(1, int(np.exp(rng.uniform(0, np.log(1025)))))
    rows = max(1, min(int(np.exp(rng.uniform(0, np.log(20000)))), 400000 // experts))
    k = int(rng.integers(1, 9))
    print(f"random balance {dtype} {rows}x{experts} k{k}", flush=True)
    logits, le = values(rng, (rows, experts), dtype, std=2.0)
    index = rng.integers(-1, experts + 1, (rows, k))
    mask = rng.random(rows) < 0.8
    live = None if seed % 2 else int(rng.integers(0, rows + 1))
    use = mask & (np.arange(rows) < (rows if live is None else live))
    lg, ig, mg, lv = logits.cuda(), torch.from_numpy(index).cuda(), torch.from_numpy(mask).cuda(), live_tensor(live)
    b = ga.balance_loss(lg, ig, 0.5, mask=mg, live_rows=lv)
    scale = 1e4 if dtype == "fp16" else 1.0
    _, out = guarded((rows, experts), TYPES[dtype])
    ga.balance_loss_backward(lg, b, dloss=torch.tensor(scale, device="cuda"), mask=mg, live_rows=lv, out=out)
    torch.cuda.synchronize()
    loss, bound, counts, offsets, n = ref.balance(le, index, 0.5, use)
    assert np.array_equal(b.counts.cpu().numpy(), counts) and np.array_equal(b.offsets.cpu().numpy(), offsets)
    assert int(b.tokens) == n and abs(float(b.loss) - loss) <= bound + 1e-12
    want, gb = ref.balance_backward(le, counts, k, 0.5, n, use, scale, dtype)
    m = rows if live is None else live
    close(out[:m], want[:m], gb[:m], "dlogits")
    untouched(out, m, "balance")
