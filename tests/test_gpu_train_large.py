"""The training operators on arrays past 2^32 elements (needs an MI355X): the
last rows, whose offsets do not fit 32 bits, against fp64."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import close

pytestmark = pytest.mark.gpu
Z = float(np.float32(1.6448536))


def _mostly_zero(rows, cols, last, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    t[-last:] = torch.randn(last, cols, device="cuda", generator=g).to(torch.bfloat16)
    return t


def test_checkpoint_and_sparse_backward():
    rows, d, last = 32780, 65536, 2                  # [rows, 2 d]: 4.3e9 elements
    print("large sparse", flush=True)
    x, dout = _mostly_zero(rows, 2 * d, last, 1), _mostly_zero(rows, d, last, 2)
    out, c = ga.activation_checkpoint(x, "gelu_sparse", z=Z)
    dx = ga.activation_backward(dout, x, "gelu_sparse", z=Z)
    torch.cuda.synchronize()
    xe, de = x[-last:].double().cpu().numpy(), dout[-last:].double().cpu().numpy()
    want, bound = ref.forward("gelu_sparse", xe, "bf16", Z)
    close(out[-last:], want, bound, "out")
    t, _, std = ref.over_cutoff(xe[:, :d], Z)
    want, bound = ref.sparse_backward(de, t, std, xe[:, d:], Z, "bf16")
    close(dx[-last:], want, bound, "dx")
    assert np.array_equal(c.codes[-last:, 1].cpu().numpy(), ref.encode(xe[:, d:])[0])
    assert float(out[:-last].abs().max()) == 0.0 and float(dx[:-last].abs().max()) == 0.0
    del dx, out
    wx = ga.activation_backward(dout, x, "silu")
    torch.cuda.synchronize()
    want, bound = ref.backward("silu", de, (xe[:, :d], xe[:, d:]), "bf16")
    close(wx[-last:], want, bound, "silu dx")


def test_layer_norm():
    rows, d, last = 131200, 32768, 2                 # 4.3e9 elements
    print("large layer norm", flush=True)
    x, dy = _mostly_zero(rows, d, last, 3), _mostly_zero(rows, d, last, 4)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    y, c = ga.layer_norm_checkpoint(x, w)
    stats = c.stats
    dx, dw, db = ga.layer_norm_backward(dy, x, w, stats=stats)
    torch.cuda.synchronize()
    xe, de, we = x[-last:].double().cpu().numpy(), dy[-last:].double().cpu().numpy(), w.double().cpu().numpy()
    want, bound, _, _ = ref.layer_norm(xe, we, np.zeros(d), 1e-5, "bf16")
    close(y[-last:], want, bound, "y")
    s = stats[-last:].double().cpu().numpy()
    grads, bounds = ref.layer_norm_backward(de, (xe - s[:, :1]) * s[:, 1:], s[:, 1:], we, "bf16", "fp32", 32)
    close(dx[-last:], grads[0], bounds[0], "dx")
    close(dw, grads[1], bounds[1], "dw")             # the other rows add zeros
    close(db, grads[2], bounds[2], "db")


def test_balance():
    rows, experts, last = 4200000, 1024, 3           # 4.3e9 logits
    print("large balance", flush=True)
    logits = _mostly_zero(rows, experts, last, 5)
    index = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    index[-last:, 0] = torch.tensor([7, 1023, 7], device="cuda", dtype=torch.int32)
    b = ga.balance_loss(logits, index)
    dlogits = ga.balance_loss_backward(logits, b, dloss=torch.tensor(1e9, device="cuda"))
    torch.cuda.synchronize()
    counts = b.counts.cpu().numpy()
    assert counts[0] == rows - last and counts[7] == 2 and counts[1023] == 1 and int(b.tokens) == rows
    le = logits[-last:].double().cpu().numpy()
    want, bound = ref.balance_backward(le, counts, 1, 1.0, rows, np.ones(last, bool), 1e9, "bf16")
    close(dlogits[-last:], want, bound, "dlogits")
