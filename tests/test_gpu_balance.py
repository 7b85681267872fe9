"""The balance loss, its counts and its gradient on the GPU against fp64 (needs
an MI355X)."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import TYPES, check_guard, close, guarded, live_tensor, untouched, values

pytestmark = pytest.mark.gpu


def _run(rng, rows, experts, k, dtype, index_type, masked, live, coefficient=0.01, bad=True):
    logits, le = values(rng, (rows, experts), dtype, std=1.5)
    index = rng.integers(0, experts, (rows, k))
    if bad and rows * k > 4:                      # dropped choices, and the same expert twice
        index.reshape(-1)[::5] = -1
        index.reshape(-1)[3] = experts + 7
        index[-1, :] = experts - 1
    mask = rng.random(rows) < 0.7 if masked else np.ones(rows, bool)
    n = rows if live is None else max(0, min(live, rows))
    use = mask & (np.arange(rows) < n)
    lv = live_tensor(live)
    m = torch.from_numpy(mask).cuda() if masked else None
    lg, ig = logits.cuda(), torch.from_numpy(index.astype(index_type)).cuda()
    bal = ga.balance_loss(lg, ig, coefficient, mask=m, live_rows=lv)
    dloss = torch.tensor(1.5, device="cuda")
    buf, out = guarded((rows, experts), TYPES[dtype])
    ga.balance_loss_backward(lg, bal, dloss=dloss, mask=m, live_rows=lv, out=out)
    torch.cuda.synchronize()
    loss, bound, counts, offsets, tokens = ref.balance(le, index, coefficient, use)
    label = f"balance {dtype} {rows}x{experts} k{k} live {live}"
    assert np.array_equal(bal.counts.cpu().numpy(), counts), label
    assert np.array_equal(bal.offsets.cpu().numpy(), offsets) and int(bal.tokens) == tokens, label
    assert abs(float(bal.loss) - loss) <= bound + 1e-12, f"{label}: loss {float(bal.loss)} want {loss} bound {bound}"
    want, gb = ref.balance_backward(le, counts, k, coefficient, tokens, use, 1.5, dtype)
    close(out[:n], want[:n], gb[:n], label + " dlogits")
    untouched(out, n, label)
    check_guard(buf, rows * experts)
    return bal


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,experts,k,live", [
    (1, 1, 1, None), (1, 2, 1, None), (5, 3, 2, None), (64, 8, 2, 50), (300, 9, 3, None), (77, 16, 4, 0), (40, 31, 1, None),
    (1000, 64, 6, 999), (513, 65, 2, None), (2048, 128, 8, None), (100, 200, 8, 5000), (70, 256, 8, None), (90, 300, 4, None),
    (33, 512, 8, None), (50, 513, 8, 49), (40, 1024, 16, None), (3000, 60, 4, 2999)])
def test_loss_counts_and_gradient(dtype, rows, experts, k, live):
    print(f"balance {dtype} {rows}x{experts} k{k}", flush=True)
    rng = np.random.default_rng(rows * 3 + experts)
    _run(rng, rows, experts, k, dtype, np.int64, rows % 2 == 0, live)
    _run(rng, rows, experts, k, dtype, np.int32, rows % 2 == 1, live, bad=False)


def test_many_tokens_and_the_same_bits():
    rng = np.random.default_rng(8)
    a = _run(rng, 20000, 96, 6, "bf16", np.int64, True, 19000)
    rng = np.random.default_rng(8)
    b = _run(rng, 20000, 96, 6, "bf16", np.int64, True, 19000)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.counts, b.counts)


def test_gradient_against_differences():
    """The kernel's own loss, differenced along random directions in fp32."""
    rng = np.random.default_rng(5)
    logits, le = values(rng, (40, 12), "fp32")
    index = torch.from_numpy(rng.integers(0, 12, (40, 2))).cuda()
    h = 2.0 ** -5
    b = ga.balance_loss(logits.cuda(), index)
    g = ga.balance_loss_backward(logits.cuda(), b).double().cpu().numpy()
    for _ in range(4):
        v = rng.normal(0, 1, le.shape).astype(np.float32)
        vg = torch.from_numpy(v).cuda()
        plus, minus = (float(ga.balance_loss(logits.cuda() + s * h * vg, index).loss) for s in (1, -1))
        # a softmax' third derivative along v is at most 8 max|v|^3 of a mean of counts (the loss, about 1), over
        # 6; the loss carries (n + 100) roundings
        slack = 1.5 * (h * h * 8 * np.abs(v).max() ** 3 / 6 + 140 * ref.U / h)
        assert abs((g * v).sum() - (plus - minus) / (2 * h)) <= slack
        assert np.abs(g * v).sum() > 4 * 140 * ref.U / h


def test_even_router_has_the_coefficient_as_its_loss():
    experts, k = 16, 2
    index = torch.arange(64 * k, device="cuda").reshape(64, k) % experts
    b = ga.balance_loss(torch.zeros(64, experts, device="cuda"), index, 0.25)
    assert abs(float(b.loss) - 0.25) < 1e-6 and b.counts.tolist() == [8] * experts


def test_tokens_without_a_choice_or_a_probability():
    """Every token masked; experts ruled out by -inf; a token with no expert left; NaN in a masked token."""
    rng = np.random.default_rng(2)
    logits = rng.normal(0, 1, (32, 12)).astype(np.float32)
    index = rng.integers(0, 12, (32, 2))
    none = torch.zeros(32, dtype=torch.bool, device="cuda")
    lg, ig = torch.from_numpy(logits).cuda(), torch.from_numpy(index).cuda()
    b = ga.balance_loss(lg, ig, mask=none)
    g = ga.balance_loss_backward(lg, b, mask=none)
    assert float(b.loss) == 0 and int(b.tokens) == 0 and int(b.offsets[-1]) == 0 and float(g.abs().max()) == 0
    logits[:, 5] = -np.inf
    logits[3, :] = -np.inf
    logits[4, 2] = np.nan
    use = np.ones(32, bool)
    use[4] = False
    lg, m = torch.from_numpy(logits).cuda(), torch.from_numpy(use).cuda()
    b = ga.balance_loss(lg, ig, mask=m)
    g = ga.balance_loss_backward(lg, b, mask=m).cpu().numpy()
    le = logits.astype(np.float64)
    le[4] = 0
    loss, bound, counts, _, n = ref.balance(le, index, 1.0, use)
    assert abs(float(b.loss) - loss) <= bound and n == 31
    assert np.isfinite(g).all() and (g[3] == 0).all() and (g[4] == 0).all() and (g[:, 5] == 0).all()
    want, gb = ref.balance_backward(le, counts, 2, 1.0, n, use, 1.0, "fp32")
    assert np.all(np.abs(g - want) <= gb)
    # a token that counts and is not finite shows
    b = ga.balance_loss(lg, ig)
    assert np.isnan(float(b.loss)) and np.array_equal(b.counts.cpu().numpy(), np.bincount(index.reshape(-1), minlength=12))
