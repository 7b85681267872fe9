"""What is not a number reaches every output of the feed-forward layer that is formed
from it, and no other, with each activation and in each form of the products (needs
an MI355X).  No bounds: NaN or the same bits."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
import train_ref as ref
from train_gpu import values

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh", "gelu", "squared_relu"]
# a stream of the weights; 64 x 64 tiles with k cut; 128 x 64 and 128 x 128; the largest
SIZES = [(3, 64, 136), (50, 512, 1024), (300, 264, 136), (700, 128, 4096), (2048, 64, 3584)]


def _inputs(rows, H, d, act, dtype):
    rng = np.random.default_rng(rows + H)
    h = ref.halves(act)
    return [values(rng, shape, dtype, std=std)[0].cuda() for shape, std in
            (((rows, H), 1.0), ((h * d, H), H ** -0.5), ((H, d), d ** -0.5), ((rows, H), 1.0))]


def _all(rows, *but):
    m = torch.ones(rows, dtype=torch.bool, device="cuda")
    m[list(but)] = False
    return m


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d", SIZES)
def test_forward(rows, H, d, act):
    print(f"forward {act} {rows}x{H}x{d}", flush=True)
    for dtype in ("bf16", "fp16"):
        x, w_in, w_down, _ = _inputs(rows, H, d, act, dtype)
        clean, z = ga.feed_forward_train(x, w_in, w_down, act)
        x[1, 5], x[rows - 1, H - 1] = float("nan"), float("inf")
        rest = _all(rows, 1, rows - 1)
        y, kept = ga.feed_forward_train(x, w_in, w_down, act)
        for got in (y, ga.feed_forward(x, w_in, w_down, act)):
            assert torch.equal(got[rest], clean[rest])
            assert bool(got[1].isnan().all()) and not bool(got[rows - 1].isfinite().any()), dtype
        assert torch.equal(kept[rest], z[rest]) and bool(kept[1].isnan().all())
        # a weight: of a feature of h every output is formed
        x, w_in, w_down, _ = _inputs(rows, H, d, act, dtype)
        w_in[d - 3, 2] = float("nan")
        assert bool(ga.feed_forward(x, w_in, w_down, act).isnan().all()), dtype


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d", SIZES)
def test_backward(rows, H, d, act):
    print(f"backward {act} {rows}x{H}x{d}", flush=True)
    x, w_in, w_down, dy = _inputs(rows, H, d, act, "bf16")
    _, kept = ga.feed_forward_train(x, w_in, w_down, act)
    clean = ga.feed_forward_backward(dy, x, kept, w_in, w_down, act)
    for at in ([3, d - 1] if act == "squared_relu" else [3, d - 1, d + 3]):
        z = kept.clone()
        z[1, at] = float("nan")
        dx, dw_in, dw_down = ga.feed_forward_backward(dy, x, z, w_in, w_down, act)
        # a gate value forms dgate, dup and h of its feature, an up value dgate and h
        features = [at] if act == "squared_relu" else [at, at + d] if at < d else [at - d]
        assert bool(dx[1].isnan().all()) and torch.equal(dx[_all(rows, 1)], clean[0][_all(rows, 1)]), at
        rest = _all(len(w_in), *features)
        assert bool(dw_in[features].isnan().all()) and torch.equal(dw_in[rest], clean[1][rest]), at
        rest = _all(d, at % d)
        assert bool(dw_down[:, at % d].isnan().all()) and torch.equal(dw_down[:, rest], clean[2][:, rest]), at


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d", [(3, 64, 160), (40, 2048, 128), (50, 512, 1024), (300, 264, 160), (1000, 64, 2048),
                                      (2000, 64, 2048), (3500, 32, 3584)])
def test_4_bit_layer(rows, H, d, act):
    print(f"4-bit layer {act} {rows}x{H}x{d}", flush=True)
    x, w_in, w_down, _ = _inputs(rows, H, d, act, "bf16")
    q_in, q_down = ga.mxfp4_quantize(w_in), ga.mxfp4_quantize(w_down)
    clean = ga.feed_forward_mxfp4(x, q_in, q_down, act)
    x[1, 5], x[rows - 1, H - 1] = float("nan"), -float("inf")
    rest = _all(rows, 1, rows - 1)
    y = ga.feed_forward_mxfp4(x, q_in, q_down, act)
    assert torch.equal(y[rest], clean[rest])
    assert bool(y[1].isnan().all()) and bool(y[rows - 1].isnan().all())
    x = _inputs(rows, H, d, act, "bf16")[0]
    q_down.scales[7, 0] = 255
    y = ga.feed_forward_mxfp4(x, q_in, q_down, act)
    rest = _all(H, 7)
    assert torch.equal(y[:, rest], clean[:, rest]) and bool(y[:, 7].isnan().all())
    q_in.scales[d - 2, H // 32 - 1] = 255
    assert bool(ga.feed_forward_mxfp4(x, q_in, q_down, act).isnan().all())


@pytest.mark.parametrize("rows", [1, 30, 500])
def test_fp16_hidden_values_past_the_type(rows):
    """h is fp16 between the two products: 65520 rounds to an infinity, 255^2 is a number."""
    x = torch.zeros(rows, 8, device="cuda").half()
    x[:, 0], x[:, 1] = 255.0, 1.0
    w_in, w_down = torch.zeros(8, 8, device="cuda").half(), torch.zeros(8, 8, device="cuda").half()
    w_in[0, 0], w_in[1, 0], w_in[1, 1] = 1.0, 1.0, 1.0     # z = 255, 256
    w_down[0, 0], w_down[1, 1] = 2.0 ** -8, 2.0 ** -8
    w_down[2:, 2:] = 1.0
    y, kept = ga.feed_forward_train(x, w_in, w_down, "squared_relu")
    assert bool((kept[:, 0] == 255).all()) and bool((kept[:, 1] == 256).all())
    assert bool((y[:, 1] == float("inf")).all())
    # (an infinity times the zeros of the other outputs' weights is NaN)
    w_down[1, 1] = 0.0
    w_in[1, 1] = 0.0                                       # z = 255, 255
    y = ga.feed_forward(x, w_in, w_down, "squared_relu")
    assert bool((y[:, 0] == torch.tensor(65025.0).half().item() / 256).all()) and bool((y[:, 1:] == 0).all())
