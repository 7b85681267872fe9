"""Calls of the feed-forward operators that the documentation allows beside the usual
ones: arrays at any alignment natural to their type, parts of larger arrays, no rows,
a live count inside another array, x twice (needs an MI355X).  The same bits as the
usual call's, unless a bound is named."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga
from train_gpu import TYPES, check_guard, guarded, placed, values

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh", "gelu", "squared_relu"]


def _quantised(rng, n, k):
    return ga.mxfp4_quantize(values(rng, (n, k), "bf16", std=k ** -0.5)[0].cuda())


def _part(q, first):
    """The rows of q from `first` on, where they lie."""
    return ga.Mxfp4(q.codes[first:], q.scales[first:], q.d)


def _whole(q):
    return ga.Mxfp4(q.codes.clone(), q.scales.clone(), q.d)


@pytest.mark.parametrize("first", [1, 2, 3])
@pytest.mark.parametrize("rows,n,k", [(1, 40, 96), (3, 5000, 33), (40, 256, 2080), (300, 264, 4099), (3500, 3600, 1120)])
def test_products_of_parts(rows, n, k, first):
    """Rows of a larger array, whose scales then begin at any byte."""
    rng = np.random.default_rng(rows + n)
    print(f"product {rows}x{n}x{k} from row {first}", flush=True)
    a, w = _part(_quantised(rng, rows + first, k), first), _part(_quantised(rng, n + first, k), first)
    for dtype in ("bf16", "fp32"):
        buf, out = guarded((rows, n), TYPES[dtype], first)
        ga.mxfp4_product(a, w, TYPES[dtype], out=out)
        assert torch.equal(out, ga.mxfp4_product(_whole(a), _whole(w), TYPES[dtype]))
        check_guard(buf, rows * n, first)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d", [(2, 72, 96), (30, 2056, 160), (300, 264, 1056), (2500, 520, 1056)])
def test_4_bit_layer_anywhere(rows, H, d, act):
    rng = np.random.default_rng(rows + H)
    print(f"4-bit layer {act} {rows}x{H}x{d}", flush=True)
    halves = 1 if act == "squared_relu" else 2
    x = values(rng, (rows, H), "bf16")[0]
    w_in, w_down = _part(_quantised(rng, halves * d + 1, H), 1), _part(_quantised(rng, H + 3, d), 3)
    want = ga.feed_forward_mxfp4(x.cuda(), _whole(w_in), _whole(w_down), act)
    live = torch.tensor([7, rows, -1], dtype=torch.int32, device="cuda")[1:]
    for offset in (1, 3):
        buf, out = guarded((rows, H), torch.bfloat16, offset)
        ga.feed_forward_mxfp4(placed(x, offset), w_in, w_down, act, live_rows=live, out=out)
        assert torch.equal(out, want)
        check_guard(buf, rows * H, offset)


@pytest.mark.parametrize("rows,H,d", [(2, 72, 96), (60, 512, 1024), (300, 264, 136), (2100, 1032, 264)])
def test_parts_of_larger_arrays(rows, H, d):
    """Expert e's rows and weights out of stacked ones, its gradients from them."""
    rng = np.random.default_rng(rows)
    x, dy = (values(rng, (rows + 8, H), "bf16")[0].cuda() for _ in range(2))
    w_in = values(rng, (3, 2 * d, H), "bf16", std=H ** -0.5)[0].cuda()
    w_down = values(rng, (3, H, d), "bf16", std=d ** -0.5)[0].cuda()
    ys = torch.zeros(rows + 8, H, device="cuda").bfloat16()
    parts = x[8:], w_in[1], w_down[1]
    alone = [t.clone() for t in parts]
    y, kept = ga.feed_forward_train(*parts, out=ys[8:])
    want, z = ga.feed_forward_train(*alone)
    assert torch.equal(y, want) and torch.equal(kept, z) and not bool(ys[:8].any())
    for a, b in zip(ga.feed_forward_backward(dy[8:], parts[0], kept, *parts[1:]),
                    ga.feed_forward_backward(dy[8:].clone(), alone[0], z, *alone[1:])):
        assert torch.equal(a, b)
    # one array as two arguments that are only read
    for a, b in zip(ga.feed_forward_backward(parts[0], parts[0], kept, *parts[1:]),
                    ga.feed_forward_backward(alone[0].clone(), alone[0], z, *alone[1:])):
        assert torch.equal(a, b)
    q = ga.mxfp4_quantize(alone[0])
    assert torch.equal(ga.mxfp4_product(q, q, torch.float32), ga.mxfp4_product(q, _whole(q), torch.float32))


def test_no_rows():
    w_in, w_down = (ga.mxfp4_quantize(torch.randn(n, k, device="cuda")) for n, k in ((64, 16), (16, 32)))
    for dtype in TYPES.values():
        x = torch.empty(0, 64, dtype=dtype, device="cuda")
        q = ga.mxfp4_quantize(x)
        assert q.codes.shape == (0, 32) and q.scales.shape == (0, 2) and q.d == 64
        assert ga.mxfp4_dequantize(q, dtype).shape == (0, 64)
        assert ga.activation_mxfp4(x, "silu").codes.shape == (0, 16)
        assert ga.mxfp4_product(ga.mxfp4_quantize(x[:, :16].contiguous()), w_in, dtype).shape == (0, 64)
        if dtype != torch.float32:
            y = ga.feed_forward_mxfp4(torch.empty(0, 16, dtype=dtype, device="cuda"), w_in, w_down)
            assert y.shape == (0, 16) and y.dtype == dtype


@pytest.mark.parametrize("rows", [1, 12, 40, 300, 2048])
def test_values_at_the_ends_of_the_types(rows):
    """Subnormal weights in fp16 and bf16 count, and so do the least and the greatest scale."""
    g = torch.Generator(device="cuda").manual_seed(rows)

    def normal(*shape, std):
        return torch.randn(*shape, device="cuda", generator=g) * std

    for dtype, x_std, w_std in ((torch.float16, 1.0, 2e-6), (torch.bfloat16, 1e30, 3e-39)):
        x, w_in, w_down = normal(rows, 512, std=x_std).to(dtype), normal(256, 512, std=w_std).to(dtype), normal(512, 128, std=1.0).to(dtype)
        _, kept = ga.feed_forward_train(x, w_in, w_down)
        z, size = x.double() @ w_in.double().T, x.double().abs() @ w_in.double().abs().T
        # z's rounding to the type (in fp16 to a multiple of 2^-24), and 520 additions in fp32, each off by 2^-23 at most
        half = torch.finfo(dtype).eps / 2
        bound = half * z.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0) + 520 * 2.0 ** -23 * size
        assert bool(((kept.double() - z).abs() <= bound).all()) and float(z.abs().max()) > 20 * float(bound.max()), dtype
    k = 1024
    a, w = (torch.randint(0, 256, (n, k // 2), device="cuda", generator=g, dtype=torch.uint8) for n in (rows, 200))

    def q(codes, s):
        return ga.Mxfp4(codes, torch.full((len(codes), k // 32), s, dtype=torch.uint8, device="cuda"), k)

    # multiples of 1/4 below 36 * 1024: exact in fp32, and so is any power of two of them
    one = ga.mxfp4_dequantize(q(a, 127), torch.float32).double() @ ga.mxfp4_dequantize(q(w, 127), torch.float32).double().T
    for sa, sw in ((254, 0), (0, 254), (253, 1), (127, 0), (0, 127), (254, 100), (127, 127)):
        got = ga.mxfp4_product(q(a, sa), q(w, sw), torch.float32).double()
        assert torch.equal(got, one * 2.0 ** (sa + sw - 254)), (sa, sw)
