"""The feed-forward layer's products at sizes that take each of their forms (a
stream of the weights, tiles of each size, k cut into slices, the backward pass's
three products together or apart), at the borders between them, at sizes drawn over
the whole range, past 2^31 elements, and on two streams at once (needs an MI355X).
Bounds: feed_forward_ref."""
import math
import random

import numpy as np
import pytest
import torch

import feed_forward_ref as ff
import gated_activation_amd as ga
from test_gpu_feed_forward import ACTS, check
from test_gpu_mxfp4 import _layer, _quantised_normal
from test_gpu_mxfp4 import test_product as check_product
from test_gpu_mxfp4 import test_product_live_rows_and_large as check_product_live
from train_gpu import PAD, close, values

pytestmark = pytest.mark.gpu


# the first product's form, the second's
@pytest.mark.parametrize("rows,H,d,act,live", [
    (1500, 64, 5632, "silu", None),            # 128 x 192; cut
    (1500, 64, 5632, "squared_relu", 1200),    # 128 x 192 without a gate
    (5700, 1536, 64, "gelu", None),            # cut; 128 x 192; the gradients' products apart and cut
    (2048, 64, 3584, "silu", 1111),            # 256 x 256
    (4096, 3584, 64, "gelu_tanh", None),       # cut; 256 x 256, also of dx
    (2200, 2000, 72, "silu", 2199),            # cut; 128 x 192; 1120 tiles of dx
    (64, 2048, 4096, "gelu_tanh", None),       # 64 x 64, cut; 256 x 256 of dw_in
    (500, 64, 4096, "silu", 400),              # 128 x 128 with four stages
    (500, 4096, 64, "gelu", None),             # the three together, none cut
    (50, 64, 8192, "silu", 33),                # 64 x 64 whole; the three together, dx cut in 32
    (2049, 264, 136, "squared_relu", None),    # the three together, the weights' gradients cut in 4 of 33 steps
    (2600, 512, 4096, "silu", 2500),           # together, all whole
    (4096, 72, 64, "gelu", 4001),              # all three cut
    (16384, 64, 64, "silu", 9000),             # cut in 32, of which some have no live row
    (9000, 512, 128, "gelu_tanh", None),       # 1128 tiles of dx
    (1024, 4096, 1024, "silu", None),          # apart
])
def test_forms(rows, H, d, act, live):
    print(f"feed forward {act} {rows}x{H}x{d} live {live}", flush=True)
    check(rows, H, d, act, "bf16", live)


@pytest.mark.parametrize("rows", [4, 5, 8, 9, 15, 16, 17, 63, 64, 65, 128, 129, 192, 193, 256, 257])
def test_borders_of_rows(rows):
    print(f"feed forward {rows} rows", flush=True)
    check(rows, 136, 264, ACTS[rows % 4], "fp16" if rows % 2 else "bf16", rows - 1 if rows % 3 == 0 else None)


@pytest.mark.parametrize("H,d", [(8, 8), (8, 4104), (4104, 8), (56, 64), (64, 120), (120, 4096), (4088, 2056)])
@pytest.mark.parametrize("rows", [1, 6, 11])
def test_few_tokens_of_odd_layers(rows, H, d):
    print(f"feed forward {rows}x{H}x{d}", flush=True)
    check(rows, H, d, ACTS[(rows + H // 8) % 4], "bf16")


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    rng = random.Random(seed)
    rows, H, d = _log(rng, 1, 5000), 8 * _log(rng, 1, 300), 8 * _log(rng, 1, 600)
    rows = max(1, min(rows, (1 << 32) // (H * d)))
    act, dtype = rng.choice(ACTS), rng.choice(["bf16", "fp16"])
    live = rng.randint(0, rows) if rng.random() < 0.4 else None
    print(f"feed forward {act} {dtype} {rows}x{H}x{d} live {live}", flush=True)
    check(rows, H, d, act, dtype, live, seed)


@pytest.mark.parametrize("seed", range(16))
def test_drawn_mxfp4(seed):
    rng = random.Random(100 + seed)
    if seed % 2:
        rows, n, k = _log(rng, 1, 4000), _log(rng, 1, 4000), _log(rng, 1, 8000)
        rows = max(1, min(rows, (1 << 32) // (n * k)))
        print(f"product {rows}x{n}x{k}", flush=True)
        check_product_live(rows, n, k, rng.choice([None, rng.randint(0, rows)]))
    else:
        rows, H, d = _log(rng, 1, 3000), 8 * _log(rng, 1, 200), 32 * _log(rng, 1, 100)
        rows = max(1, min(rows, (1 << 31) // (H * d)))
        act, dtype = rng.choice(ACTS), rng.choice(["bf16", "fp16"])
        print(f"layer {act} {dtype} {rows}x{H}x{d}", flush=True)
        _layer(act, rows, H, d, rng.choice([None, rng.randint(1, rows)]), dtype)


@pytest.mark.parametrize("rows,n,k", [(3500, 3584, 96), (1000, 4096, 288), (2000, 4000, 544), (300, 500, 8192), (64, 8192, 64),
                                      (40, 256, 8192)])
def test_forms_of_the_4_bit_product(rows, n, k):
    check_product(rows, n, k)


@pytest.mark.parametrize("act,rows,H,d,live", [("silu", 3500, 32, 3584, 3000), ("gelu", 1000, 64, 2048, None),
                                               ("squared_relu", 2000, 64, 2048, None), ("gelu_tanh", 50, 64, 4096, None),
                                               ("silu", 40, 4096, 64, 31), ("squared_relu", 100, 4096, 128, None),
                                               ("silu", 16, 136, 96, 15), ("gelu", 17, 136, 96, None)])
def test_forms_of_the_4_bit_layer(act, rows, H, d, live):
    print(f"layer {act} {rows}x{H}x{d} live {live}", flush=True)
    _layer(act, rows, H, d, live, "bf16")


def test_past_2_to_the_31_elements():
    """Rows whose kept values lie past 2^31 elements, and the gradients of a batch in which only they count."""
    rows, H, d, last = 70000, 8, 16384, 5
    rng = np.random.default_rng(3)
    s = {k: values(rng, shape, "bf16", std=std) for k, shape, std in
         (("x", (rows, H), 1.0), ("w_in", (2 * d, H), H ** -0.5), ("w_down", (H, d), d ** -0.5), ("dy", (rows, H), 1.0))}
    g = {k: v[0].cuda() for k, v in s.items()}
    e = {k: v[1] for k, v in s.items()}
    print("forward", flush=True)
    y, kept = ga.feed_forward_train(g["x"], g["w_in"], g["w_down"])
    assert kept.numel() > 2 ** 31
    at = [0, 1, 32767, 32768, 65535, 65536, rows - 2, rows - 1]
    want, bound, _, z, bz = ff.forward("silu", e["x"][at], e["w_in"], e["w_down"], "bf16")
    close(y[at], want, bound, "y")
    close(kept[at], z, bz, "kept")
    g["dy"][:-last] = 0
    print("backward", flush=True)
    dx, dw_in, dw_down = ga.feed_forward_backward(g["dy"], g["x"], kept, g["w_in"], g["w_down"])
    grads = ff.backward("silu", e["dy"][-last:], e["x"][-last:], kept[-last:].double().cpu().numpy(), e["w_in"], e["w_down"],
                        "bf16")
    for got, (w, b, _), what in zip((dx[-last:], dw_in, dw_down), grads, ("dx", "dw_in", "dw_down")):
        close(got, w, b, what)
    assert not bool(dx[:-last].any())
    del kept, dx, dw_in, dw_down
    torch.cuda.empty_cache()


def test_4_bits_past_2_to_the_31_elements():
    rows, d, n = 70000, 32768, 40000
    base = values(np.random.default_rng(4), (1000, d), "bf16")[0].cuda()
    x = base.repeat(rows // 1000, 1)
    assert x.numel() > 2 ** 31
    print("quantize", flush=True)
    q, part = ga.mxfp4_quantize(x), ga.mxfp4_quantize(base)
    assert torch.equal(q.codes.view(-1, 1000, d // 2)[-1], part.codes) and torch.equal(q.scales.view(-1, 1000, d // 32)[-1], part.scales)
    print("dequantize", flush=True)
    back = ga.mxfp4_dequantize(q, torch.bfloat16, out=x)
    assert torch.equal(back[-1000:], ga.mxfp4_dequantize(part, torch.bfloat16))
    del x, back, q
    print("product", flush=True)
    a = ga.mxfp4_quantize(base[:, :64].contiguous().repeat(rows // 1000, 1))
    w = ga.mxfp4_quantize(values(np.random.default_rng(5), (n, 64), "bf16")[0].cuda())
    out = ga.mxfp4_product(a, w, torch.bfloat16)
    assert out.numel() > 2 ** 31
    few = [0, 999, 52428, 53687, rows - 1]
    ae = ga.mxfp4_dequantize(a, torch.float32)[few].double().cpu().numpy()
    want, bound = ff.product4(ae, ga.mxfp4_dequantize(w, torch.float32).double().cpu().numpy(), "bf16")
    close(out[few], want, bound, "product")
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [1, 40])
def test_weights_past_2_to_the_31_bytes(rows):
    """A weight whose rows repeat: so must the outputs, of a stream of it and of tiles."""
    n, k, block = 9000 * 1000, 512, 1000
    a = ga.mxfp4_quantize(values(np.random.default_rng(6), (rows, k), "bf16")[0].cuda())
    part = ga.mxfp4_quantize(values(np.random.default_rng(7), (block, k), "bf16")[0].cuda())
    w = ga.Mxfp4(part.codes.repeat(n // block, 1), part.scales.repeat(n // block, 1), k)
    assert w.codes.numel() > 2 ** 31
    print("product", flush=True)
    out = ga.mxfp4_product(a, w, torch.bfloat16).view(rows, -1, block)
    want, bound = ff.product4(*(ga.mxfp4_dequantize(q, torch.float32).double().cpu().numpy() for q in (a, part)), "bf16")
    close(out[:, 0].contiguous(), want, bound, "product")
    assert bool((out == out[:, :1]).all())
    del out, w
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls that cut k, on two streams, neither waiting for the other; their scratch memory is their own."""
    rng = np.random.default_rng(8)
    rows, H, d = 96, 1024, 2048
    sets = []
    for _ in range(2):
        t = {k: values(rng, shape, "bf16", std=std)[0].cuda() for k, shape, std in
             (("x", (rows, H), 1.0), ("w_in", (2 * d, H), H ** -0.5), ("w_down", (H, d), d ** -0.5), ("dy", (rows, H), 1.0))}
        w_in, _ = _quantised_normal(rng, 2 * d, H)
        w_down, _ = _quantised_normal(rng, H, d)
        sets.append((t, w_in, w_down))
    assert ga.feed_forward_workspace_bytes(rows, H, d) > rows * d * 2 + 256  # sums of slices

    def step(t, w_in, w_down):
        y, kept = ga.feed_forward_train(t["x"], t["w_in"], t["w_down"])
        return (y, kept, *ga.feed_forward_backward(t["dy"], t["x"], kept, t["w_in"], t["w_down"]),
                ga.feed_forward_mxfp4(t["x"], w_in, w_down))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(8):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(step(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("rows,H,d", [(4096, 72, 64), (100, 1024, 1024), (40, 512, 4096), (5700, 1536, 64)])
def test_workspaces_of_cut_products(rows, H, d):
    """Sums of slices stay within the workspace, and need all that is asked for."""
    rng = np.random.default_rng(rows)
    t = {k: values(rng, shape, "bf16", std=std)[0].cuda() for k, shape, std in
         (("x", (rows, H), 1.0), ("w_in", (2 * d, H), H ** -0.5), ("w_down", (H, d), d ** -0.5), ("dy", (rows, H), 1.0))}
    y, kept = ga.feed_forward_train(t["x"], t["w_in"], t["w_down"])
    q_in, q_down = ga.mxfp4_quantize(t["w_in"]), ga.mxfp4_quantize(t["w_down"])
    calls = [(ga.feed_forward_workspace_bytes, lambda w: (ga.feed_forward(t["x"], t["w_in"], t["w_down"], workspace=w),)),
             (ga.feed_forward_backward_workspace_bytes,
              lambda w: ga.feed_forward_backward(t["dy"], t["x"], kept, t["w_in"], t["w_down"], workspace=w)),
             (ga.feed_forward_mxfp4_workspace_bytes, lambda w: (ga.feed_forward_mxfp4(t["x"], q_in, q_down, workspace=w),))]
    for bytes_of, call in calls:
        need, want = bytes_of(rows, H, d), call(None)
        buf = torch.full((need + 4096,), PAD, dtype=torch.uint8, device="cuda")
        for a, b in zip(call(buf[:need]), want):
            assert torch.equal(a, b)
        assert bool((buf[need:] == PAD).all())
        with pytest.raises(ga.GaError):
            call(buf[:need - 1])


def test_two_graphs_of_one_workspace():
    """Two captured calls that share the caller's workspace, replayed in turn."""
    rng = np.random.default_rng(10)
    t = {k: values(rng, shape, "fp16", std=std)[0].cuda() for k, shape, std in
         (("x", (80, 512), 1.0), ("w_in", (512, 512), 512 ** -0.5), ("w_down", (512, 256), 256 ** -0.5))}
    ws = torch.empty(ga.feed_forward_workspace_bytes(80, 512, 256), dtype=torch.uint8, device="cuda")
    xs = [t["x"].clone(), t["x"].flip(0).contiguous()]
    want = [ga.feed_forward(x, t["w_in"], t["w_down"]) for x in xs]
    outs, graphs = [], []
    for x in xs:
        outs.append(torch.empty_like(x))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ga.feed_forward(x, t["w_in"], t["w_down"], out=outs[-1], workspace=ws)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)
