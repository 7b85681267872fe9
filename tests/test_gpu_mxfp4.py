"""Microscaled 4-bit arrays, their product and the feed-forward layer on them,
against fp64 (needs an MI355X).  Bounds: feed_forward_ref."""
import numpy as np
import pytest
import torch

import feed_forward_ref as ff
import gated_activation_amd as ga
import train_ref as ref
from train_gpu import PAD, TYPES, check_guard, close, guarded, live_tensor, untouched, values

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh", "gelu", "squared_relu"]


def _weight(rng, n, k):
    """A Mxfp4 of random codes on the GPU, and its exact values."""
    codes = rng.integers(0, 16, (n, ff.groups(k) * 32)).astype(np.uint8)
    codes[:, k:] = 0
    scales = rng.integers(118, 128, (n, ff.groups(k))).astype(np.uint8)
    packed = ff.pack(codes)
    return ga.Mxfp4(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), k), ff.values(packed, scales, k)


def _same(q, x, label):
    packed, scales = ff.quantize(x)
    s = q.scales.cpu().numpy()
    assert np.array_equal(s, scales), f"{label}: scales differ at {np.argwhere(s != scales)[:4].tolist()}"
    c = q.codes.cpu().numpy()
    if not np.array_equal(c, packed):
        at = np.argwhere(ff.unpack(c) != ff.unpack(packed))[0]
        raise AssertionError(f"{label}: code at {at.tolist()} of {x[at[0], at[1]]!r} is {ff.unpack(c)[tuple(at)]}, "
                             f"not {ff.unpack(packed)[tuple(at)]} (scale {scales[at[0], at[1] // 32]})")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,d,live", [(1, 1, None), (3, 7, None), (1, 31, None), (2, 32, None), (5, 33, None), (4, 100, 3),
                                         (7, 127, None), (6, 128, 0), (3, 129, None), (64, 2048, 50), (33, 4099, None),
                                         (2, 65536, None), (300, 160, 1000)])
def test_quantize_is_exact(dtype, rows, d, live):
    print(f"mxfp4 {dtype} {rows}x{d}", flush=True)
    rng = np.random.default_rng(rows * 5 + d)
    t, x = values(rng, (rows, d), dtype)
    t = (t.double() * torch.from_numpy(np.exp2(rng.integers(-12, 12, (rows, d)))).double()).to(TYPES[dtype])
    x = t.double().numpy()
    n = rows if live is None else max(0, min(live, rows))
    nb = ff.groups(d)
    cb, codes = guarded((rows, 16 * nb), torch.uint8)
    sb, scales = guarded((rows, nb), torch.uint8, 3)
    q = ga.mxfp4_quantize(t.cuda(), live_rows=live_tensor(live), out=ga.Mxfp4(codes, scales, d))
    _same(ga.Mxfp4(q.codes[:n], q.scales[:n], d), x[:n], f"{rows}x{d}")
    check_guard(cb, codes.numel())
    check_guard(sb, scales.numel(), 3)
    assert bool((codes[n:] == PAD).all()) and bool((scales[n:] == PAD).all())
    buf, out = guarded((rows, d), TYPES[dtype], 1)
    ga.mxfp4_dequantize(q, TYPES[dtype], live_rows=live_tensor(live), out=out)
    want = ff.quantized(x[:n])
    # a value of two bits and a power of two in fp16 and bf16's range is exact
    close(out[:n], want, np.where(np.abs(want) < 2.0 ** -14, 2.0 ** -25, 0.0), "values")
    untouched(out, n, "values")
    check_guard(buf, out.numel(), 1)


def test_every_bf16_value():
    """All finite bf16 magnitudes and signs, each in a block whose largest value is itself, and each in a block
    with a fixed largest value."""
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    x = bits.view(np.float32)
    x = x[np.isfinite(x)]
    alone = np.zeros((len(x), 32), np.float32)
    alone[np.arange(len(x)), np.arange(len(x)) % 32] = x
    small = x[np.abs(x) <= 5.0]
    beside = np.concatenate([small, np.zeros(-len(small) % 31, np.float32)]).reshape(-1, 31)
    beside = np.concatenate([beside, np.full((len(beside), 1), 5.0, np.float32)], axis=1)
    for a in (alone, beside):
        t = torch.from_numpy(a).cuda()
        for dt in (torch.bfloat16, torch.float32):
            q = ga.mxfp4_quantize(t.to(dt))
            _same(q, a.astype(np.float64), str(dt))
            got = ga.mxfp4_dequantize(q, torch.float32).double().cpu().numpy()
            assert np.array_equal(got, ff.quantized(a.astype(np.float64)))


def test_blocks_that_are_not_numbers():
    x = np.random.default_rng(1).normal(0, 1, (4, 100)).astype(np.float32)
    x[0, 33], x[1, 99], x[2, 0] = np.nan, np.inf, -np.inf
    x[3] = 0.0
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        t = torch.from_numpy(x).to(dt)
        q = ga.mxfp4_quantize(t.cuda())
        _same(q, t.double().numpy(), str(dt))
        v = ga.mxfp4_dequantize(q, dt).double().cpu().numpy()
        assert np.isnan(v[0, 32:64]).all() and np.isnan(v[1, 96:]).all() and np.isnan(v[2, :32]).all()
        assert np.isfinite(v).sum() == 400 - 32 - 4 - 32 and (v[3] == 0).all()
        # and through a product: the rows of a, the columns of w
        w, we = _weight(np.random.default_rng(2), 40, 100)
        y = ga.mxfp4_product(q, w, torch.float32).cpu()
        assert bool(y[:3].isnan().all()) and bool((y[3] == 0).all())
        w.scales[5, 1] = 255
        y = ga.mxfp4_product(w, q, torch.float32).cpu()
        assert bool(y[:, :3].isnan().all()) and bool(y[5].isnan().all()) and float(y[:5, 3].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_activation_is_the_activation_then_quantised(act, dtype):
    """Bit for bit what the forward-only activation stores, quantised."""
    rng = np.random.default_rng(3)
    for rows, d, live in ((1, 5, None), (3, 32, None), (40, 100, 29), (7, 4100, None), (64, 2048, 40)):
        print(f"activation {act} {dtype} {rows}x{d}", flush=True)
        t, _ = values(rng, (rows, ref.halves(act) * d), dtype, std=1.5)
        x, n = t.cuda(), rows if live is None else live
        lv = live_tensor(rows if live is None else live)
        if act == "silu":
            y = ga.silu_and_mul_bounded(x, lv)
        elif act == "squared_relu":
            y = ga.squared_relu_bounded(x, lv)
        else:
            y = ga.gelu_and_mul(x, "tanh" if act == "gelu_tanh" else "none")
        cb, codes = guarded((rows, 16 * ff.groups(d)), torch.uint8)
        q = ga.activation_mxfp4(x, act, live_rows=lv, out=ga.Mxfp4(codes, torch.full((rows, ff.groups(d)), PAD, dtype=torch.uint8,
                                                                                   device="cuda"), d))
        want = ga.mxfp4_quantize(y)
        assert torch.equal(q.codes[:n], want.codes[:n]) and torch.equal(q.scales[:n], want.scales[:n]), (act, rows, d)
        assert bool((q.codes[n:] == PAD).all()) and bool((q.scales[n:] == PAD).all())
        check_guard(cb, codes.numel())


PRODUCTS = [(1, 1, 1), (1, 16, 32), (2, 7, 33), (5, 40, 100), (16, 64, 256), (17, 129, 257), (33, 100, 1000), (64, 333, 512),
            (128, 128, 4099), (130, 1, 64), (257, 520, 288), (1, 2048, 4096), (4, 1000, 16384), (100, 264, 65536)]


@pytest.mark.parametrize("rows,n,k", PRODUCTS)
def test_product(rows, n, k):
    print(f"product {rows}x{n}x{k}", flush=True)
    rng = np.random.default_rng(rows + n + k)
    a, ae = _weight(rng, rows, k)
    w, we = _weight(rng, n, k)
    for dtype in ("fp32", "bf16", "fp16"):
        buf, out = guarded((rows, n), TYPES[dtype], 1)
        ga.mxfp4_product(a, w, TYPES[dtype], out=out)
        want, bound = ff.product4(ae, we, dtype)
        if dtype == "fp16":
            want = np.where(np.abs(want) >= 65520, np.copysign(np.inf, want), want)
        close(out, want, bound, f"product {rows}x{n}x{k} {dtype}")
        check_guard(buf, rows * n, 1)


@pytest.mark.parametrize("rows,n,k,live", [(40, 72, 96, 13), (300, 40, 640, 256), (20, 33, 32, 0), (9, 64, 64, 100),
                                           (2048, 2048, 512, 1500), (3000, 1024, 2112, None), (70, 20000, 320, 69)])
def test_product_live_rows_and_large(rows, n, k, live):
    print(f"product {rows}x{n}x{k} live {live}", flush=True)
    rng = np.random.default_rng(rows + n + k)
    a, ae = _weight(rng, rows, k)
    w, we = _weight(rng, n, k)
    m = rows if live is None else max(0, min(live, rows))
    a.scales[m:] = 255
    buf, out = guarded((rows, n), torch.float32)
    ga.mxfp4_product(a, w, torch.float32, live_rows=live_tensor(live), out=out)
    want, bound = ff.product4(ae[:m], we, "fp32")
    close(out[:m], want, bound, "product")
    untouched(out, m, "product")
    check_guard(buf, rows * n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d,live,dtype", [(1, 64, 96, None, "bf16"), (3, 8, 32, None, "fp16"), (40, 136, 256, 17, "bf16"),
                                                 (130, 264, 160, None, "bf16"), (300, 72, 544, 290, "fp16"),
                                                 (64, 512, 64, 0, "bf16")])
def test_layer(act, rows, H, d, live, dtype):
    print(f"layer {act} {rows}x{H}x{d} live {live}", flush=True)
    _layer(act, rows, H, d, live, dtype)


@pytest.mark.parametrize("act,rows,H,d", [("silu", 1, 2048, 4096), ("gelu_tanh", 4, 1024, 8192), ("gelu", 1100, 1032, 2080),
                                          ("squared_relu", 2300, 1024, 1024), ("silu", 2500, 520, 1056)])
def test_larger_layer(act, rows, H, d):
    print(f"layer {act} {rows}x{H}x{d}", flush=True)
    _layer(act, rows, H, d, None, "bf16")


def _layer(act, rows, H, d, live, dtype):
    rng = np.random.default_rng(rows + H + d)
    t, x = values(rng, (rows, H), dtype)
    n = rows if live is None else live
    # weights whose sums are of the order of 1
    w_in, wie = _quantised_normal(rng, ref.halves(act) * d, H)
    w_down, wde = _quantised_normal(rng, H, d)
    t = t.cuda()
    t[n:] = float("nan")
    buf, out = guarded((rows, H), TYPES[dtype], 1)
    y = ga.feed_forward_mxfp4(t, w_in, w_down, act, live_rows=live_tensor(live), out=out)
    want, bound = ff.layer4(act, x[:n], wie, wde, dtype)
    close(y[:n], want, bound, f"layer {act} {rows}x{H}x{d}")
    if n > 0:
        off = np.linalg.norm(y[:n].double().cpu().numpy() - want)
        # one rounding of the type; the codes that the last bit decides are a few in 10^5 of the terms
        assert off <= (ref.HALF_EPS[dtype] + 1e-3) * np.linalg.norm(want) + 1e-30, off / np.linalg.norm(want)
    untouched(y, n, "layer")
    check_guard(buf, y.numel(), 1)


def _quantised_normal(rng, n, k):
    x = rng.normal(0, k ** -0.5, (n, k))
    packed, scales = ff.quantize(x)
    return ga.Mxfp4(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), k), ff.values(packed, scales, k)


@pytest.mark.parametrize("rows", [1, 24, 1500])
def test_the_layer_is_its_parts(rows):
    """The layer against its parts called one after another, gate | up in fp32 between them; and a captured step."""
    rng = np.random.default_rng(rows)
    H, d = 512, 1024
    x = values(rng, (rows, H), "bf16")[0].cuda()
    w_in, _ = _quantised_normal(rng, 2 * d, H)
    w_down, wde = _quantised_normal(rng, H, d)

    def parts():
        z = ga.mxfp4_product(ga.mxfp4_quantize(x), w_in, torch.float32)
        return ga.mxfp4_product(ga.activation_mxfp4(z, "silu"), w_down, torch.bfloat16)

    whole, chain = ga.feed_forward_mxfp4(x, w_in, w_down), parts()
    want, bound = ff.layer4("silu", x.double().cpu().numpy(), ff.values(w_in.codes.cpu().numpy(), w_in.scales.cpu().numpy(), H),
                            wde, "bf16")
    close(whole, want, bound, "layer")
    close(chain, want, bound, "its parts")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ga.feed_forward_mxfp4(x, w_in, w_down), parts()
    for i in range(3):
        x.mul_(0.75)
        graph.replay()
        eager = ga.feed_forward_mxfp4(x, w_in, w_down), parts()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), i


def test_other_streams_and_workspaces():
    rng = np.random.default_rng(5)
    a, _ = _weight(rng, 30, 4096)
    w, _ = _weight(rng, 200, 4096)
    want = ga.mxfp4_product(a, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(ga.mxfp4_product(a, w), want)
    torch.cuda.current_stream().wait_stream(side)
    need = ga.mxfp4_product_workspace_bytes(30, 200, 4096)
    buf = torch.full((need + 512,), PAD, dtype=torch.uint8, device="cuda")
    assert torch.equal(ga.mxfp4_product(a, w, workspace=buf[:need]), want) and bool((buf[need:] == PAD).all())


def test_arguments():
    x = torch.randn(4, 64, device="cuda")
    q = ga.mxfp4_quantize(x)
    w = ga.mxfp4_quantize(torch.randn(8, 64, device="cuda"))
    for f in (lambda: ga.mxfp4_quantize(x.t()), lambda: ga.mxfp4_quantize(x[:, ::2]), lambda: ga.mxfp4_quantize(x.double()),
              lambda: ga.mxfp4_quantize(x, out=w), lambda: ga.mxfp4_dequantize(q._replace(d=65), torch.float32),
              lambda: ga.mxfp4_dequantize(q._replace(scales=q.scales[:, :1]), torch.float32),
              lambda: ga.mxfp4_dequantize(q, torch.float32, out=x.half()), lambda: ga.mxfp4_product(q, w._replace(d=63)),
              lambda: ga.mxfp4_product(q, None), lambda: ga.mxfp4_product(q, w, out=x), lambda: ga.activation_mxfp4(x[:, :63], "silu"),
              lambda: ga.activation_mxfp4(x, "gelu_sparse"), lambda: ga.feed_forward_mxfp4(x, w, w),
              lambda: ga.feed_forward_mxfp4(x.half(), w, q), lambda: ga.feed_forward_mxfp4(x.half(), None, q)):
        with pytest.raises(ValueError):
            f()
