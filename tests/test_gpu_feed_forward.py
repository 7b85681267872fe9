"""The feed-forward layer in 16 bits, forward and backward, against fp64 (needs an
MI355X).  Bounds: feed_forward_ref."""
import numpy as np
import pytest
import torch

import feed_forward_ref as ff
import gated_activation_amd as ga
import train_ref as ref
from train_gpu import PAD, TYPES, check_guard, close, guarded, live_tensor, untouched, values

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh", "gelu", "squared_relu"]


def _inputs(rng, rows, H, d, act, dtype):
    h = ref.halves(act)
    return {"x": values(rng, (rows, H), dtype), "w_in": values(rng, (h * d, H), dtype, std=H ** -0.5),
            "w_down": values(rng, (H, d), dtype, std=d ** -0.5), "dy": values(rng, (rows, H), dtype)}


def _held(got, want, bound, spread, dtype, label):
    close(got, want, bound, label)
    if np.size(want) >= 256:
        off = np.linalg.norm(got.double().cpu().numpy() - want)
        assert off <= ff.norm_bound(want, spread, dtype), f"{label}: errors of norm {off}"


def check(rows, H, d, act, dtype, live=None, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + H * 3 + d)
    s = _inputs(rng, rows, H, d, act, dtype)
    g = {k: v[0].cuda() for k, v in s.items()}
    e = {k: v[1] for k, v in s.items()}
    n = rows if live is None else max(0, min(live, rows))
    lv, zd = live_tensor(live), ref.halves(act) * d
    label = f"{rows}x{H}x{d} {act} {dtype} live {live}"
    if n < rows:  # what lies past the live rows is not read
        for k in ("x", "dy"):
            g[k][n:] = float("nan")
    bufs = {k: guarded(shape, TYPES[dtype]) for k, shape in (("y", (rows, H)), ("kept", (rows, zd)), ("dx", (rows, H)))}
    y, kept = ga.feed_forward_train(g["x"], g["w_in"], g["w_down"], act, live_rows=lv, out=bufs["y"][1], kept=bufs["kept"][1])
    alone = ga.feed_forward(g["x"], g["w_in"], g["w_down"], act, live_rows=lv)
    want, bound, spread, z, bz = ff.forward(act, e["x"][:n], e["w_in"], e["w_down"], dtype)
    _held(y[:n], want, bound, spread, dtype, label + " y")
    close(kept[:n], z, bz, label + " kept")
    assert torch.equal(alone[:n], y[:n]), f"{label}: keeping z changed y"
    # the backward pass from z as it was kept
    zk = kept[:n].double().cpu().numpy()
    if n < rows:
        kept[n:] = float("nan")
    dx, dw_in, dw_down = ga.feed_forward_backward(g["dy"], g["x"], kept, g["w_in"], g["w_down"], act, live_rows=lv,
                                                  out=bufs["dx"][1])
    for got, (w, b, sp), what in zip((dx[:n], dw_in, dw_down),
                                     ff.backward(act, e["dy"][:n], e["x"][:n], zk, e["w_in"], e["w_down"], dtype),
                                     ("dx", "dw_in", "dw_down")):
        _held(got, w, b, sp, dtype, f"{label} {what}")
    untouched(y, n, label + " y")
    untouched(dx, n, label + " dx")
    for k, (buf, t) in bufs.items():
        check_guard(buf, t.numel())


SIZES = [(1, 8, 8), (1, 64, 72), (2, 16, 8), (3, 8, 200), (5, 136, 64), (16, 64, 64), (17, 72, 136), (33, 128, 256),
         (64, 256, 264), (127, 264, 128), (129, 248, 520), (200, 512, 72), (257, 64, 1032), (300, 1024, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,H,d", SIZES)
def test_forward_and_backward(dtype, rows, H, d):
    print(f"feed forward {dtype} {rows}x{H}x{d}", flush=True)
    check(rows, H, d, ACTS[(rows + d // 8) % 4], dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,H,d,live", [(40, 64, 136, 17), (300, 136, 128, 257), (70, 128, 64, 0), (20, 72, 80, 500),
                                           (20, 72, 80, -3), (520, 64, 72, 256), (9, 256, 512, 1)])
def test_live_rows(act, rows, H, d, live):
    print(f"feed forward {act} {rows}x{H}x{d} live {live}", flush=True)
    check(rows, H, d, act, "bf16", live)


@pytest.mark.parametrize("rows,H,d,act", [(2500, 2048, 768, "silu"), (1500, 1032, 2056, "gelu"), (700, 512, 4096, "gelu_tanh"),
                                          (4096, 264, 520, "squared_relu"), (130, 4096, 256, "silu"), (16, 2048, 4096, "gelu_tanh"),
                                          (1, 4096, 8192, "silu"), (3, 1024, 16384, "gelu")])
def test_larger(rows, H, d, act):
    print(f"feed forward {act} {rows}x{H}x{d}", flush=True)
    check(rows, H, d, act, "bf16")


def test_no_rows():
    w_in, w_down = torch.randn(32, 16, device="cuda").bfloat16(), torch.randn(16, 16, device="cuda").bfloat16()
    x, kept = torch.empty(0, 16, device="cuda").bfloat16(), torch.empty(0, 32, device="cuda").bfloat16()
    y, z = ga.feed_forward_train(x, w_in, w_down)
    assert y.shape == (0, 16) and z.shape == (0, 32)
    dx, dw_in, dw_down = ga.feed_forward_backward(x, x, kept, w_in, w_down)
    assert dx.shape == (0, 16) and float(dw_in.abs().max()) == 0 and float(dw_down.abs().max()) == 0


def test_gradients_against_differences():
    """The kernels' own forward pass, differenced along random directions."""
    rng = np.random.default_rng(4)
    rows, H, d = 48, 64, 96
    inputs = _inputs(rng, rows, H, d, "silu", "fp16")
    s = {k: v[0].cuda() for k, v in inputs.items()}
    e = {k: v[1] for k, v in inputs.items()}
    _, kept = ga.feed_forward_train(s["x"], s["w_in"], s["w_down"])
    grads = ga.feed_forward_backward(s["dy"], s["x"], kept, s["w_in"], s["w_down"])
    exact = ff.backward("silu", e["dy"], e["x"], e["x"] @ e["w_in"].T, e["w_in"], e["w_down"], "fp32")
    for what, g, (g64, _, _) in zip(("x", "w_in", "w_down"), grads, exact):
        v = torch.from_numpy(rng.normal(0, 1, g.shape)).cuda()
        h, at, at64 = 2.0 ** -4, [], []
        for sign in (1, -1):
            # the step that fp16 really takes
            moved = dict(s, **{what: (s[what].double() + sign * h * v).half()})
            y = ga.feed_forward(moved["x"], moved["w_in"], moved["w_down"])
            at.append((float((y.double() * s["dy"].double()).sum()), moved[what].double()))
            m = {k: moved[k].double().cpu().numpy() for k in ("x", "w_in", "w_down")}
            at64.append((ff.forward("silu", m["x"], m["w_in"], m["w_down"], "fp32")[0] * e["dy"]).sum())
        slope, step = at[0][0] - at[1][0], at[0][1] - at[1][1]
        want = float((g.double() * step).sum())
        # The step is not small (that of w_in moves z by h sqrt(H) = 1/2), so a difference is off the slope by the
        # derivatives past the first: by exactly what the same difference of the fp64 forms is off at the same
        # inputs.  Beside that: y's rounding and h's in both passes (2^-11 each, independent, sqrt(2 rows H) of
        # them, y of rms below 1), and the gradient's three roundings (z, dz or h, its own).
        past = abs(at64[0] - at64[1] - (g64 * step.cpu().numpy()).sum())
        size = float((g.double() * step).norm())
        slack = 4 * 2.0 ** -11 * (2 * rows * H) ** 0.5 + 4 * 3 * 2.0 ** -11 * size + past
        assert abs(slope - want) <= slack, (what, slope, want, slack)
        assert size > 20 * 4 * 2.0 ** -11, what


def test_infinities_and_nans_stay_in_their_rows():
    rng = np.random.default_rng(6)
    s = {k: v[0].cuda() for k, v in _inputs(rng, 40, 64, 72, "silu", "bf16").items()}
    clean = ga.feed_forward(s["x"], s["w_in"], s["w_down"])
    x = s["x"].clone()
    x[7, 3], x[21, 60] = float("nan"), float("inf")
    y = ga.feed_forward(x, s["w_in"], s["w_down"])
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[[7, 21]] = False
    assert torch.equal(y[rows], clean[rows]) and bool(y[7].isnan().all()) and not bool(y[21].isfinite().any())
    y, kept = ga.feed_forward_train(s["x"], s["w_in"], s["w_down"])
    dx0 = ga.feed_forward_backward(s["dy"], s["x"], kept, s["w_in"], s["w_down"])[0]
    kept[11, 5] = float("nan")
    dx = ga.feed_forward_backward(s["dy"], s["x"], kept, s["w_in"], s["w_down"])[0]
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[11] = False
    assert torch.equal(dx[rows], dx0[rows]) and bool(dx[11].isnan().all())


@pytest.mark.parametrize("rows,H,d", [(4, 256, 512), (300, 512, 264), (2200, 1024, 1024)])
def test_same_bits_every_time_and_in_graphs(rows, H, d):
    """A training step captured and replayed, with other work on the same stream between the replays, on new
    inputs, and on a second stream."""
    rng = np.random.default_rng(9)
    s = {k: v[0].cuda() for k, v in _inputs(rng, rows, H, d, "silu", "bf16").items()}

    def step(x):
        y, kept = ga.feed_forward_train(x, s["w_in"], s["w_down"])
        return (y, kept) + tuple(ga.feed_forward_backward(s["dy"], x, kept, s["w_in"], s["w_down"]))

    x = s["x"].clone()
    first = [t.clone() for t in step(x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(x), first):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(x)
    for i in range(4):
        x.copy_(s["x"] if i % 2 == 0 else s["dy"])
        graph.replay()
        eager = step(x)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), i
    for a, b in zip(step(s["x"]), first):
        assert torch.equal(a, b)


def test_workspace_of_the_callers():
    rng = np.random.default_rng(11)
    s = {k: v[0].cuda() for k, v in _inputs(rng, 60, 128, 256, "gelu", "bf16").items()}
    want, kept = ga.feed_forward_train(s["x"], s["w_in"], s["w_down"], "gelu")
    grads = ga.feed_forward_backward(s["dy"], s["x"], kept, s["w_in"], s["w_down"], "gelu")
    for need, call, expect in (
            (ga.feed_forward_workspace_bytes(60, 128, 256, "gelu"),
             lambda w: (ga.feed_forward(s["x"], s["w_in"], s["w_down"], "gelu", workspace=w),), (want,)),
            (ga.feed_forward_backward_workspace_bytes(60, 128, 256, "gelu"),
             lambda w: ga.feed_forward_backward(s["dy"], s["x"], kept, s["w_in"], s["w_down"], "gelu", workspace=w), grads)):
        buf = torch.full((need + 512,), PAD, dtype=torch.uint8, device="cuda")
        for a, b in zip(call(buf[:need]), expect):
            assert torch.equal(a, b)
        assert bool((buf[need:] == PAD).all())
        with pytest.raises(ga.GaError):
            call(buf[:need - 1])


def test_arguments():
    x, w_in, w_down = (torch.randn(*s, device="cuda").bfloat16() for s in ((4, 64), (64, 64), (64, 32)))
    ga.feed_forward(x, w_in, w_down)
    for bad in (dict(x=x.float()), dict(x=x.t()), dict(x=x[:, ::2]), dict(w_in=w_in[:63]), dict(w_in=w_in.half()),
                dict(w_down=w_down[:, :16]), dict(w_down=w_down.t()), dict(w_in=None), dict(w_down=None), dict(w_in=w_in.cpu()),
                dict(live_rows=torch.tensor([4], device="cuda")), dict(out=x.float()), dict(activation="gelu_sparse")):
        with pytest.raises(ValueError):
            ga.feed_forward(**{**dict(x=x, w_in=w_in, w_down=w_down), **bad})
    with pytest.raises(ga.GaError):
        ga.feed_forward(x, w_in, w_down, out=x)
    off = torch.randn(4 * 64 + 1, device="cuda").bfloat16()[1:].view(4, 64)
    with pytest.raises(ga.GaError):
        ga.feed_forward(off, w_in, w_down)
    kept = torch.randn(4, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        ga.feed_forward_backward(x, x, kept[:, :32].contiguous(), w_in, w_down)
    with pytest.raises(ValueError):
        ga.feed_forward_backward(x, x, None, w_in, w_down)
