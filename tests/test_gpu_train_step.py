"""The training operators together, as a layer uses them (needs an MI355X): an
expert feed-forward step with the norm, the router and the bounded activation;
graphs, streams and workspaces."""
import numpy as np
import pytest
import torch

import gated_activation_amd as ga

pytestmark = pytest.mark.gpu
ROWS, D, F, E, K = 256, 192, 320, 8, 2
CAPACITY = ROWS * K + 64


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * std

    return {"x": t(ROWS, D, std=2.0) + 0.3, "w": 1 + 0.1 * t(D), "b": 0.1 * t(D), "router": t(E, D, std=D ** -0.5),
            "up": t(E, 2 * F, D, std=D ** -0.5), "down": t(E, D, F, std=F ** -0.5), "dy": t(ROWS, D)}


def _sorted_rows(index, counts_len):
    """Rows of the expert-sorted buffer: the token of each, by expert, then by token."""
    flat = index.reshape(-1)
    order = torch.argsort(flat, stable=True)
    return order // index.shape[1], flat[order]


def _step(p, activation, keep):
    """One forward and backward pass; keep: activations in 8 bits.  Returns the gradients."""
    if keep:
        n, nc = ga.layer_norm_checkpoint(p["x"], p["w"], p["b"])
    else:
        n, st = ga.layer_norm(p["x"], p["w"], p["b"])
    logits = n @ p["router"].t()
    index = torch.topk(logits, K, dim=1).indices
    bal = ga.balance_loss(logits, index, 0.05)
    token, expert = _sorted_rows(index, E)
    live = bal.offsets[-1:]
    gate_up = torch.zeros(CAPACITY, 2 * F, device="cuda")
    gate_up[:ROWS * K] = torch.bmm(p["up"][expert].contiguous(), n[token].unsqueeze(2)).squeeze(2)
    a = torch.zeros(CAPACITY, F, device="cuda")
    kept_gate_up = gate_up
    if keep:
        a, kept_gate_up = ga.activation_checkpoint(gate_up, activation, live_rows=live, out=a)
        kept_a = ga.checkpoint_store(a, live_rows=live)
    else:
        a, _ = ga.activation_checkpoint(gate_up, activation, live_rows=live, out=a)
    y = torch.zeros(ROWS, D, device="cuda")
    part = torch.bmm(p["down"][expert].contiguous(), a[:ROWS * K].unsqueeze(2)).squeeze(2)
    y.index_add_(0, token, part)
    # backward, the gates of the router's choice left out
    dpart = p["dy"][token]
    a_back = ga.checkpoint_restore(kept_a, torch.float32, live_rows=live)[:ROWS * K] if keep else a[:ROWS * K]
    ddown = torch.zeros_like(p["down"]).index_add_(0, expert, dpart.unsqueeze(2) * a_back.unsqueeze(1))
    da = torch.zeros(CAPACITY, F, device="cuda")
    da[:ROWS * K] = torch.bmm(p["down"][expert].transpose(1, 2).contiguous(), dpart.unsqueeze(2)).squeeze(2)
    dgate_up = ga.activation_backward(da, kept_gate_up, activation, live_rows=live,
                                      out=torch.zeros(CAPACITY, 2 * F, device="cuda"))[:ROWS * K]
    dlogits = ga.balance_loss_backward(logits, bal, dloss=torch.tensor(2.0, device="cuda"))
    dn = dlogits @ p["router"]
    dn.index_add_(0, token, torch.bmm(p["up"][expert].transpose(1, 2).contiguous(), dgate_up.unsqueeze(2)).squeeze(2))
    dx, dw, db = ga.layer_norm_backward(dn, nc, p["w"]) if keep else ga.layer_norm_backward(dn, p["x"], p["w"], stats=st)
    return {"y": y, "loss": bal.loss, "dx": dx, "dw": dw, "db": db, "drouter": dlogits.t() @ n, "ddown": ddown}, index


def _plain(p, activation, index):
    """The same step by autograd in fp64 on the CPU, the router's choice given."""
    q = {k: v.double().cpu().requires_grad_(k != "dy") for k, v in p.items()}
    index = index.cpu()
    x = q["x"]
    mean = x.mean(1, keepdim=True)
    n = (x - mean) / (((x - mean) ** 2).mean(1, keepdim=True) + 1e-5).sqrt() * q["w"] + q["b"]
    logits = n @ q["router"].t()
    counts = torch.bincount(index.reshape(-1), minlength=E).double()
    loss = 0.05 * E / (K * ROWS) * (counts * torch.softmax(logits, 1).mean(0)).sum()
    token, expert = _sorted_rows(index, E)
    h = torch.bmm(q["up"][expert], n[token].unsqueeze(2)).squeeze(2)
    gate, up = h[:, :F], h[:, F:]
    if activation == "silu":
        a = gate * torch.sigmoid(gate) * up
    else:
        m = gate.mean(1, keepdim=True)
        s = ((gate - m) ** 2).mean(1, keepdim=True).sqrt()
        t = torch.relu(gate - m - ga.Z_SPARSITY_095 * s)
        a = 0.5 * t * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (t + 0.044715 * t ** 3))) * up
    y = torch.zeros(ROWS, D, dtype=torch.float64).index_add(0, token, torch.bmm(q["down"][expert], a.unsqueeze(2)).squeeze(2))
    ((y * q["dy"]).sum() + 2.0 * loss).backward()
    return {"y": y.detach(), "loss": loss.detach(), "dx": q["x"].grad, "dw": q["w"].grad, "db": q["b"].grad,
            "drouter": None, "ddown": q["down"].grad}


@pytest.mark.parametrize("activation", ["silu", "gelu_sparse"])
def test_expert_layer_step(activation):
    """Gradients of a whole step.  fp32 throughout: products of up to 320 terms and the kernels' bounds give
    relative errors of 1e-6 or so in the 2-norm.  In 8 bits a value is off by at most half a step, m / 254, with m
    about 2.8 times the rms of normal values (largest of 128); the sparse form keeps gate - cutoff, whose largest
    is 1.64 (the multiplier) further out.  Gradients are products of two such values and slopes of about 1, over
    values that are smaller than their block's rms in the sparse form: a whole step, relative, covers them."""
    p = _inputs(3)
    want = None
    for keep, most in ((False, 2e-5), (True, (2.8 + (1.65 if activation == "gelu_sparse" else 0.0)) / 127)):
        got, index = _step(p, activation, keep)
        torch.cuda.synchronize()
        want = want or _plain(p, activation, index)
        for name, w in want.items():
            if w is None:
                continue
            g = got[name].double().cpu()
            rel = float((g - w).norm() / w.norm())
            # forward results do not go through 8 bits; the sparse form's slope jumps at the cutoff, where no
            # value may change sides, so its gradients are held to the same bound
            limit = 2e-5 if name in ("y", "loss") else most
            assert rel <= limit, f"{activation} keep {keep} {name}: {rel:.3g} > {limit:.3g}"


def _everything(p16, buf):
    """Every operator once, into preallocated outputs where it has them."""
    out, c = ga.activation_checkpoint(p16["gu"], "gelu_sparse", live_rows=p16["live"], out=buf["out"], checkpoint=buf["kept"])
    dx = ga.activation_backward(p16["dout"], c, "gelu_sparse", live_rows=p16["live"], out=buf["dgu"])
    dx2 = ga.activation_backward(p16["dout"], p16["gu"], "silu", live_rows=p16["live"], out=buf["dgu2"])
    y, nc = ga.layer_norm_checkpoint(p16["x"], p16["w"], p16["w"])
    nx, dw, db = ga.layer_norm_backward(p16["dy"], nc, p16["w"])
    bal = ga.balance_loss(p16["logits"], p16["index"], live_rows=p16["live"])
    dl = ga.balance_loss_backward(p16["logits"], bal, live_rows=p16["live"], out=buf["dlogits"])
    back = ga.checkpoint_restore(ga.checkpoint_store(p16["x"]), torch.bfloat16)
    return [out, dx, dx2, y, nx, dw, db, bal.loss, bal.counts, bal.offsets, dl, back]


def _everything_inputs(seed, rows=600):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    p = {"gu": r(rows, 2 * 768), "dout": r(rows, 768), "x": r(rows, 1500), "dy": r(rows, 1500), "w": r(1500),
         "logits": r(rows, 128), "live": torch.tensor([rows], dtype=torch.int32, device="cuda")}
    p["index"] = torch.topk(p["logits"].float(), 4, dim=1).indices
    return p


def _buffers(rows=600):
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    return {"out": z(rows, 768), "dgu": z(rows, 1536), "dgu2": z(rows, 1536), "dlogits": z(rows, 128),
            "kept": ga.Checkpoint(z(rows, 2, 768, t=torch.int8), z(rows, 2, 6, t=torch.float32), z(rows, 2, t=torch.float32))}


def test_graph_replays():
    """Captured once, replayed with other inputs and live counts, eager work and synchronisation in between; two
    graphs of the same stream in turn, so that what one leaves does not reach the other."""
    p, buf = _everything_inputs(1), _buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(p, buf)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        b = _buffers()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            res = _everything(p, b)
        graphs.append((graph, b, res))
    for turn, live in enumerate([600, 17, 0, 599, 600]):
        fresh = _everything_inputs(10 + turn)
        for k in p:
            p[k].copy_(fresh[k])
        p["live"].fill_(live)
        e = _buffers()
        want = _everything(p, e)
        torch.cuda.synchronize()
        for graph, b, res in graphs:
            for t in (b["out"], b["dgu"], b["dgu2"], b["dlogits"]):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for i, (a, w) in enumerate(zip(res, want)):
                assert torch.equal(a, w), f"replay {turn} live {live} output {i}"


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    ps = [_everything_inputs(30 + i) for i in range(2)]
    want = [[t.clone() for t in _everything(p, _buffers())] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [[_buffers() for _ in range(3)] for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for turn in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_everything(ps[i], bufs[i][turn]))
    torch.cuda.synchronize()
    for i in range(2):
        for res in got[i]:
            for k, (a, w) in enumerate(zip(res, want[i])):
                assert torch.equal(a, w), f"stream {i} output {k}"


def test_tensors_on_a_device_that_is_not_current(monkeypatch):
    """The binding makes the tensors' device current for the launch (here told that another one is)."""
    from gated_activation_amd import _train
    p, b = _everything_inputs(5), _buffers()
    want = [t.clone() for t in _everything(p, b)]
    monkeypatch.setattr(_train, "_current_device", lambda: -1)
    got = _everything(p, _buffers())
    torch.cuda.synchronize()
    for a, w in zip(got, want):
        assert torch.equal(a, w)


def test_empty_arrays():
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    for act in ga.ACTIVATIONS:
        h = 1 if act == "squared_relu" else 2
        out, c = ga.activation_checkpoint(z(0, h * 8), act)
        assert out.shape == (0, 8) and ga.activation_backward(z(0, 8), c, act).shape == (0, h * 8)
        assert ga.activation_backward(z(0, 8), z(0, h * 8), act).shape == (0, h * 8)
    assert ga.checkpoint_restore(ga.checkpoint_store(z(0, 5)), torch.float32).shape == (0, 5)
    y, st = ga.layer_norm(z(0, 9), z(9), z(9))
    dx, dw, db = ga.layer_norm_backward(z(0, 9), z(0, 9), z(9) + 1, stats=st)
    assert y.shape == (0, 9) and dx.shape == (0, 9) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0
    b = ga.balance_loss(z(0, 4), z(0, 2, t=torch.int64))
    assert float(b.loss) == 0 and b.counts.tolist() == [0] * 4 and b.offsets.tolist() == [0] * 5
    assert ga.balance_loss_backward(z(0, 4), b).shape == (0, 4)
    torch.cuda.synchronize()


def test_refusals_on_the_device():
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x = z(4, 16)
    with pytest.raises(ValueError):
        ga.activation_checkpoint(z(4, 32)[:, ::2], "silu")                       # strided
    with pytest.raises(ValueError):
        ga.activation_backward(z(4, 8), z(4, 16, t=torch.float16), "silu")       # another type
    with pytest.raises(ValueError):
        ga.activation_backward(z(4, 8), ga.checkpoint_store(x), "silu")          # one half where two are needed
    with pytest.raises(ValueError):
        ga.activation_backward(z(4, 8), ga.Checkpoint(z(4, 2, 8, t=torch.int8), z(4, 2, 1)), "gelu_sparse")  # no stats
    for act, kept in (("silu", ga.activation_checkpoint(z(4, 32), "gelu_sparse")[1]),
                      ("squared_relu", ga.layer_norm_checkpoint(x, z(16))[1])):  # codes relative to their rows
        with pytest.raises(ValueError):
            ga.activation_backward(x, kept, act)
    with pytest.raises(ga.GaError):
        ga.activation_backward(x, x, "squared_relu", out=x)                      # in place
    with pytest.raises(ValueError):
        ga.layer_norm(x, z(16, t=torch.float16))
    with pytest.raises(ga.GaError):
        ga.layer_norm(x, z(16), eps=float("nan"))
    with pytest.raises(ga.GaError):
        ga.layer_norm(z(1, 32769), z(32769))
    with pytest.raises(ValueError):
        ga.layer_norm_backward(x, x, z(16))                                      # no stats
    with pytest.raises(ga.GaError):
        ga.layer_norm_backward(z(64, 8192), z(64, 8192), z(8192), stats=z(64, 2), workspace=z(16, t=torch.uint8))
    with pytest.raises(ga.GaError):
        ga.balance_loss(z(2, 1025), z(2, 1, t=torch.int64))
    with pytest.raises(ValueError):
        ga.balance_loss(x, z(4, 2))                                              # indices that are not integers
    with pytest.raises(ValueError):
        ga.balance_loss(x, z(4, 2, t=torch.int32), mask=z(3, t=torch.bool))
    torch.cuda.synchronize()
    assert np.isfinite(x.cpu().numpy()).all()
