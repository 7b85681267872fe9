"""The training operators around the gated activations, as measured cases.

Three operators, each forward and backward:

  activation checkpoints   an array kept in 8 bits for the backward pass: blocks
                           of 128 values along a row (the gate half and the up
                           half are blocked apart), one fp32 scale a block,
                           code = round(x * 127 / max|x|).  Written by the gated
                           activations' forward pass and read by their backward.
  layer norm               the norm in front of the layer: y, then dx and the
                           reduced gradients of the weight and the bias, from x
                           or from x - mean kept in 8 bits.
  balance loss             the router's loss E / (k n) sum_e counts_e P_e over n
                           tokens, the per-expert counts and offsets that bound
                           the experts' buffers, and the logits' gradient.

`run` computes them with elementary torch operations in 32 bits (64 where a
value is compared with a row's cutoff, or rounded to a code) where `own` is false, and by the calls of
gated_activation_amd where it is true.
"""
import math

import torch

own = False

BLOCK = 128                  # values of one scale
LEAST = 2.0 ** -100          # a block's largest magnitude counts as at least this
Z = 1.6448536                # Phi^-1(0.95), the sparse form's cutoff multiplier
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # An expert's buffer of a mixture-of-experts layer in training: capture-sized,
        # three quarters of it live, forward with the kept gate | up and its backward.
        {"name": "silu_step_16384x768_live", "op": "activation_step", "act": "silu", "dtype": "bf16", "rows": 16384,
         "d": 768, "live": 12288},
        # The sparse feed-forward activation at the library's headline size, one training step.
        {"name": "sparse_step_2048x16384", "op": "activation_step", "act": "gelu_sparse", "dtype": "bf16", "rows": 2048,
         "d": 16384, "live": -1},
        # A few tokens of a small layer: what a step costs when launches are all of it.
        {"name": "gelu_step_16x2048", "op": "activation_step", "act": "gelu_tanh", "dtype": "bf16", "rows": 16,
         "d": 2048, "live": -1},
        # The sparse activation's backward where gate | up is kept whole.
        {"name": "sparse_backward_2048x8192", "op": "activation_backward", "act": "gelu_sparse", "dtype": "bf16",
         "rows": 2048, "d": 8192, "live": -1},
        # Rows off 16-byte alignment, the exact GELU in half precision.
        {"name": "gelu_backward_1023x4099_fp16", "op": "activation_backward", "act": "gelu", "dtype": "fp16",
         "rows": 1023, "d": 4099, "live": -1},
        # The down projection's input kept for its weight gradient: stored, then read back.
        {"name": "checkpoint_4096x16384", "op": "checkpoint", "dtype": "bf16", "rows": 4096, "d": 16384, "live": -1},
        # The norm in front of the layer, a batch of sequences, forward only.
        {"name": "layer_norm_16384x2048", "op": "layer_norm", "dtype": "bf16", "wdtype": "bf16", "rows": 16384, "d": 2048,
         "live": -1},
        # One token of a decode loop.
        {"name": "layer_norm_1x4096", "op": "layer_norm", "dtype": "bf16", "wdtype": "bf16", "rows": 1, "d": 4096,
         "live": -1},
        # A training step of the norm with its centred rows in 8 bits.
        {"name": "layer_norm_step_8192x4096", "op": "layer_norm_step", "dtype": "bf16", "wdtype": "bf16", "rows": 8192,
         "d": 4096, "live": -1},
        # Single precision, odd rows and columns, weights in single precision.
        {"name": "layer_norm_backward_4001x1027_fp32", "op": "layer_norm_backward", "dtype": "fp32", "wdtype": "fp32",
         "rows": 4001, "d": 1027, "live": -1},
        # A router over 128 experts, eight a token, a batch with some padding tokens.
        {"name": "balance_16384x128_top8", "op": "balance", "dtype": "bf16", "rows": 16384, "experts": 128, "k": 8,
         "masked": True},
        # A small router in single precision.
        {"name": "balance_64x8_top2", "op": "balance", "dtype": "fp32", "rows": 64, "experts": 8, "k": 2, "masked": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["activation_step", "activation_step", "activation_backward", "activation_backward", "checkpoint",
                     "layer_norm", "layer_norm_step", "layer_norm_backward", "balance", "balance"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "balance":
        experts = _log(rng, 2, 1024)
        rows = min(_log(rng, 8, 65536), (1 << 23) // experts)
        # fewer choices than experts: with all of them every count is the same and there is no gradient
        return {"op": op, "dtype": dtype, "rows": rows, "experts": experts, "k": rng.randint(1, max(1, min(experts // 2, 8))),
                "masked": rng.random() < 0.5}
    norm = op.startswith("layer_norm")
    d = _log(rng, 64, 32768)
    if rng.random() < 0.6:
        d = -(-d // 64) * 64
    rows = min(_log(rng, 1, 32768), (1 << 25 if dtype != "fp32" else 1 << 24) // d)
    live = rng.randint(1, rows) if rng.random() < 0.3 else -1
    case = {"op": op, "dtype": dtype, "rows": rows, "d": d, "live": live}
    if norm:
        case["wdtype"] = dtype if op == "layer_norm_step" or rng.random() < 0.7 else "fp32"
    elif op != "checkpoint":
        case["act"] = rng.choice(["silu", "gelu_tanh", "gelu", "gelu_sparse", "gelu_sparse", "squared_relu"])
    return case


def _halves(case):
    return 1 if case["op"] == "checkpoint" or case.get("act") == "squared_relu" else 2


def _blocks(d):
    return -(-d // BLOCK)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows, op = case["rows"], case["op"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=g) * std + mean).to(dtype)

    s = {"case": case, "op": op, "dtype": dt}
    if op == "balance":
        e = case["experts"]
        # experts of unequal popularity, as a router has before it is balanced
        s["logits"] = (torch.randn(rows, e, device="cuda", generator=g)
                       + torch.randn(e, device="cuda", generator=g) * 0.5).to(dt)
        s["experts"] = torch.topk(s["logits"].float(), case["k"], dim=1).indices
        s["mask"] = torch.rand(rows, device="cuda", generator=g) < 0.9 if case["masked"] else None
        # the gradient falls with the tokens' number: half precision trains with a scaled loss
        s["dloss"] = (torch.rand((), device="cuda", generator=g) + 0.5) * (65536.0 if dt == torch.float16 else 1.0)
        return s
    d = case["d"]
    live = rows if case["live"] < 0 else case["live"]
    s["live"] = None if case["live"] < 0 else torch.tensor([live], dtype=torch.int32, device="cuda")
    s["keep"] = None if s["live"] is None else torch.arange(rows, device="cuda")[:, None] < s["live"]
    if op == "checkpoint":
        # an activation's output: mostly small, some large
        s["x"] = (torch.randn(rows, d, device="cuda", generator=g)
                  * torch.randn(rows, d, device="cuda", generator=g)).to(dt)
        s["out"] = torch.zeros(rows, d, dtype=dt, device="cuda")
        s["codes"], s["scales"] = _empty_checkpoint(rows, 1, d)
        return s
    if op in ("activation_step", "activation_backward"):
        s["act"] = case["act"]
        h = _halves(case)
        s["x"] = normal(rows, h * d, std=1.5)
        s["dout"] = normal(rows, d)
        s["dx"] = torch.zeros(rows, h * d, dtype=dt, device="cuda")
        if op == "activation_step":
            s["out"] = torch.zeros(rows, d, dtype=dt, device="cuda")
            s["codes"], s["scales"] = _empty_checkpoint(rows, h, d)
            s["stats"] = torch.zeros(rows, 2, device="cuda") if case["act"] == "gelu_sparse" else None
        return s
    wdt = DTYPES[case["wdtype"]]
    s["x"] = normal(rows, d, mean=0.3, std=2.0)
    s["weight"], s["bias"] = normal(d, mean=1.0, std=0.2, dtype=wdt), normal(d, std=0.2, dtype=wdt)
    if op != "layer_norm_backward":
        s["out"] = torch.zeros(rows, d, dtype=dt, device="cuda")
    if op != "layer_norm":
        s["dy"] = normal(rows, d)
        s["dx"] = torch.zeros(rows, d, dtype=dt, device="cuda")
    if op == "layer_norm_step":
        s["codes"], s["scales"] = _empty_checkpoint(rows, 1, d)
    if op == "layer_norm":
        s["stats"] = torch.zeros(rows, 2, device="cuda")
    elif op == "layer_norm_step":
        s["stats"] = torch.zeros(rows, 2, device="cuda")
    else:  # what the forward pass left behind
        x = s["x"].float()
        s["stats"] = torch.stack([x.mean(1), torch.rsqrt(x.var(1, unbiased=False) + EPS)], dim=1)
    return s


def _empty_checkpoint(rows, halves, d):
    shape = (rows, d) if halves == 1 else (rows, halves, d)
    return (torch.zeros(shape, dtype=torch.int8, device="cuda"),
            torch.zeros(*shape[:-1], _blocks(d), device="cuda"))


# ---- the calls of the library -------------------------------------------------

def _own_run(s):
    import gated_activation_amd as ga
    op = s["op"]
    if op == "balance":
        b = ga.balance_loss(s["logits"], s["experts"], mask=s["mask"])
        dlogits = ga.balance_loss_backward(s["logits"], b, dloss=s["dloss"], mask=s["mask"])
        return b.loss, b.counts, b.offsets, dlogits
    live = s["live"]
    if op == "checkpoint":
        c = ga.checkpoint_store(s["x"], live_rows=live, checkpoint=ga.Checkpoint(s["codes"], s["scales"]))
        return ga.checkpoint_restore(c, s["dtype"], live_rows=live, out=s["out"])
    if op == "activation_step":
        kept = ga.Checkpoint(s["codes"], s["scales"], s["stats"])
        out, kept = ga.activation_checkpoint(s["x"], s["act"], z=Z, live_rows=live, out=s["out"], checkpoint=kept)
        return out, ga.activation_backward(s["dout"], kept, s["act"], z=Z, live_rows=live, out=s["dx"])
    if op == "activation_backward":
        return ga.activation_backward(s["dout"], s["x"], s["act"], z=Z, live_rows=live, out=s["dx"])
    if op == "layer_norm":
        return ga.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, live_rows=live, out=s["out"], stats=s["stats"])
    if op == "layer_norm_step":
        kept = ga.Checkpoint(s["codes"], s["scales"], s["stats"])
        y, kept = ga.layer_norm_checkpoint(s["x"], s["weight"], s["bias"], eps=EPS, live_rows=live, out=s["out"],
                                           checkpoint=kept)
        return (y,) + tuple(ga.layer_norm_backward(s["dy"], kept, s["weight"], live_rows=live, out=s["dx"]))
    return ga.layer_norm_backward(s["dy"], s["x"], s["weight"], stats=s["stats"], live_rows=live, out=s["dx"])


# ---- the plain forms ----------------------------------------------------------

def _pass_live(s, value, into):
    """`value` in the live rows, the others as they were."""
    value = value.to(into.dtype)
    return value if s["keep"] is None else torch.where(s["keep"], value, into)


def _store(t, active=None):
    """Codes and scales of fp32 rows [..., d] in blocks of 128 along the last axis; where `active`
    is given, its values stay above zero."""
    d = t.shape[-1]
    pad = _blocks(d) * BLOCK - d
    t = torch.nn.functional.pad(t, (0, pad)).unflatten(-1, (-1, BLOCK))
    top = t.abs().amax(-1, keepdim=True).clamp(min=LEAST)
    codes = (t.double() * 127.0 / top.double()).round()
    if active is not None:
        active = torch.nn.functional.pad(active, (0, pad)).unflatten(-1, (-1, BLOCK))
        codes = torch.where(active, codes.clamp(min=1.0), codes)
    return codes.to(torch.int8), top / 127.0, d


def _restore(kept):
    codes, scales, d = kept
    return (codes.float() * scales).flatten(-2)[..., :d]


def _gate_gradient(act, g):
    """The activation's value and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if act == "squared_relu":
        r = g.clamp(min=0.0)
        return r * r, 2.0 * r
    c, k = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(c * (g + k * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * k * g * g)


def _split(x, d):
    return x[:, :d].float(), x[:, d:].float()


def _sparse_statistics(gate):
    g = gate.double()
    mean = g.mean(1, keepdim=True)
    std = torch.sqrt((g - mean).square().mean(1, keepdim=True))
    cutoff = mean + Z * std
    return (g - cutoff).float(), std.float()


def _sparse_backward(dout, t, std, up):
    """Gradients of gelu(max(t, 0)) * up, t = gate - mean - Z std, through the row's mean and std."""
    value, slope = _gate_gradient("gelu_tanh", t.clamp(min=0.0))
    g = torch.where(t > 0, dout * up * slope, torch.zeros_like(t))
    d = t.shape[1]
    spread = torch.where(std > 0, Z * (t + Z * std) / std, torch.zeros_like(t))
    return torch.cat([g - g.sum(1, keepdim=True) * (1.0 + spread) / d, dout * value], dim=1)


def _plain_backward(act, dout, parts):
    if act == "squared_relu":
        return dout * _gate_gradient(act, parts[0])[1]
    value, slope = _gate_gradient(act, parts[0])
    return torch.cat([dout * parts[1] * slope, dout * value], dim=1)


def _norm_backward(s, n, rstd):
    dy = s["dy"].float()
    if s["keep"] is not None:
        dy = torch.where(s["keep"], dy, torch.zeros_like(dy))
    dn = dy * s["weight"].float()
    dx = rstd * (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True))
    wdt = s["weight"].dtype
    return _pass_live(s, dx, s["dx"]), (dy * n).sum(0).to(wdt), dy.sum(0).to(wdt)


def _plain_run(s):
    op = s["op"]
    if op == "balance":
        return _plain_balance(s)
    x = s["x"].float()
    if op == "checkpoint":
        return _pass_live(s, _restore(_store(x)), s["out"])
    if op.startswith("layer_norm"):
        if op == "layer_norm_backward":
            mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
            return _norm_backward(s, (x - mean) * rstd, rstd)
        if op == "layer_norm_step":
            mean = x.double().mean(1, keepdim=True)
            centred = (x.double() - mean).float()
            rstd = torch.rsqrt(centred.square().mean(1, keepdim=True) + EPS)
        else:
            mean = x.mean(1, keepdim=True)
            centred = x - mean
            rstd = torch.rsqrt(centred.square().mean(1, keepdim=True) + EPS)
        n = centred * rstd
        y = _pass_live(s, n * s["weight"].float() + s["bias"].float(), s["out"])
        if op == "layer_norm":
            return y, _pass_live(s, torch.cat([mean, rstd], dim=1), s["stats"])
        return (y,) + _norm_backward(s, _restore(_store(centred)) * rstd, rstd)
    act, dout, d = s["act"], s["dout"].float(), s["dout"].shape[1]
    if act == "squared_relu":
        if op == "activation_backward":
            return _pass_live(s, _plain_backward(act, dout, (x,)), s["dx"])
        return (_pass_live(s, _gate_gradient(act, x)[0], s["out"]),
                _pass_live(s, _plain_backward(act, dout, (_restore(_store(x)),)), s["dx"]))
    gate, up = _split(x, d)
    if act == "gelu_sparse":
        t, std = _sparse_statistics(gate)
        if op == "activation_backward":
            return _pass_live(s, _sparse_backward(dout, t, std, up), s["dx"])
        out = _gate_gradient("gelu_tanh", t.clamp(min=0.0))[0] * up
        dx = _sparse_backward(dout, _restore(_store(t, t > 0)), std, _restore(_store(up)))
        return _pass_live(s, out, s["out"]), _pass_live(s, dx, s["dx"])
    if op == "activation_backward":
        return _pass_live(s, _plain_backward(act, dout, (gate, up)), s["dx"])
    out = _gate_gradient(act, gate)[0] * up
    dx = _plain_backward(act, dout, (_restore(_store(gate)), _restore(_store(up))))
    return _pass_live(s, out, s["out"]), _pass_live(s, dx, s["dx"])


def _plain_balance(s):
    logits, experts, mask = s["logits"].float(), s["experts"], s["mask"]
    e, k = logits.shape[1], experts.shape[1]
    if mask is None:
        mask = torch.ones(logits.shape[0], dtype=torch.bool, device=logits.device)
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * mask[:, None]
    chosen = (mask[:, None].expand_as(experts)).reshape(-1).to(torch.int32)
    counts = torch.zeros(e, dtype=torch.int32, device=logits.device).index_add_(0, experts.reshape(-1), chosen)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0).to(torch.int32)])
    n = mask.sum().clamp(min=1).float()
    share = p.sum(0) / n
    factor = e / (k * n)
    loss = factor * (counts.float() * share).sum()
    # sum_j p_j = 1, so the counts may be taken from their mean, where less cancels
    off = counts.float() - counts.float().mean()
    dlogits = s["dloss"] * (factor / n) * p * (off - (p * off).sum(1, keepdim=True))
    return loss, counts, offsets, dlogits.to(s["dtype"])


def run(s):
    if own:
        return _own_run(s)
    return _plain_run(s)


def work(case):
    rows = case["rows"]
    es = 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op == "balance":
        n = rows * case["experts"]
        # logits read in either direction (the loss' gradient needs all counts first), indices, gradient written
        return {"bytes": n * es * 3 + rows * case["k"] * 8 + rows * case["masked"] * 2 + case["experts"] * 8,
                "flops": 12 * n}
    d = case["d"]
    live = rows if case["live"] < 0 else case["live"]
    n = max(1, live) * d
    kept = 1 + 4 / BLOCK          # bytes of a value kept in 8 bits
    if op == "checkpoint":
        return {"bytes": n * (2 * es + 2 * kept), "flops": 4 * n}
    if op.startswith("layer_norm"):
        wes = 4 if case["wdtype"] == "fp32" else 2
        forward = n * 2 * es + 2 * d * wes + 8 * max(1, live)
        if op == "layer_norm":
            return {"bytes": forward, "flops": 8 * n}
        back = 3 * d * wes + 8 * max(1, live)
        if op == "layer_norm_backward":
            return {"bytes": n * 3 * es + back, "flops": 14 * n}
        return {"bytes": forward + n * kept + n * (2 * es + kept) + back, "flops": 26 * n}
    h = _halves(case)
    if op == "activation_backward":
        return {"bytes": n * es * (1 + 2 * h), "flops": 30 * n}
    return {"bytes": n * (es * (h + 1) + kept * h) + n * (es * (1 + h) + kept * h), "flops": 60 * n}


# ---- 64 bits ------------------------------------------------------------------

def _kept64(v, positive=None):
    """What 8 bits keep of v [rows, d]: block by block along the rows, in 64 bits.  A value relative to
    its row (x - mean, gate - cutoff) is by definition rounded to fp32 before it is coded."""
    rows, d = v.shape
    whole = v.new_zeros(rows, _blocks(d) * BLOCK)
    whole[:, :d] = v
    whole = whole.view(rows, _blocks(d), BLOCK)
    step = whole.abs().max(dim=2, keepdim=True).values.clamp(min=LEAST) / 127
    q = torch.round(whole / step).view(rows, -1)[:, :d]
    if positive is not None:
        q[positive & (q < 1)] = 1
    return q * step.expand_as(whole).reshape(rows, -1)[:, :d]


def _value64(act, g):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return g * torch.special.ndtr(g)
    if act == "squared_relu":
        return torch.relu(g) ** 2
    u = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(u)  # (1 + tanh(u / 2)) / 2


def _gradient64(f, inputs, dout):
    with torch.enable_grad():
        leaves = [v.detach().clone().requires_grad_(True) for v in inputs]
        return torch.autograd.grad(f(*leaves), leaves, dout)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        return _balance64(s)
    live = case["rows"] if case["live"] < 0 else case["live"]
    x = s["x"][:live].double()

    def padded(v, width):
        whole = torch.zeros(case["rows"], width, dtype=torch.float64, device="cuda")
        whole[:live] = v
        return whole

    d = case["d"]
    if op == "checkpoint":
        return padded(_kept64(x), d)
    if op.startswith("layer_norm"):
        w, b = s["weight"].double(), s["bias"].double()
        if op == "layer_norm_backward":
            mean, rstd = s["stats"][:live, :1].double(), s["stats"][:live, 1:].double()
        else:
            mean = x.sum(1, keepdim=True) / d
            rstd = ((x - mean).pow(2).sum(1, keepdim=True) / d + EPS).pow(-0.5)
        n = (x - mean) * rstd
        y = padded(n * w + b, d)
        if op == "layer_norm":
            return y, padded(torch.cat([mean, rstd], 1), 2)
        if op == "layer_norm_step":
            n = _kept64((x - mean).float().double()) * rstd
        dy = s["dy"][:live].double()
        v = dy * w
        dx = (v - v.sum(1, keepdim=True) / d - n * ((v * n).sum(1, keepdim=True) / d)) * rstd
        back = padded(dx, d), (dy * n).sum(0), dy.sum(0)
        return back if op == "layer_norm_backward" else (y,) + back
    act, dout = case["act"], s["dout"][:live].double()
    step = op == "activation_step"
    if act == "squared_relu":
        dx, = _gradient64(lambda v: _value64(act, v), [_kept64(x) if step else x], dout)
        return (padded(_value64(act, x), d), padded(dx, d)) if step else padded(dx, d)
    gate, up = x[:, :d], x[:, d:]
    if act != "gelu_sparse":
        kept = [_kept64(gate), _kept64(up)] if step else [gate, up]
        dx = torch.cat(_gradient64(lambda g, u: _value64(act, g) * u, kept, dout), 1)
        return (padded(_value64(act, gate) * up, d), padded(dx, 2 * d)) if step else padded(dx, 2 * d)
    mean = gate.sum(1, keepdim=True) / d
    std = ((gate - mean) ** 2).sum(1, keepdim=True).div(d).sqrt()
    t = gate - mean - Z * std
    out = padded(_value64("gelu_tanh", torch.relu(t)) * up, d)
    if step:
        t, up = _kept64(t.float().double(), t > 0), _kept64(up)
    gt, gu = _gradient64(lambda v, u: _value64("gelu_tanh", torch.relu(v)) * u, [t, up], dout)
    total = gt.sum(1, keepdim=True)
    dgate = gt - total / d - total * Z / d * ((t + Z * std) / std)
    dx = padded(torch.cat([dgate, gu], 1), 2 * d)
    return (out, dx) if step else dx


def _balance64(s):
    logits, experts = s["logits"].double(), s["experts"]
    rows, e = logits.shape
    k = experts.shape[1]
    use = torch.ones(rows, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    counts = torch.bincount(experts[use].reshape(-1), minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    n = int(use.sum())
    if n == 0:
        return torch.zeros((), dtype=torch.float64, device="cuda"), counts.int(), offsets.int(), torch.zeros_like(logits)
    f = counts.double()
    loss = e / (k * n * n) * (f * torch.softmax(logits[use], 1).sum(0)).sum()
    # d softmax: p (c - <c, p>), of every token by itself
    p = torch.softmax(logits, 1)
    grad = e / (k * n * n) * p * (f - (p @ f)[:, None]) * use[:, None]
    return loss, counts.int(), offsets.int(), grad * s["dloss"].double()
