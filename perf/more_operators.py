"""The feed-forward layer's products around the gated activations, as measured
cases, in 16 bits and in microscaled 4 bits.

  feed forward     y = (act(x Wg^T) * (x Wu^T)) Wd^T with the gate's and up's rows
                   stacked in one weight, and its backward pass from the kept
                   gate | up: the input's and both weights' gradients.
  mxfp4            e2m1 values in blocks of 32 along a row, one power of two (E8M0)
                   a block: quantisation (of an array, or of an activation's
                   result), the product of two such arrays, and the feed-forward
                   layer on 4-bit operands.

`run` computes them with elementary torch operations in 32 bits where `own` is
false, and by the calls of gated_activation_amd where it is true.
"""
import math

import torch

own = False

GROUP = 32                   # values of one scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One token of a decode loop through a wide layer: both weights are read once.
        {"name": "forward_1x2048x16384", "op": "forward", "act": "gelu_tanh", "dtype": "bf16", "rows": 1, "H": 2048,
         "d": 16384, "live": -1},
        # A serving batch of some tens of tokens.
        {"name": "forward_64x4096x8192", "op": "forward", "act": "silu", "dtype": "bf16", "rows": 64, "H": 4096, "d": 8192,
         "live": -1},
        # An expert's capture-sized buffer, three quarters of it live, the forward pass of a training step.
        {"name": "train_16384x2048x768_live", "op": "train", "act": "silu", "dtype": "bf16", "rows": 16384, "H": 2048,
         "d": 768, "live": 12288},
        # A batch of sequences through a wide layer, forward pass of a training step, and its backward pass.
        {"name": "train_8192x4096x16384", "op": "train", "act": "gelu_tanh", "dtype": "bf16", "rows": 8192, "H": 4096,
         "d": 16384, "live": -1},
        {"name": "backward_8192x4096x16384", "op": "backward", "act": "gelu_tanh", "dtype": "bf16", "rows": 8192, "H": 4096,
         "d": 16384, "live": -1},
        # Ragged sizes in half precision, the exact GELU.
        {"name": "backward_1001x1032x2056_fp16", "op": "backward", "act": "gelu", "dtype": "fp16", "rows": 1001, "H": 1032,
         "d": 2056, "live": -1},
        # A weight, or a long batch's activation, brought to 4 bits and back.
        {"name": "mxfp4_4096x16384", "op": "quantize", "dtype": "bf16", "rows": 4096, "d": 16384, "live": -1},
        # A few rows: what the two calls cost when launches are all of it.
        {"name": "mxfp4_16x2048_fp16", "op": "quantize", "dtype": "fp16", "rows": 16, "d": 2048, "live": -1},
        # The down projection after the activation, both operands in 4 bits: a batch, and one token.
        {"name": "product_4096x16384x4096", "op": "product", "act": "silu", "dtype": "bf16", "rows": 4096, "d": 16384,
         "n": 4096, "live": -1},
        {"name": "product_1x16384x2048", "op": "product", "act": "gelu_tanh", "dtype": "bf16", "rows": 1, "d": 16384,
         "n": 2048, "live": -1},
        # The whole layer in 4 bits: a decode batch, and a prefill of odd length.
        {"name": "forward4_4x4096x16384", "op": "forward4", "act": "silu", "dtype": "bf16", "rows": 4, "H": 4096, "d": 16384,
         "live": -1},
        {"name": "forward4_4095x4096x8192", "op": "forward4", "act": "silu", "dtype": "bf16", "rows": 4095, "H": 4096,
         "d": 8192, "live": -1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "backward", "backward", "quantize", "product", "product", "forward4",
                     "forward4"])
    act = rng.choice(["silu", "gelu_tanh", "gelu", "squared_relu"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    rows = _log(rng, 1, 16384)
    if op == "quantize":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        case = {"op": op, "dtype": dtype, "rows": rows, "d": min(_log(rng, 1, 65536), (1 << 26) // rows)}
    elif op == "product":
        d, n = _log(rng, 32, 16384), _log(rng, 1, 16384)
        if rng.random() < 0.6:
            d, n = -(-d // 64) * 64, -(-n // 16) * 16
        # single precision where the operand is quantised as it is: a code that an activation's last bit decides
        # is worth more than single precision holds
        act = rng.choice(["", act, act])
        case = {"op": op, "act": act, "dtype": dtype if act else rng.choice(["bf16", "fp16", "fp32"]),
                "rows": min(rows, (1 << 38) // (d * n)), "d": d, "n": n}
    else:
        step = 32 if op == "forward4" else 8
        H, d = 8 * _log(rng, 8, 512), step * _log(rng, 64 // step, 16384 // step)
        case = {"op": op, "act": act, "dtype": dtype, "rows": min(rows, (1 << 38) // (H * d)), "H": H, "d": d}
    case["live"] = rng.randint(1, case["rows"]) if rng.random() < 0.3 else -1
    return case


def _halves(act):
    return 1 if act in ("", "squared_relu") else 2


def _groups(d):
    return -(-d // GROUP)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows, op, act = case["rows"], case["op"], case.get("act", "")
    d = case["d"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dt)

    def zeros(*shape):
        return torch.zeros(*shape, dtype=dt, device="cuda")

    def weight(n, k):
        """A weight in 4 bits: what quantising normal values of variance 1 / k in blocks of 32 leaves,
        codes of e2m1 (sign, two bits of exponent, one of mantissa) and powers of two a few steps apart."""
        w = torch.randn(n, _groups(k) * GROUP, device="cuda", generator=g)
        codes = ((w.abs() * 2.0).clamp(max=7.0).to(torch.uint8) + (w < 0).to(torch.uint8) * 8)
        if k % GROUP:
            codes[:, k:] = 0
        e = torch.randint(0, 3, (n, _groups(k)), device="cuda", generator=g) + (126 - round(math.log2(max(k, 1)) / 2))
        return codes[:, 0::2] | codes[:, 1::2] << 4, e.to(torch.uint8)

    s = {"case": case, "op": op, "dtype": dt, "act": act}
    live = rows if case["live"] < 0 else case["live"]
    s["live"] = None if case["live"] < 0 else torch.tensor([live], dtype=torch.int32, device="cuda")
    s["keep"] = None if s["live"] is None else torch.arange(rows, device="cuda")[:, None] < s["live"]
    h = _halves(act)
    if op == "quantize":
        # an activation's output: mostly small, some large
        s["x"] = (torch.randn(rows, d, device="cuda", generator=g) * torch.randn(rows, d, device="cuda", generator=g)).to(dt)
        s["codes"] = torch.zeros(rows, _groups(d) * GROUP // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(rows, _groups(d), dtype=torch.uint8, device="cuda")
        s["out"] = zeros(rows, d)
    elif op == "product":
        s["x"] = normal(rows, h * d, std=1.5 if act else 1.0)
        s["w"] = weight(case["n"], d)
        s["out"] = zeros(rows, case["n"])
    else:
        H = case["H"]
        s["x"], s["out"] = normal(rows, H), zeros(rows, H)
        if op == "forward4":
            s["w_in"], s["w_down"] = weight(h * d, H), weight(H, d)
        else:
            s["w_in"], s["w_down"] = normal(h * d, H, std=H ** -0.5), normal(H, d, std=d ** -0.5)
        if op == "train":
            s["kept"] = zeros(rows, h * d)
        if op == "backward":
            # what the forward pass left behind
            s["kept"], s["dy"] = normal(rows, h * d), normal(rows, H)
    return s


# ---- the calls of the library -------------------------------------------------

def _own_run(s):
    import gated_activation_amd as ga
    op, act, live, x = s["op"], s["act"], s["live"], s["x"]
    if op == "forward":
        return ga.feed_forward(x, s["w_in"], s["w_down"], act, live_rows=live, out=s["out"])
    if op == "train":
        return ga.feed_forward_train(x, s["w_in"], s["w_down"], act, live_rows=live, out=s["out"], kept=s["kept"])
    if op == "backward":
        return ga.feed_forward_backward(s["dy"], x, s["kept"], s["w_in"], s["w_down"], act, live_rows=live, out=s["out"])
    d = s["case"]["d"]
    if op == "quantize":
        q = ga.mxfp4_quantize(x, live_rows=live, out=ga.Mxfp4(s["codes"], s["scales"], d))
        return ga.mxfp4_dequantize(q, s["dtype"], live_rows=live, out=s["out"])
    if op == "product":
        a = ga.activation_mxfp4(x, act, live_rows=live) if act else ga.mxfp4_quantize(x, live_rows=live)
        return ga.mxfp4_product(a, ga.Mxfp4(*s["w"], d), s["dtype"], live_rows=live, out=s["out"])
    return ga.feed_forward_mxfp4(x, ga.Mxfp4(*s["w_in"], s["case"]["H"]), ga.Mxfp4(*s["w_down"], d), act, live_rows=live,
                                 out=s["out"])


# ---- the plain forms ----------------------------------------------------------

def _into(s, value, into):
    """`value` in the live rows, the others as they were."""
    value = value.to(into.dtype)
    return value if s["keep"] is None else torch.where(s["keep"], value, into)


def _slope(act, g):
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


def _gated(act, z):
    if act == "squared_relu":
        return _slope(act, z)[0]
    d = z.shape[1] // 2
    return _slope(act, z[:, :d])[0] * z[:, d:]


def _quantized(x):
    """The values that 4 bits keep of fp32 rows [rows, d]."""
    rows, d = x.shape
    x = torch.nn.functional.pad(x, (0, _groups(d) * GROUP - d)).view(rows, -1, GROUP)
    top = x.abs().amax(-1, keepdim=True)
    # floor(log2) from the exponent itself; a block of zeros has the least
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127).int()).clamp(min=-127)
    y = torch.ldexp(x, -e).abs()
    # steps of 1/2 up to 2, of 1 up to 4, of 2 up to 6, ties to even
    step = torch.where(y < 2.0, 0.5, torch.where(y < 4.0, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    return torch.ldexp(torch.copysign(y, x), e).view(rows, -1)[:, :d]


def _values(q, d):
    """The fp32 values of codes and scales."""
    codes, scales = q
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(1)
    v = table[both.int()].view(codes.shape[0], -1, GROUP)
    return torch.ldexp(v, scales.int()[..., None] - 127).flatten(1)[:, :d]


def _plain_run(s):
    op, act, x = s["op"], s["act"], s["x"].float()
    if op == "quantize":
        return _into(s, _quantized(x), s["out"])
    if op == "product":
        # the activation as it is stored, then in 4 bits
        a = _gated(act, x).to(s["dtype"]).float() if act else x
        return _into(s, _quantized(a) @ _values(s["w"], a.shape[1]).T, s["out"])
    if op == "forward4":
        z = _quantized(x) @ _values(s["w_in"], x.shape[1]).T
        h = _gated(act, z)
        return _into(s, _quantized(h) @ _values(s["w_down"], h.shape[1]).T, s["out"])
    w_in, w_down = s["w_in"].float(), s["w_down"].float()
    if op in ("forward", "train"):
        z = x @ w_in.T
        y = _into(s, _gated(act, z) @ w_down.T, s["out"])
        return y if op == "forward" else (y, _into(s, z, s["kept"]))
    dy, z = s["dy"].float(), s["kept"].float()
    if s["keep"] is not None:
        dy, x, z = (torch.where(s["keep"], t, torch.zeros_like(t)) for t in (dy, x, z))
    dh = dy @ w_down
    if act == "squared_relu":
        value, slope = _slope(act, z)
        dz, h = dh * slope, value
    else:
        d = dh.shape[1]
        value, slope = _slope(act, z[:, :d])
        dz, h = torch.cat([dh * z[:, d:] * slope, dh * value], dim=1), value * z[:, d:]
    dt = s["dtype"]
    return _into(s, dz @ w_in, s["out"]), (dz.T @ x).to(dt), (dy.T @ h).to(dt)


def run(s):
    if own:
        return _own_run(s)
    return _plain_run(s)


def work(case):
    op, act, d = case["op"], case.get("act", ""), case["d"]
    es = 4 if case["dtype"] == "fp32" else 2
    rows = max(1, case["rows"] if case["live"] < 0 else case["live"])
    h = _halves(act)
    kept = 0.5 + 1.0 / GROUP      # bytes of a value in 4 bits
    if op == "quantize":
        return {"bytes": rows * d * (2 * es + 2 * kept), "flops": 4 * rows * d}
    if op == "product":
        n = case["n"]
        return {"bytes": rows * d * (h * es + 2 * kept) + n * d * kept + rows * n * es, "flops": 2 * rows * n * d}
    H = case["H"]
    weights = (h + 1) * d * H
    if op == "forward4":
        return {"bytes": weights * kept + 2 * rows * H * es, "flops": 2 * rows * weights}
    if op == "backward":
        return {"bytes": 2 * weights * es + rows * (3 * H + h * d) * es, "flops": 4 * rows * weights}
    return {"bytes": weights * es + rows * 2 * H * es + (rows * h * d * es if op == "train" else 0),
            "flops": 2 * rows * weights}


# ---- 64 bits ------------------------------------------------------------------

_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _kept64(v):
    """The nearest of e2m1's values, times the block's power of two, in 64 bits."""
    rows, d = v.shape
    whole = v.new_zeros(rows, _groups(d) * GROUP)
    whole[:, :d] = v
    whole = whole.view(-1, GROUP)
    top = whole.abs().max(dim=1, keepdim=True).values
    # 2^floor(log2 top) is top's fp64 bits without their significand
    power = (top.view(torch.int64) & 0x7FF0000000000000).view(torch.float64)
    unit = (power / 4.0).clamp(min=2.0 ** -127)
    size = (whole / unit).abs()
    rank = torch.zeros_like(size)
    for k in range(1, 8):
        border = 0.5 * (_LEVELS[k - 1] + _LEVELS[k])
        # a tie goes to the level of even index
        rank += (size >= border) if k % 2 == 0 else (size > border)
    levels = torch.tensor(_LEVELS, dtype=torch.float64, device=v.device)
    return (levels[rank.long()] * torch.sign(whole) * unit).view(rows, -1)[:, :d]


def _weight64(q, d):
    codes, scales = q
    n = codes.shape[0]
    v = torch.empty(n, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    for half in range(2):
        c = (codes >> (4 * half)).long() & 15
        e, m = (c >> 1) & 3, (c & 1).double()
        size = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * 2.0 ** (e.double() - 1.0))
        v[:, half::2] = torch.where(c >= 8, -size, size)
    return (v.view(n, -1, GROUP) * torch.pow(2.0, scales.double() - 127.0)[:, :, None]).view(n, -1)[:, :d]


def _act64(act, z):
    if act == "squared_relu":
        return torch.relu(z) ** 2
    g, u = z.chunk(2, dim=1)
    if act == "silu":
        return g * torch.sigmoid(g) * u
    if act == "gelu":
        return g * torch.special.ndtr(g) * u
    return g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)) * u  # (1 + tanh(t)) / 2 = sigmoid(2 t)


def exact(case, seed):
    s = prepare(case, seed)
    op, act, d = case["op"], case.get("act", ""), case["d"]
    live = case["rows"] if case["live"] < 0 else case["live"]
    x = s["x"][:live].double()

    def padded(v):
        whole = torch.zeros(case["rows"], v.shape[1], dtype=torch.float64, device="cuda")
        whole[:live] = v
        return whole

    if op == "quantize":
        return padded(_kept64(x))
    if op == "product":
        # by definition of the operator the activation is rounded to its type before it is quantised
        a = _act64(act, x).to(s["dtype"]).double() if act else x
        return padded(torch.matmul(_kept64(a), _weight64(s["w"], d).T))
    if op == "forward4":
        z = torch.matmul(_kept64(x), _weight64(s["w_in"], case["H"]).T)
        return padded(torch.matmul(_kept64(_act64(act, z)), _weight64(s["w_down"], d).T))
    if op in ("forward", "train"):
        z = torch.matmul(x, s["w_in"].double().T)
        y = padded(torch.matmul(_act64(act, z), s["w_down"].double().T))
        return y if op == "forward" else (y, padded(z))
    dy = s["dy"][:live].double()
    dh = torch.matmul(dy, s["w_down"].double())
    with torch.enable_grad():
        z = s["kept"][:live].double().requires_grad_(True)
        h = _act64(act, z)
        dz, = torch.autograd.grad(h, z, dh)
    return (padded(torch.matmul(dz, s["w_in"].double())), torch.matmul(dz.T, x), torch.matmul(dy.T, h.detach()))
