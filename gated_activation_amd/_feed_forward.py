"""ctypes binding of libga.so's feed-forward entry points, in 16 bits and in
microscaled 4 bits.  Argument checks and marshalling only; every computation is
in the HIP kernels."""
import ctypes
from typing import NamedTuple

import torch

from ._lib import _TORCH_DTYPE, _check, lib
from ._train import ACTIVATIONS, _call, _like, _live, _matrix, _ptr, _scratch

GA_MXFP4_BLOCK = 32
(GA_PRODUCT_HIDDEN, GA_PRODUCT_OUT, GA_PRODUCT_DHIDDEN, GA_PRODUCT_DX, GA_PRODUCT_DW_IN,
 GA_PRODUCT_DW_DOWN) = range(6)

_Tensor, _uint8 = torch.Tensor, torch.uint8

# Those that need a token's gate and up values alone.
ELEMENTWISE = tuple(a for a in ACTIVATIONS if a != "gelu_sparse")


class ProductPlan(ctypes.Structure):
    """How one of the layer's products runs."""
    _fields_ = [("features", ctypes.c_int32), ("tokens", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("k_step", ctypes.c_int32), ("splits", ctypes.c_int32), ("joint", ctypes.c_int32),
                ("k_slice", ctypes.c_int64), ("grid", ctypes.c_int64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


def _bind():
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    sigs = {
        "ga_feed_forward": [vp] * 5 + [i64] * 3 + [i32, i32, vp, vp, sz, vp],
        "ga_feed_forward_backward": [vp] * 8 + [i64] * 3 + [i32, i32, vp, vp, sz, vp],
        "ga_mxfp4_quantize": [vp, vp, vp, i64, i64, i32, vp, vp],
        "ga_mxfp4_dequantize": [vp, vp, vp, i64, i64, i32, vp, vp],
        "ga_activation_mxfp4": [vp, vp, vp, i64, i64, i32, i32, vp, vp],
        "ga_mxfp4_product": [vp] * 5 + [i64] * 3 + [i32, vp, vp, sz, vp],
        "ga_feed_forward_mxfp4": [vp] * 6 + [i64] * 3 + [i32, i32, vp, vp, sz, vp],
        "ga_plan_feed_forward": [i64, i64, i64, i32, i32, i32, ctypes.POINTER(ProductPlan)],
        "ga_plan_mxfp4_product": [i64, i64, i64, ctypes.POINTER(ProductPlan)],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("ga_feed_forward_workspace_bytes", "ga_feed_forward_backward_workspace_bytes",
                 "ga_feed_forward_mxfp4_workspace_bytes"):
        fn = getattr(lib, name)
        fn.argtypes = [i64, i64, i64, i32]
        fn.restype = sz
    lib.ga_mxfp4_product_workspace_bytes.argtypes = [i64, i64, i64]
    lib.ga_mxfp4_product_workspace_bytes.restype = sz


_bind()


class Mxfp4(NamedTuple):
    """An array [rows, d] in microscaled 4 bits: codes uint8 [rows, 16 ceil(d /
    32)] (two values a byte, the first in the low half), scales uint8 [rows,
    ceil(d / 32)] (s stands for 2^(s - 127), 255 for NaNs), and d."""
    codes: torch.Tensor
    scales: torch.Tensor
    d: int


def _activation(activation, name):
    if activation not in ELEMENTWISE:
        raise ValueError(f"{name}: activation must be one of {sorted(ELEMENTWISE)}, got {activation!r}")
    return ACTIVATIONS[activation]


def _gated(activation):
    return 1 if activation == "squared_relu" else 2


def _weights(x, w_in, w_down, activation, name):
    """rows, H, d of the 16-bit layer."""
    _matrix(x, "x", name)
    if x.dtype == torch.float32:
        raise ValueError(f"{name}: bf16 or fp16 only, got {x.dtype}")
    rows, H = x.shape
    if not isinstance(w_down, torch.Tensor) or w_down.dim() != 2 or w_down.shape[0] != H or w_down.shape[1] == 0:
        raise ValueError(f"{name}: w_down must be a [{H}, d] tensor")
    d = w_down.shape[1]
    for w, shape, what in ((w_down, (H, d), "w_down"), (w_in, (_gated(activation) * d, H), "w_in")):
        _given(w, shape, x.dtype, x.device, what, name)
    return rows, H, d


def _given(t, shape, dtype, device, what, name):
    if t is None:
        raise ValueError(f"{name}: {what} must be a contiguous {list(shape)} {dtype} tensor on {device}")
    return _like(t, shape, dtype, device, what, name)


def feed_forward_workspace_bytes(rows, H, d, activation="silu"):
    return int(lib.ga_feed_forward_workspace_bytes(rows, H, d, _activation(activation, "feed_forward_workspace_bytes")))


def feed_forward_backward_workspace_bytes(rows, H, d, activation="silu"):
    return int(lib.ga_feed_forward_backward_workspace_bytes(
        rows, H, d, _activation(activation, "feed_forward_backward_workspace_bytes")))


def feed_forward_mxfp4_workspace_bytes(rows, H, d, activation="silu"):
    return int(lib.ga_feed_forward_mxfp4_workspace_bytes(rows, H, d, _activation(activation, "feed_forward_mxfp4_workspace_bytes")))


def mxfp4_product_workspace_bytes(rows, n, d):
    return int(lib.ga_mxfp4_product_workspace_bytes(rows, n, d))


def plan_feed_forward(rows, H, d, activation, product, bits=16):
    """How the product GA_PRODUCT_* of a layer of these sizes runs (host only):
    feed_forward's and its backward pass's, with bits=4 feed_forward_mxfp4's."""
    p = ProductPlan()
    _check(lib.ga_plan_feed_forward(rows, H, d, _activation(activation, "plan_feed_forward"), bits, product, ctypes.byref(p)))
    return p


def plan_mxfp4_product(rows, n, d):
    """How mxfp4_product of [rows, d] and [n, d] runs (host only)."""
    p = ProductPlan()
    _check(lib.ga_plan_mxfp4_product(rows, n, d, ctypes.byref(p)))
    return p


def _forward(name, x, w_in, w_down, activation, live_rows, out, kept, keep, workspace):
    act = _activation(activation, name)
    rows, H, d = _weights(x, w_in, w_down, activation, name)
    device, dtype = x.device, x.dtype
    out = _like(out, (rows, H), dtype, device, "out", name)
    if keep:
        kept = _like(kept, (rows, _gated(activation) * d), dtype, device, "kept", name)
    live = _live(live_rows, device, name)
    ws, ws_bytes, held = _scratch(workspace, lib.ga_feed_forward_workspace_bytes(rows, H, d, act), device, name)
    _call(lib.ga_feed_forward, device, x.data_ptr(), w_in.data_ptr(), w_down.data_ptr(), out.data_ptr(), _ptr(kept), rows, H,
          d, _TORCH_DTYPE[dtype], act, live, ws, ws_bytes)
    del held
    return out, kept


def feed_forward(x, w_in, w_down, activation="silu", live_rows=None, out=None, workspace=None):
    """The gated feed-forward layer, y = h w_down^T with h = act(gate) * up and
    gate | up = x w_in^T: x [rows, H], w_in [2d, H] (gate rows, then up rows; [d,
    H] for "squared_relu", which is not gated), w_down [H, d], bf16 or fp16, H
    and d multiples of 8.  activation: "silu", "gelu_tanh", "gelu" (erf) or
    "squared_relu".  Returns y [rows, H]; rows past live_rows stay as they are.
    workspace: None, or feed_forward_workspace_bytes(rows, H, d, activation)
    bytes of the caller's."""
    return _forward("feed_forward", x, w_in, w_down, activation, live_rows, out, None, False, workspace)[0]


def feed_forward_train(x, w_in, w_down, activation="silu", live_rows=None, out=None, kept=None, workspace=None):
    """feed_forward that keeps gate | up for the backward pass: returns (y,
    kept), kept [rows, 2d] ([rows, d] for "squared_relu") of x's dtype."""
    return _forward("feed_forward_train", x, w_in, w_down, activation, live_rows, out, kept, True, workspace)


def feed_forward_backward(dy, x, kept, w_in, w_down, activation="silu", live_rows=None, out=None, workspace=None):
    """The feed-forward layer's gradients from dy [rows, H], the input x and what
    feed_forward_train kept.  Returns (dx, dw_in, dw_down); the weights'
    gradients are summed over the live rows.  workspace: None, or
    feed_forward_backward_workspace_bytes(rows, H, d, activation) bytes of the
    caller's."""
    name = "feed_forward_backward"
    act = _activation(activation, name)
    rows, H, d = _weights(x, w_in, w_down, activation, name)
    device, dtype = x.device, x.dtype
    _given(dy, (rows, H), dtype, device, "dy", name)
    _given(kept, (rows, _gated(activation) * d), dtype, device, "kept", name)
    out = _like(out, (rows, H), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    dw_in, dw_down = torch.empty_like(w_in), torch.empty_like(w_down)
    ws, ws_bytes, held = _scratch(workspace, lib.ga_feed_forward_backward_workspace_bytes(rows, H, d, act), device, name)
    _call(lib.ga_feed_forward_backward, device, dy.data_ptr(), x.data_ptr(), kept.data_ptr(), w_in.data_ptr(),
          w_down.data_ptr(), out.data_ptr(), dw_in.data_ptr(), dw_down.data_ptr(), rows, H, d, _TORCH_DTYPE[dtype], act, live,
          ws, ws_bytes)
    del held
    return out, dw_in, dw_down


def _mxfp4(q, rows, d, device, what, name):
    """q checked, or a new Mxfp4 where it is None."""
    if q is None:
        nb = -(-d // GA_MXFP4_BLOCK)
        return Mxfp4(torch.empty((rows, 16 * nb), dtype=torch.uint8, device=device),
                     torch.empty((rows, nb), dtype=torch.uint8, device=device), d)
    if _rows(q) != rows or q.d != d or q.codes.device != device:
        raise ValueError(f"{name}: {what} must be a Mxfp4 of [{rows}, {d}] with contiguous arrays on {device}")
    return q


def _rows(q):
    """The rows of a Mxfp4 whose arrays fit one another and are on a GPU, else -1."""
    if not isinstance(q, Mxfp4):
        return -1
    codes, scales, d = q
    if (not isinstance(codes, _Tensor) or not isinstance(scales, _Tensor) or not isinstance(d, int) or d < 1
            or codes.dtype is not _uint8 or scales.dtype is not _uint8):
        return -1
    nb = -(-d // GA_MXFP4_BLOCK)
    shape, index = codes.shape, codes.get_device()
    if (len(shape) != 2 or shape[1] != 16 * nb or scales.shape != (shape[0], nb) or index < 0
            or index != scales.get_device() or not codes.is_contiguous() or not scales.is_contiguous()):
        return -1
    return shape[0]


def _held(q, what, name):
    """A Mxfp4 of the caller's, checked: (codes, scales, rows, d, device)."""
    rows = _rows(q)
    if rows < 0:
        raise ValueError(f"{name}: {what} must be a Mxfp4 of contiguous CUDA (HIP) tensors")
    codes, scales, d = q
    return codes, scales, rows, d, codes.device


def mxfp4_quantize(x, live_rows=None, out=None):
    """x [rows, d] in microscaled 4 bits: blocks of 32 values along a row, one
    power of two a block.  out: a Mxfp4 to write into (else a new one); rows past
    live_rows stay as they are."""
    name = "mxfp4_quantize"
    _matrix(x, "x", name)
    rows, d = x.shape
    q = _mxfp4(out, rows, d, x.device, "out", name)
    live = _live(live_rows, x.device, name)
    _call(lib.ga_mxfp4_quantize, x.device, x.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr(), rows, d,
          _TORCH_DTYPE[x.dtype], live)
    return q


def mxfp4_dequantize(q, dtype, live_rows=None, out=None):
    """The values a Mxfp4 stands for, [rows, d] of `dtype`."""
    name = "mxfp4_dequantize"
    if dtype not in _TORCH_DTYPE:
        raise ValueError(f"{name}: unsupported dtype {dtype}")
    codes, scales, rows, d, device = _held(q, "q", name)
    out = _like(out, (rows, d), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    _call(lib.ga_mxfp4_dequantize, device, codes.data_ptr(), scales.data_ptr(), out.data_ptr(), rows, d,
          _TORCH_DTYPE[dtype], live)
    return out


def activation_mxfp4(x, activation, live_rows=None, out=None):
    """A gated activation's result in microscaled 4 bits, in one pass: x = [gate |
    up] ([rows, 2d]; "squared_relu" [rows, d]) -> Mxfp4 of [rows, d], the same as
    mxfp4_quantize of the activation's output in x's dtype."""
    name = "activation_mxfp4"
    act = _activation(activation, name)
    _matrix(x, "x", name)
    rows, cols = x.shape
    if cols % _gated(activation) != 0:
        raise ValueError(f"{name}: x must be [rows, 2d], got {tuple(x.shape)}")
    d = cols // _gated(activation)
    q = _mxfp4(out, rows, d, x.device, "out", name)
    live = _live(live_rows, x.device, name)
    _call(lib.ga_activation_mxfp4, x.device, x.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr(), rows, d,
          _TORCH_DTYPE[x.dtype], act, live)
    return q


def mxfp4_product(a, w, dtype=torch.bfloat16, live_rows=None, out=None, workspace=None):
    """a w^T of two Mxfp4, a of [rows, d] and w of [n, d] (a linear layer's
    weight): [rows, n] of `dtype`, summed in fp32.  Rows past live_rows stay as
    they are.  workspace: None, or mxfp4_product_workspace_bytes(rows, n, d)
    bytes of the caller's."""
    name = "mxfp4_product"
    if dtype not in _TORCH_DTYPE:
        raise ValueError(f"{name}: unsupported dtype {dtype}")
    a_codes, a_scales, rows, d, device = _held(a, "a", name)
    w_codes, w_scales, n, wd, wdevice = _held(w, "w", name)
    if wd != d or wdevice != device or n < 1:
        raise ValueError(f"{name}: w must be a Mxfp4 of [n, {d}] on {device}, got [{n}, {wd}] on {wdevice}")
    out = _like(out, (rows, n), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    ws, ws_bytes, held = _scratch(workspace, lib.ga_mxfp4_product_workspace_bytes(rows, n, d), device, name)
    _call(lib.ga_mxfp4_product, device, a_codes.data_ptr(), a_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
          out.data_ptr(), rows, n, d, _TORCH_DTYPE[dtype], live, ws, ws_bytes)
    del held
    return out


def feed_forward_mxfp4(x, w_in, w_down, activation="silu", live_rows=None, out=None, workspace=None):
    """feed_forward on microscaled 4-bit operands: x [rows, H] (bf16 or fp16) and
    h = act(gate) * up are quantised in blocks of 32, w_in (of [2d, H]; [d, H] for
    "squared_relu") and w_down (of [H, d]) are Mxfp4; gate, up and h stay in fp32
    up to the quantiser.  H a multiple of 8, d of 32.  Returns y [rows, H] of x's
    dtype."""
    name = "feed_forward_mxfp4"
    act = _activation(activation, name)
    _matrix(x, "x", name)
    if x.dtype == torch.float32:
        raise ValueError(f"{name}: bf16 or fp16 only, got {x.dtype}")
    rows, H = x.shape
    device = x.device
    down, down_scales, h2, d, down_device = _held(w_down, "w_down", name)
    if h2 != H or down_device != device:
        raise ValueError(f"{name}: w_down must be a Mxfp4 of [{H}, d] on {device}, got [{h2}, {d}] on {down_device}")
    if w_in is None:
        raise ValueError(f"{name}: w_in must be a Mxfp4")
    _mxfp4(w_in, _gated(activation) * d, H, device, "w_in", name)
    out = _like(out, (rows, H), x.dtype, device, "out", name)
    live = _live(live_rows, device, name)
    ws, ws_bytes, held = _scratch(workspace, lib.ga_feed_forward_mxfp4_workspace_bytes(rows, H, d, act), device, name)
    _call(lib.ga_feed_forward_mxfp4, device, x.data_ptr(), w_in.codes.data_ptr(), w_in.scales.data_ptr(),
          down.data_ptr(), down_scales.data_ptr(), out.data_ptr(), rows, H, d, _TORCH_DTYPE[x.dtype], act, live, ws,
          ws_bytes)
    del held
    return out
