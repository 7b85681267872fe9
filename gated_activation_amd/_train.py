"""ctypes binding of libga.so's training entry points.  Argument checks and
marshalling only; every computation is in the HIP kernels."""
import ctypes
from typing import NamedTuple, Optional

import torch

from ._lib import Z_SPARSITY_095, _TORCH_DTYPE, _check, lib

GA_ACT_SILU, GA_ACT_GELU_TANH, GA_ACT_GELU_ERF, GA_ACT_SQUARED_RELU, GA_ACT_GELU_SPARSE = range(5)
GA_CHECKPOINT_BLOCK = 128
GA_LAYER_NORM_MAX_D = 32768
GA_BALANCE_MAX_EXPERTS = 1024

ACTIVATIONS = {"silu": GA_ACT_SILU, "gelu_tanh": GA_ACT_GELU_TANH, "gelu": GA_ACT_GELU_ERF,
               "squared_relu": GA_ACT_SQUARED_RELU, "gelu_sparse": GA_ACT_GELU_SPARSE}


def _bind():
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    sigs = {
        "ga_checkpoint_store": [vp, vp, vp, i64, i64, i32, vp, vp],
        "ga_checkpoint_restore": [vp, vp, vp, vp, i64, i64, i32, i32, vp, vp],
        "ga_activation_checkpoint": [vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, vp, vp],
        "ga_activation_backward": [vp, vp, vp, i64, i64, i32, i32, f32, vp, vp],
        "ga_activation_backward_checkpoint": [vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, vp, vp],
        "ga_layer_norm": [vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, vp, vp],
        "ga_layer_norm_checkpoint": [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, vp, vp],
        "ga_layer_norm_backward": [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp, vp, sz, vp],
        "ga_layer_norm_backward_checkpoint": [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp, vp, sz, vp],
        "ga_balance_loss": [vp, vp, i32, vp, vp, vp, vp, vp, i64, i64, i64, i32, f32, vp, vp, sz, vp],
        "ga_balance_loss_backward": [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, f32, vp, vp],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("ga_layer_norm_backward_workspace_bytes", "ga_balance_loss_workspace_bytes"):
        fn = getattr(lib, name)
        fn.argtypes = [i64, i64]
        fn.restype = sz


_bind()


class _Arrays(NamedTuple):
    codes: torch.Tensor
    scales: torch.Tensor
    stats: Optional[torch.Tensor] = None


class Checkpoint(_Arrays):
    """An array kept in 8 bits, a tuple of three: codes int8 [rows, d] or, gate
    and up apart, [rows, 2, d]; scales fp32 [rows, ceil(d / 128)] or [rows, 2,
    ceil(d / 128)]; stats fp32 [rows, 2] where the codes are relative to their
    row.  The one that activation_checkpoint returns says whose input it is, by
    its attributes activation and, of gelu_sparse, z.  None (a Checkpoint made of
    tensors alone): the caller's knowledge."""
    activation: Optional[str] = None
    z: Optional[float] = None

    def _replace(self, **arrays):
        c = super()._replace(**arrays)
        c.activation, c.z = self.activation, self.z
        return c


class Balance(NamedTuple):
    """What balance_loss returns: the loss (fp32 scalar), counts int32
    [experts], offsets int32 [experts + 1] (offsets[-1:] is the live count of a
    buffer sorted by expert), tokens int32 [1] (the tokens that counted), and
    the k and coefficient its gradient needs."""
    loss: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    tokens: torch.Tensor
    k: int
    coefficient: float


# The current device and a device's current stream as plain numbers: 0.1 us
# each, where torch.cuda.current_stream(...).cuda_stream takes 1.8 us of a call
# whose launch takes 3.8.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(fn, device, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _matrix(t, what, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: {what} must be a CUDA (HIP) tensor")
    if t.dim() != 2 or t.shape[1] == 0 or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be a contiguous [rows, columns] tensor, got {tuple(t.shape)}")
    if t.dtype not in _TORCH_DTYPE:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")


def _like(t, shape, dtype, device, what, name):
    """t itself, or a new tensor where it is None."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device
            or not t.is_contiguous()):
        raise ValueError(f"{name}: {what} must be a contiguous {list(shape)} {dtype} tensor on {device}")
    return t


def _live(live_rows, device, name):
    if live_rows is None:
        return None
    if (not isinstance(live_rows, torch.Tensor) or live_rows.dtype != torch.int32 or live_rows.device != device
            or live_rows.numel() < 1):
        raise ValueError(f"{name}: live_rows must be an int32 tensor on {device}")
    return live_rows.data_ptr()


def _checkpoint(c, rows, halves, d, stats, device, name, activation=None, z=None):
    """A Checkpoint of c's tensors, checked, or of new ones where c is None."""
    codes, scales, st = (None, None, None) if c is None else c
    lead = (rows,) if halves == 1 else (rows, halves)
    codes = _like(codes, lead + (d,), torch.int8, device, "checkpoint.codes", name)
    scales = _like(scales, lead + (-(-d // GA_CHECKPOINT_BLOCK),), torch.float32, device, "checkpoint.scales", name)
    st = _like(st, (rows, 2), torch.float32, device, "checkpoint.stats", name) if stats else None
    c = Checkpoint(codes, scales, st)
    if activation is not None:
        c.activation, c.z = activation, z
    return c


def _given(c, stats, name):
    if not isinstance(c, Checkpoint) or any(not isinstance(t, torch.Tensor) for t in (c.codes, c.scales)) \
            or (stats and c.stats is None):
        raise ValueError(f"{name}: a Checkpoint with codes, scales{' and stats' if stats else ''} is needed")


def _activation(activation, name):
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"{name}: activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    return act


def checkpoint_store(x, live_rows=None, checkpoint=None):
    """x [rows, d] kept in 8 bits: blocks of 128 values along a row, one fp32
    scale a block.  checkpoint: a Checkpoint to write into (else a new one)."""
    name = "checkpoint_store"
    _matrix(x, "x", name)
    rows, d = x.shape
    device = x.device
    c = _checkpoint(checkpoint, rows, 1, d, False, device, name)
    live = _live(live_rows, device, name)
    _call(lib.ga_checkpoint_store, device, x.data_ptr(), c.codes.data_ptr(), c.scales.data_ptr(), rows, d,
          _TORCH_DTYPE[x.dtype], live)
    return c


def checkpoint_restore(checkpoint, dtype, live_rows=None, out=None):
    """The values a Checkpoint stands for, [rows, d] (or [rows, 2d], gate | up)
    of `dtype`.  Codes that are relative to their row (a Checkpoint with stats)
    have the row's cutoff or mean added back."""
    name = "checkpoint_restore"
    _given(checkpoint, False, name)
    if dtype not in _TORCH_DTYPE:
        raise ValueError(f"{name}: unsupported dtype {dtype}")
    codes = checkpoint.codes
    if not codes.is_cuda or codes.dim() not in (2, 3) or (codes.dim() == 3 and codes.shape[1] != 2):
        raise ValueError(f"{name}: codes must be a [rows, d] or [rows, 2, d] CUDA (HIP) tensor")
    rows, d, halves, device = codes.shape[0], codes.shape[-1], codes.dim() - 1, codes.device
    c = _checkpoint(checkpoint, rows, halves, d, checkpoint.stats is not None, device, name)
    out = _like(out, (rows, halves * d), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    _call(lib.ga_checkpoint_restore, device, c.codes.data_ptr(), c.scales.data_ptr(), _ptr(c.stats), out.data_ptr(), rows,
          d, halves, _TORCH_DTYPE[dtype], live)
    return out


def activation_checkpoint(x, activation, z=Z_SPARSITY_095, live_rows=None, out=None, checkpoint=None):
    """The forward pass of a gated activation that keeps its input in 8 bits:
    returns (out [rows, d], Checkpoint).  activation: "silu", "gelu_tanh",
    "gelu" (erf) or "gelu_sparse" (cutoff multiplier z) on x = [gate | up]
    ([rows, 2d]), or "squared_relu" on x [rows, d].  out and checkpoint: tensors
    to write into; rows past live_rows stay as they are.  The Checkpoint returned
    knows its activation and z."""
    name = "activation_checkpoint"
    act = _activation(activation, name)
    _matrix(x, "x", name)
    halves = 1 if act == GA_ACT_SQUARED_RELU else 2
    rows, cols = x.shape
    if cols % halves != 0:
        raise ValueError(f"{name}: x must be [rows, 2d], got {tuple(x.shape)}")
    d, device = cols // halves, x.device
    sparse = act == GA_ACT_GELU_SPARSE
    out = _like(out, (rows, d), x.dtype, device, "out", name)
    c = _checkpoint(checkpoint, rows, halves, d, sparse, device, name, activation, float(z) if sparse else None)
    live = _live(live_rows, device, name)
    _call(lib.ga_activation_checkpoint, device, x.data_ptr(), out.data_ptr(), c.codes.data_ptr(), c.scales.data_ptr(),
          _ptr(c.stats), rows, d, _TORCH_DTYPE[x.dtype], act, z, live)
    return out, c


def activation_backward(dout, kept, activation, z=None, live_rows=None, out=None):
    """The gradient of a gated activation's input from dout [rows, d] and what
    the forward pass kept: the input x itself (of dout's dtype) or the
    Checkpoint of activation_checkpoint.  z, of gelu_sparse: None is the
    Checkpoint's own or, where it has none and with x, activation_checkpoint's
    default.  A Checkpoint of another activation or z is refused.  Returns dx ([rows, 2d]; [rows, d] for
    "squared_relu"); rows past live_rows stay as they are."""
    name = "activation_backward"
    act = _activation(activation, name)
    _matrix(dout, "dout", name)
    halves = 1 if act == GA_ACT_SQUARED_RELU else 2
    rows, d = dout.shape
    device, dtype = dout.device, dout.dtype
    sparse = act == GA_ACT_GELU_SPARSE
    from_x = isinstance(kept, torch.Tensor)
    if from_x:
        _like(kept, (rows, halves * d), dtype, device, "x", name)
    else:
        _given(kept, sparse, name)
        if not sparse and kept.stats is not None:
            raise ValueError(f"{name}: the Checkpoint's codes are relative to their rows (it has stats): not of {activation}")
        if kept.activation is not None and kept.activation != activation:
            raise ValueError(f"{name}: the Checkpoint is of {kept.activation}, not of {activation}")
        if sparse and kept.z is not None:
            # the kernels take z in fp32
            if z is not None and z != kept.z and ctypes.c_float(z).value != ctypes.c_float(kept.z).value:
                raise ValueError(f"{name}: the Checkpoint is of z = {kept.z}, not of {z}")
            z = kept.z
        kept = _checkpoint(kept, rows, halves, d, sparse, device, name)
    out = _like(out, (rows, halves * d), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    if z is None:
        z = Z_SPARSITY_095
    if from_x:
        _call(lib.ga_activation_backward, device, dout.data_ptr(), kept.data_ptr(), out.data_ptr(), rows, d,
              _TORCH_DTYPE[dtype], act, z, live)
    else:
        _call(lib.ga_activation_backward_checkpoint, device, dout.data_ptr(), kept.codes.data_ptr(),
              kept.scales.data_ptr(), _ptr(kept.stats), out.data_ptr(), rows, d, _TORCH_DTYPE[dtype], act, z, live)
    return out


def _vector(t, d, dtypes, device, what, name):
    if (not isinstance(t, torch.Tensor) or t.shape != (d,) or t.dtype not in dtypes or t.device != device
            or not t.is_contiguous()):
        raise ValueError(f"{name}: {what} must be a contiguous [{d}] tensor of {' or '.join(map(str, dtypes))} on {device}")


def _norm_args(x, weight, bias, name):
    _matrix(x, "x", name)
    d = x.shape[1]
    _vector(weight, d, (x.dtype, torch.float32), x.device, "weight", name)
    if bias is not None:
        _vector(bias, d, (weight.dtype,), x.device, "bias", name)
    return x.shape[0], d, x.device


def layer_norm(x, weight, bias=None, eps=1e-5, live_rows=None, out=None, stats=None):
    """Layer norm of x [rows, d] (d <= GA_LAYER_NORM_MAX_D): returns (y, stats),
    stats fp32 [rows, 2] = (mean, 1 / sqrt(variance + eps)) for the backward
    pass.  weight and bias [d] are of x's dtype or fp32."""
    name = "layer_norm"
    rows, d, device = _norm_args(x, weight, bias, name)
    out = _like(out, (rows, d), x.dtype, device, "out", name)
    stats = _like(stats, (rows, 2), torch.float32, device, "stats", name)
    live = _live(live_rows, device, name)
    _call(lib.ga_layer_norm, device, x.data_ptr(), weight.data_ptr(), _ptr(bias), out.data_ptr(), stats.data_ptr(), rows,
          d, _TORCH_DTYPE[x.dtype], _TORCH_DTYPE[weight.dtype], eps, live)
    return out, stats


def layer_norm_checkpoint(x, weight, bias=None, eps=1e-5, live_rows=None, out=None, checkpoint=None):
    """layer_norm that keeps x - mean in 8 bits: returns (y, Checkpoint), its
    stats as layer_norm's."""
    name = "layer_norm_checkpoint"
    rows, d, device = _norm_args(x, weight, bias, name)
    out = _like(out, (rows, d), x.dtype, device, "out", name)
    c = _checkpoint(checkpoint, rows, 1, d, True, device, name)
    live = _live(live_rows, device, name)
    _call(lib.ga_layer_norm_checkpoint, device, x.data_ptr(), weight.data_ptr(), _ptr(bias), out.data_ptr(),
          c.codes.data_ptr(), c.scales.data_ptr(), c.stats.data_ptr(), rows, d, _TORCH_DTYPE[x.dtype],
          _TORCH_DTYPE[weight.dtype], eps, live)
    return out, c


def _scratch(workspace, need, device, name):
    """(address, bytes, tensor) of the caller's workspace or, where it is None,
    of memory of this call's own: from the stream's pool, or a capturing
    graph's, so calls never share it.  The tensor is to be held until the
    launch."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def layer_norm_backward_workspace_bytes(rows, d):
    return int(lib.ga_layer_norm_backward_workspace_bytes(rows, d))


def layer_norm_backward(dy, kept, weight, stats=None, live_rows=None, out=None, bias=True, workspace=None):
    """Layer norm's gradients from dy [rows, d] and what the forward pass kept:
    x with layer_norm's stats, or layer_norm_checkpoint's Checkpoint.  Returns
    (dx, dweight, dbias), the latter two of weight's dtype, summed over the live
    rows; bias=False: dbias is None.  workspace: None, or
    layer_norm_backward_workspace_bytes(rows, d) bytes of the caller's."""
    name = "layer_norm_backward"
    rows, d, device = _norm_args(dy, weight, None, name)
    dtype = dy.dtype
    from_x = isinstance(kept, torch.Tensor)
    if from_x:
        _like(kept, (rows, d), dtype, device, "x", name)
        if stats is None:
            raise ValueError(f"{name}: x needs the forward pass' stats")
        _like(stats, (rows, 2), torch.float32, device, "stats", name)
    else:
        if stats is not None:
            raise ValueError(f"{name}: a Checkpoint brings its own stats")
        _given(kept, True, name)
        kept = _checkpoint(kept, rows, 1, d, True, device, name)
    out = _like(out, (rows, d), dtype, device, "out", name)
    live = _live(live_rows, device, name)
    dweight = torch.empty_like(weight)
    dbias = torch.empty_like(weight) if bias else None
    ws, ws_bytes, held = _scratch(workspace, lib.ga_layer_norm_backward_workspace_bytes(rows, d), device, name)
    tail = (weight.data_ptr(), out.data_ptr(), dweight.data_ptr(), _ptr(dbias), rows, d, _TORCH_DTYPE[dtype],
            _TORCH_DTYPE[weight.dtype], live, ws, ws_bytes)
    if from_x:
        _call(lib.ga_layer_norm_backward, device, dy.data_ptr(), kept.data_ptr(), stats.data_ptr(), *tail)
    else:
        _call(lib.ga_layer_norm_backward_checkpoint, device, dy.data_ptr(), kept.codes.data_ptr(), kept.scales.data_ptr(),
              kept.stats.data_ptr(), *tail)
    del held
    return out, dweight, dbias


def _mask(mask, rows, device, name):
    if mask is None:
        return None
    if (not isinstance(mask, torch.Tensor) or mask.shape != (rows,) or mask.dtype not in (torch.bool, torch.uint8)
            or mask.device != device or not mask.is_contiguous()):
        raise ValueError(f"{name}: mask must be a contiguous [{rows}] bool or uint8 tensor on {device}")
    return mask.data_ptr()


def balance_loss_workspace_bytes(rows, experts):
    return int(lib.ga_balance_loss_workspace_bytes(rows, experts))


def balance_loss(logits, experts, coefficient=1.0, mask=None, live_rows=None, workspace=None):
    """The router's balance loss and per-expert counts: logits [rows, E] (E <=
    GA_BALANCE_MAX_EXPERTS), experts [rows, k] int32 or int64 (the experts
    chosen for each token; values outside [0, E) are not counted).  Tokens past
    live_rows or with a false mask ([rows]) do not count.  Returns a Balance."""
    name = "balance_loss"
    _matrix(logits, "logits", name)
    rows, e = logits.shape
    device = logits.device
    if (not isinstance(experts, torch.Tensor) or experts.dim() != 2 or experts.shape[0] != rows
            or experts.shape[1] < 1 or experts.dtype not in (torch.int32, torch.int64) or experts.device != device
            or not experts.is_contiguous()):
        raise ValueError(f"{name}: experts must be a contiguous [{rows}, k] int32 or int64 tensor on {device}")
    k = experts.shape[1]
    m = _mask(mask, rows, device, name)
    live = _live(live_rows, device, name)
    loss = torch.empty((), dtype=torch.float32, device=device)
    whole = torch.empty(2 * e + 2, dtype=torch.int32, device=device)
    counts, offsets, tokens = whole.split_with_sizes((e, e + 1, 1))
    at = whole.data_ptr()
    ws, ws_bytes, held = _scratch(workspace, lib.ga_balance_loss_workspace_bytes(rows, e), device, name)
    _call(lib.ga_balance_loss, device, logits.data_ptr(), experts.data_ptr(), experts.element_size(), m, loss.data_ptr(),
          at, at + 4 * e, at + 8 * e + 4, rows, e, k, _TORCH_DTYPE[logits.dtype], coefficient, live, ws, ws_bytes)
    del held
    return Balance(loss, counts, offsets, tokens, k, coefficient)


def balance_loss_backward(logits, balance, dloss=None, mask=None, live_rows=None, out=None):
    """The gradient of logits from balance_loss' result and dloss (an fp32
    device scalar; None: 1).  mask and live_rows as in the forward pass.  Tokens
    that do not count get 0; rows past live_rows stay as they are."""
    name = "balance_loss_backward"
    _matrix(logits, "logits", name)
    rows, e = logits.shape
    device = logits.device
    if not isinstance(balance, Balance):
        raise ValueError(f"{name}: balance must be balance_loss' result")
    for t, n, what in ((balance.counts, e, "counts"), (balance.offsets, e + 1, "offsets"), (balance.tokens, 1, "tokens")):
        _vector(t, n, (torch.int32,), device, what, name)
    if dloss is None:
        dloss = torch.ones((), dtype=torch.float32, device=device)
    elif (not isinstance(dloss, torch.Tensor) or dloss.numel() != 1 or dloss.dtype != torch.float32
          or dloss.device != device):
        raise ValueError(f"{name}: dloss must be an fp32 scalar tensor on {device}")
    m = _mask(mask, rows, device, name)
    live = _live(live_rows, device, name)
    out = _like(out, (rows, e), logits.dtype, device, "out", name)
    _call(lib.ga_balance_loss_backward, device, logits.data_ptr(), m, balance.counts.data_ptr(),
          balance.offsets.data_ptr(), balance.tokens.data_ptr(), dloss.data_ptr(), out.data_ptr(), rows, e, balance.k,
          _TORCH_DTYPE[logits.dtype], balance.coefficient, live)
    return out
