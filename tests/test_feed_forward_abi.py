"""The feed-forward entry points on the host: every call below is refused by a
check, or has no rows, before the library makes any HIP call."""
import ctypes

import pytest
import torch

import gated_activation_amd as ga

L = ga.lib
OK, EINVAL, EUNSUP = ga.GA_OK, ga.GA_EINVAL, ga.GA_EUNSUPPORTED
BF16, F32 = ga.GA_BF16, ga.GA_F32
SPARSE = ga.GA_ACT_GELU_SPARSE


def P(i, add=0):
    """Fake device addresses 1 TiB apart; never dereferenced."""
    return ctypes.c_void_p((0x100 + i) * (1 << 40) + add)


def forward(x=P(0), w_in=P(1), w_down=P(2), y=P(3), kept=P(4), rows=4, H=64, d=128, dt=BF16, act=0, live=None, ws=P(5),
            ws_bytes=1 << 32):
    return L.ga_feed_forward(x, w_in, w_down, y, kept, rows, H, d, dt, act, live, ws, ws_bytes, None)


def backward(dy=P(6), x=P(0), kept=P(4), w_in=P(1), w_down=P(2), dx=P(7), dw_in=P(8), dw_down=P(9), rows=4, H=64, d=128,
             dt=BF16, act=0, live=None, ws=P(5), ws_bytes=1 << 32):
    return L.ga_feed_forward_backward(dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, dt, act, live, ws, ws_bytes,
                                      None)


def quantize(x=P(0), codes=P(1), scales=P(2), rows=4, d=128, dt=BF16, live=None):
    return L.ga_mxfp4_quantize(x, codes, scales, rows, d, dt, live, None)


def dequantize(codes=P(1), scales=P(2), out=P(3), rows=4, d=128, dt=BF16, live=None):
    return L.ga_mxfp4_dequantize(codes, scales, out, rows, d, dt, live, None)


def activation(x=P(0), codes=P(1), scales=P(2), rows=4, d=128, dt=BF16, act=0, live=None):
    return L.ga_activation_mxfp4(x, codes, scales, rows, d, dt, act, live, None)


def product(a=P(0), a_s=P(1), w=P(2), w_s=P(3), out=P(4), rows=4, n=96, d=128, dt=BF16, live=None, ws=P(5), ws_bytes=1 << 32):
    return L.ga_mxfp4_product(a, a_s, w, w_s, out, rows, n, d, dt, live, ws, ws_bytes, None)


def forward4(x=P(0), w_in=P(1), w_in_s=P(2), w_down=P(3), w_down_s=P(4), y=P(6), rows=4, H=64, d=128, dt=BF16, act=0,
             live=None, ws=P(5), ws_bytes=1 << 32):
    return L.ga_feed_forward_mxfp4(x, w_in, w_in_s, w_down, w_down_s, y, rows, H, d, dt, act, live, ws, ws_bytes, None)


ALL = [forward, backward, quantize, dequantize, activation, product, forward4]
LAYER = [forward, backward, forward4]


@pytest.mark.parametrize("call", ALL)
@pytest.mark.parametrize("kwargs,status", [(dict(rows=-1), EINVAL), (dict(rows=2 ** 31), EINVAL), (dict(d=0), EINVAL),
                                           (dict(d=-8), EINVAL), (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL),
                                           (dict(d=65536 + 32), EUNSUP), (dict(live=P(11, 2)), EINVAL)])
def test_sizes_and_types(call, kwargs, status):
    assert call(**kwargs) == status and len(L.ga_last_error()) > 0


@pytest.mark.parametrize("call", LAYER)
@pytest.mark.parametrize("kwargs,status", [
    (dict(H=0), EINVAL), (dict(H=-8), EINVAL), (dict(H=65544), EUNSUP), (dict(H=60), EUNSUP), (dict(d=100), EUNSUP),
    (dict(dt=F32), EUNSUP), (dict(act=SPARSE), EUNSUP), (dict(act=5), EINVAL), (dict(act=-1), EINVAL),
    (dict(ws=None), EINVAL), (dict(ws_bytes=64), EINVAL), (dict(ws=P(5, 128)), EINVAL), (dict(ws=P(0)), EINVAL),
    (dict(rows=2 ** 31 - 1, ws=ctypes.c_void_p(1 << 60), ws_bytes=1 << 59), EUNSUP)])
def test_layer(call, kwargs, status):
    assert call(**kwargs) == status and len(L.ga_last_error()) > 0


def test_blocks_of_a_layer_stay_whole():
    assert forward4(d=48) == EUNSUP and forward4(d=72) == EUNSUP and forward(d=72, rows=0) == OK


@pytest.mark.parametrize("call,pointers", [
    (forward, ["x", "w_in", "w_down", "y"]), (backward, ["dy", "x", "kept", "w_in", "w_down", "dx", "dw_in", "dw_down"]),
    (quantize, ["x", "codes", "scales"]), (dequantize, ["codes", "scales", "out"]), (activation, ["x", "codes", "scales"]),
    (product, ["a", "a_s", "w", "w_s", "out"]), (forward4, ["x", "w_in", "w_in_s", "w_down", "w_down_s", "y"])])
def test_null_pointers(call, pointers):
    for p in pointers:
        assert call(**{p: None}) == EINVAL, p


@pytest.mark.parametrize("call,kwargs", [
    (forward, dict(x=P(0, 8))), (forward, dict(w_in=P(1, 2))), (forward, dict(y=P(3, 8))), (forward, dict(kept=P(4, 8))),
    (forward, dict(y=P(0))), (forward, dict(kept=P(3, 16))), (forward, dict(y=P(2, 16))), (forward, dict(ws=P(3))),
    (backward, dict(dx=P(6))), (backward, dict(dw_in=P(1))), (backward, dict(dw_down=P(8, 16))), (backward, dict(dx=P(7, 4))),
    (quantize, dict(codes=P(1, 8))), (quantize, dict(x=P(0, 1))), (quantize, dict(codes=P(0))), (quantize, dict(scales=P(1, 3))),
    (dequantize, dict(codes=P(1, 4))), (dequantize, dict(out=P(3, 1))), (dequantize, dict(out=P(1))),
    (activation, dict(act=7)), (activation, dict(codes=P(1, 8))), (activation, dict(codes=P(0, 4 * 256 * 2 - 16))),
    (product, dict(a=P(0, 8))), (product, dict(w=P(2, 4))), (product, dict(out=P(4, 1))), (product, dict(out=P(0))),
    (product, dict(n=0)), (product, dict(n=-5)), (product, dict(ws=P(5, 16))), (product, dict(out=P(3))),
    (forward4, dict(y=P(0))), (forward4, dict(y=P(6, 1))), (forward4, dict(w_in=P(1, 8))), (forward4, dict(ws=P(4)))])
def test_malformed(call, kwargs):
    assert call(**kwargs) == EINVAL and len(L.ga_last_error()) > 0


@pytest.mark.parametrize("call,kwargs", [
    (activation, dict(act=SPARSE)), (product, dict(n=2 ** 31 - 1)), (quantize, dict(rows=2 ** 30, d=300)),
    (dequantize, dict(rows=2 ** 30, d=300)), (activation, dict(rows=2 ** 30, d=300, codes=ctypes.c_void_p(1 << 60)))])
def test_unsupported(call, kwargs):
    assert call(**kwargs) == EUNSUP


def test_no_rows_launch_nothing():
    for call in (forward, quantize, dequantize, activation, product, forward4):
        assert call(rows=0) == OK
    assert forward(rows=0, x=None, y=None, kept=None, ws=None, ws_bytes=0) == OK
    assert product(rows=0, a=None, a_s=None, out=None, ws=None, ws_bytes=0) == OK


def test_workspaces():
    f, b, q = ga.feed_forward_workspace_bytes, ga.feed_forward_backward_workspace_bytes, ga.feed_forward_mxfp4_workspace_bytes
    assert f(0, 64, 64) == 0 and f(4, 65537, 64) == 0 and f(-1, 64, 64) == 0
    for rows in (1, 7, 300, 5000):
        assert f(rows, 512, 1024) >= rows * 1024 * 2
        assert b(rows, 512, 1024) >= rows * 1024 * 6 and b(rows, 512, 1024, "squared_relu") >= rows * 1024 * 4
        assert q(rows, 512, 1024) >= rows * (512 + 1024) // 32 * 17
    assert ga.mxfp4_product_workspace_bytes(0, 5, 5) == 0 and ga.mxfp4_product_workspace_bytes(8192, 8192, 512) == 0
    with pytest.raises(ValueError):
        f(4, 64, 64, "gelu_sparse")


def test_binding_refuses_host_tensors_and_other_activations():
    x, w, wd = torch.zeros(4, 16).bfloat16(), torch.zeros(64, 16).bfloat16(), torch.zeros(16, 32).bfloat16()
    q = ga.Mxfp4(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8), 16)
    for f in (lambda: ga.feed_forward(x, w, wd), lambda: ga.feed_forward_train(x, w, wd),
              lambda: ga.feed_forward_backward(x, x, x, w, wd), lambda: ga.mxfp4_quantize(x),
              lambda: ga.mxfp4_dequantize(q, torch.float32), lambda: ga.activation_mxfp4(x, "silu"),
              lambda: ga.mxfp4_product(q, q), lambda: ga.feed_forward_mxfp4(x, q, q),
              lambda: ga.feed_forward(x, w, wd, "gelu_sparse"), lambda: ga.activation_mxfp4(x, "relu"),
              lambda: ga.mxfp4_dequantize(q, torch.int8), lambda: ga.mxfp4_product(q, q, torch.float64)):
        with pytest.raises(ValueError):
            f()
