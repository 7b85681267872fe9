"""The training entry points on the host: every call below is refused by a
check, or has no rows, before the library makes any HIP call."""
import ctypes

import pytest
import torch

import gated_activation_amd as ga

L = ga.lib
OK, EINVAL, EUNSUP = ga.GA_OK, ga.GA_EINVAL, ga.GA_EUNSUPPORTED
BF16, F32 = ga.GA_BF16, ga.GA_F32


def P(i, add=0):
    """Fake device addresses 1 TiB apart; never dereferenced."""
    return ctypes.c_void_p((0x100 + i) * (1 << 40) + add)


NAN, INF = float("nan"), float("inf")


def store(x=P(0), codes=P(1), scales=P(2), rows=4, d=256, dt=BF16, live=None):
    return L.ga_checkpoint_store(x, codes, scales, rows, d, dt, live, None)


def restore(codes=P(1), scales=P(2), stats=None, out=P(3), rows=4, d=256, halves=1, dt=BF16, live=None):
    return L.ga_checkpoint_restore(codes, scales, stats, out, rows, d, halves, dt, live, None)


def forward(x=P(0), out=P(3), codes=P(1), scales=P(2), stats=P(4), rows=4, d=256, dt=BF16, act=0, z=1.6, live=None):
    return L.ga_activation_checkpoint(x, out, codes, scales, stats, rows, d, dt, act, z, live, None)


def backward(dout=P(5), x=P(0), dx=P(6), rows=4, d=256, dt=BF16, act=0, z=1.6, live=None):
    return L.ga_activation_backward(dout, x, dx, rows, d, dt, act, z, live, None)


def backward8(dout=P(5), codes=P(1), scales=P(2), stats=P(4), dx=P(6), rows=4, d=256, dt=BF16, act=0, z=1.6, live=None):
    return L.ga_activation_backward_checkpoint(dout, codes, scales, stats, dx, rows, d, dt, act, z, live, None)


def norm(x=P(0), w=P(7), b=P(8), out=P(3), stats=P(4), rows=4, d=256, dt=BF16, wdt=BF16, eps=1e-5, live=None):
    return L.ga_layer_norm(x, w, b, out, stats, rows, d, dt, wdt, eps, live, None)


def norm8(x=P(0), w=P(7), b=P(8), out=P(3), codes=P(1), scales=P(2), stats=P(4), rows=4, d=256, dt=BF16, wdt=BF16, eps=1e-5):
    return L.ga_layer_norm_checkpoint(x, w, b, out, codes, scales, stats, rows, d, dt, wdt, eps, None, None)


def norm_back(dout=P(5), x=P(0), stats=P(4), w=P(7), dx=P(6), dw=P(9), db=P(10), rows=4000, d=256, dt=BF16, wdt=BF16,
              live=None, ws=P(11), ws_bytes=1 << 30):
    return L.ga_layer_norm_backward(dout, x, stats, w, dx, dw, db, rows, d, dt, wdt, live, ws, ws_bytes, None)


def norm_back8(dout=P(5), codes=P(1), scales=P(2), stats=P(4), w=P(7), dx=P(6), dw=P(9), db=P(10), rows=4000, d=256,
               dt=BF16, wdt=BF16, ws=P(11), ws_bytes=1 << 30):
    return L.ga_layer_norm_backward_checkpoint(dout, codes, scales, stats, w, dx, dw, db, rows, d, dt, wdt, None, ws,
                                               ws_bytes, None)


def balance(logits=P(0), index=P(1), ib=8, mask=None, loss=P(2), counts=P(3), offsets=P(4), tokens=P(5), rows=4096, e=64,
            k=2, dt=BF16, c=1.0, live=None, ws=P(6), ws_bytes=1 << 30):
    return L.ga_balance_loss(logits, index, ib, mask, loss, counts, offsets, tokens, rows, e, k, dt, c, live, ws, ws_bytes,
                             None)


def balance_back(logits=P(0), mask=None, counts=P(3), offsets=P(4), tokens=P(5), dloss=P(7), dlogits=P(8), rows=64, e=64,
                 k=2, dt=BF16, c=1.0, live=None):
    return L.ga_balance_loss_backward(logits, mask, counts, offsets, tokens, dloss, dlogits, rows, e, k, dt, c, live, None)


ROWWISE = [store, restore, forward, backward, backward8, norm, norm8, norm_back, norm_back8]


@pytest.mark.parametrize("call", ROWWISE)
@pytest.mark.parametrize("kwargs,status", [(dict(rows=-1), EINVAL), (dict(rows=2 ** 31), EINVAL), (dict(d=0), EINVAL),
                                           (dict(d=-3), EINVAL), (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL),
                                           (dict(d=65537), EUNSUP)])
def test_sizes_and_types(call, kwargs, status):
    assert call(**kwargs) == status and len(L.ga_last_error()) > 0


@pytest.mark.parametrize("call,pointers", [
    (store, ["x", "codes", "scales"]), (restore, ["codes", "scales", "out"]), (forward, ["x", "out", "codes", "scales"]),
    (backward, ["dout", "x", "dx"]), (backward8, ["dout", "codes", "scales", "dx"]), (norm, ["x", "w", "out", "stats"]),
    (norm8, ["x", "w", "out", "codes", "scales", "stats"]), (norm_back, ["dout", "x", "stats", "w", "dx", "dw", "ws"]),
    (norm_back8, ["dout", "codes", "scales", "stats", "w", "dx", "dw", "ws"]),
    (balance, ["logits", "index", "loss", "counts", "offsets", "tokens", "ws"]),
    (balance_back, ["logits", "counts", "offsets", "tokens", "dloss", "dlogits"])])
def test_null_pointers(call, pointers):
    for p in pointers:
        assert call(**{p: None}) == EINVAL, p


@pytest.mark.parametrize("call,kwargs", [
    (store, dict(x=P(0, 1))), (store, dict(scales=P(2, 2))), (store, dict(live=P(9, 2))), (restore, dict(out=P(3, 1))),
    (restore, dict(halves=3)), (restore, dict(halves=0)), (restore, dict(stats=P(4, 1))),
    (forward, dict(act=5)), (forward, dict(act=-1)), (forward, dict(act=4, z=NAN)), (forward, dict(act=4, z=INF)),
    (forward, dict(act=4, stats=None)), (forward, dict(out=P(0))), (forward, dict(codes=P(0, 4 * 256 * 2 * 2 - 1))),
    (backward, dict(dx=P(0))), (backward, dict(dx=P(5, 2))), (backward, dict(act=7)), (backward8, dict(act=4, stats=None)),
    (backward8, dict(dx=P(1))), (norm, dict(wdt=ga.GA_F16)), (norm, dict(eps=-1.0)), (norm, dict(eps=NAN)),
    (norm, dict(eps=INF)), (norm, dict(dt=F32, wdt=BF16)), (norm, dict(out=P(0))), (norm, dict(stats=P(7, 4))),
    (norm_back, dict(ws_bytes=64)), (norm_back, dict(ws=P(11, 8))), (norm_back, dict(ws=P(6))), (norm_back, dict(dw=P(10))),
    (norm_back, dict(dx=P(5))), (norm_back8, dict(ws_bytes=0)),
    (balance, dict(ib=2)), (balance, dict(ib=8, index=P(1, 4))), (balance, dict(rows=-1)), (balance, dict(e=0)),
    (balance, dict(k=0)), (balance, dict(c=NAN)), (balance, dict(dt=9)), (balance, dict(ws_bytes=16)),
    (balance, dict(counts=P(4))), (balance, dict(live=P(12, 1))), (balance_back, dict(dlogits=P(0))),
    (balance_back, dict(c=INF)), (balance_back, dict(dloss=P(7, 2)))])
def test_malformed(call, kwargs):
    assert call(**kwargs) == EINVAL and len(L.ga_last_error()) > 0


@pytest.mark.parametrize("call,kwargs", [
    (norm, dict(d=32769)), (norm_back, dict(d=40000)), (balance, dict(e=1025)), (balance, dict(rows=2 ** 30, k=2)),
    (store, dict(rows=2 ** 30, d=300)), (backward, dict(rows=2 ** 30, d=300)), (forward, dict(rows=2 ** 22, d=16384, act=4)),
    (backward, dict(rows=2 ** 26, d=1, act=4)), (norm, dict(rows=2 ** 28, d=100)), (norm, dict(rows=2 ** 26, d=512)),
    (restore, dict(rows=2 ** 30, d=128, halves=2))])
def test_unsupported(call, kwargs):
    assert call(**kwargs) == EUNSUP


def test_no_rows_launch_nothing():
    for call in (store, restore, forward, backward, backward8, norm, norm8, balance_back):
        assert call(rows=0) == OK
    assert forward(rows=0, x=None, out=None, codes=None, scales=None, act=4, stats=None) == OK


def test_workspaces():
    w = ga.layer_norm_backward_workspace_bytes
    assert w(0, 100) == 0 and w(1, 100) == 0 and w(10 ** 6, 40000) == 0
    assert w(10 ** 6, 4096) % (2 * 4096 * 4) == 0 and w(10 ** 6, 4096) >= w(100, 4096) > 0
    b = ga.balance_loss_workspace_bytes
    assert b(0, 8) == 0 and b(64, 8) == 0 and b(65536, 128) > 0 and b(100, 1025) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    i = torch.zeros(4, 2, dtype=torch.int64)
    c = ga.Checkpoint(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1))
    for f in (lambda: ga.checkpoint_store(x), lambda: ga.checkpoint_restore(c, torch.float32),
              lambda: ga.activation_checkpoint(x, "silu"), lambda: ga.activation_backward(x, x, "squared_relu"),
              lambda: ga.layer_norm(x, w), lambda: ga.layer_norm_checkpoint(x, w),
              lambda: ga.layer_norm_backward(x, x, w, stats=torch.zeros(4, 2)), lambda: ga.balance_loss(x, i),
              lambda: ga.activation_checkpoint(x, "relu"), lambda: ga.checkpoint_restore(c, torch.float64)):
        with pytest.raises(ValueError):
            f()
