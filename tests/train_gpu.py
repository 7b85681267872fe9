"""Shared by the GPU tests of the training operators: inputs, canaries, and
element-wise comparison with a bound."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TAIL = 512
PAD = 77          # what untouched rows and tails hold (exact in every type)


def values(rng, shape, dtype, mean=0.0, std=1.0):
    """A CPU tensor of the type and its exact values in fp64."""
    t = torch.from_numpy(rng.normal(mean, std, shape).astype(np.float32)).to(TYPES[dtype])
    return t, t.double().numpy()


def guarded(shape, dtype, offset=0):
    """A contiguous CUDA tensor `offset` elements into a larger one, all of it PAD."""
    n = int(np.prod(shape))
    buf = torch.full((offset + n + TAIL,), PAD, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + n].view(*shape)


def placed(t, offset):
    """t's values on the GPU, `offset` elements into their buffer."""
    buf, v = guarded(tuple(t.shape), t.dtype, offset)
    v.copy_(t)
    return v


def check_guard(buf, n, offset=0):
    assert bool((buf[:offset] == PAD).all()) and bool((buf[offset + n:] == PAD).all()), "written outside the array"


def live_tensor(n):
    return None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")


def close(got, want, bound, label):
    g = got.detach().double().cpu().numpy().reshape(np.shape(want))
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{label}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(g[inf], np.asarray(want)[inf]), f"{label}: infinities differ"
    ok = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        off = np.where(ok, np.abs(g - want) - bound, -1.0)
    if off.size and off.max() > 0:
        i = np.unravel_index(np.argmax(off), off.shape)
        raise AssertionError(f"{label}: {int((off > 0).sum())} of {off.size} out of bound, at {tuple(map(int, i))} got {g[i]!r} "
                             f"want {np.asarray(want)[i]!r} bound {np.broadcast_to(bound, off.shape)[i]!r}")


def untouched(t, live, label):
    assert bool((t[live:] == PAD).all()), f"{label}: rows past the live count were written"
