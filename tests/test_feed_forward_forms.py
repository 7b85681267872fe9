"""The planners of the feed-forward products, on the host: that the cases which the
GPU tests run take every form that there is, past the first steps of its loop; what
the planners refuse; and how large a launch gets."""
import random

import pytest

import feed_forward_forms as forms
import gated_activation_amd as ga


def test_cases_take_every_form():
    covered = set().union(*(forms.layer(*c) for c in forms.LAYERS), *(forms.layer4(*c[:4]) for c in forms.LAYERS4),
                          *(forms.product4(*c) for c in forms.PRODUCTS4))
    rng, met = random.Random(0), {}
    for _ in range(60000):
        kind, sizes = forms.drawn(rng)
        for cell in forms.CELLS[kind](*sizes):
            met.setdefault(cell, (kind, sizes))
    missing = {cell: at for cell, at in met.items() if cell not in covered}
    assert not missing, missing
    # the largest tile in each of its uses, several steps
    for cell in ((16, "hidden", 256, 256, 2), (16, "hidden of one half", 256, 256, 2), (16, "out", 256, 256, 2),
                 (16, "dhidden", 256, 256, 2), (16, "dx", 256, 256, 2), (16, "dw", 256, 256, 2), (4, "hidden", 256, 256, 2),
                 (4, "hidden of one half", 256, 256, 2), (4, "out", 256, 256, 2), (4, "product", 256, 256, 2)):
        assert {cell + ("odd",), cell + ("even",)} <= covered, cell


def test_plans():
    hidden, out, dh, dx, dw_in, dw_down = (ga.plan_feed_forward(8192, 4096, 16384, "silu", i).as_dict() for i in range(6))
    for p, k, grid in ((hidden, 4096, 32 * 128), (out, 16384, 32 * 16), (dh, 4096, 32 * 64), (dx, 32768, 32 * 16),
                       (dw_in, 8192, 16 * 128), (dw_down, 8192, 64 * 16)):
        assert p == dict(features=256, tokens=256, stages=2, k_step=64, splits=1, joint=0, k_slice=k, grid=grid)
    assert ga.plan_feed_forward(1, 2048, 16384, "gelu", ga.GA_PRODUCT_HIDDEN).features == 0
    p = ga.plan_feed_forward(64, 4096, 8192, "silu", ga.GA_PRODUCT_OUT, bits=4)
    assert p.k_step == 256 and p.splits > 1 and p.k_slice % 256 == 0 and (p.splits - 1) * p.k_slice < 8192 <= p.splits * p.k_slice
    # the two calls take the same plan of the same product
    assert ga.plan_mxfp4_product(64, 4096, 8192).as_dict() == p.as_dict()
    assert [ga.plan_feed_forward(128, 512, 1024, "silu", i).joint for i in range(6)] == [0, 0, 0, 1, 1, 1]


@pytest.mark.parametrize("args", [(0, 64, 64, "silu", 0), (2 ** 31, 64, 64, "silu", 0), (4, 60, 64, "silu", 0), (4, 64, 65544, "silu", 0),
                                  (4, 64, 64, "silu", 6), (4, 64, 64, "silu", -1), (4, 64, 64, "silu", 2, 4), (4, 64, 40, "silu", 0, 4),
                                  (4, 64, 64, "silu", 0, 8)])
def test_refused(args):
    with pytest.raises(ga.GaError):
        ga.plan_feed_forward(*args)


def test_products_refused():
    for args in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 2 ** 31, 4), (4, 4, 65537)):
        with pytest.raises(ga.GaError):
            ga.plan_mxfp4_product(*args)
    with pytest.raises(ValueError):
        ga.plan_feed_forward(4, 64, 64, "gelu_sparse", 0)
    assert ga.lib.ga_plan_mxfp4_product(4, 4, 4, None) == ga.GA_EINVAL
    assert ga.lib.ga_plan_feed_forward(4, 64, 64, 0, 16, 0, None) == ga.GA_EINVAL


def _items(p):
    return p.grid * (512 if p.features in (0, 256) else 256)


def test_launches_that_the_header_promises():
    """rows * max(H, d) of 2^36 or less, and rows * n of 2^37 past 16 rows, stay below 2^32 work-items."""
    rng, most = random.Random(1), 2 ** 31 - 1025
    for _ in range(20000):
        act, bits = rng.choice(["silu", "squared_relu"]), rng.choice([4, 16])
        H, d = 8 * forms.log_int(rng, 1, 8192), 32 * forms.log_int(rng, 1, 2048)
        rows = min(most, 2 ** 36 // max(H, d))
        for i in range(2 if bits == 4 else 6):
            assert _items(ga.plan_feed_forward(rows, H, d, act, i, bits)) < 2 ** 32, (rows, H, d, act, i, bits)
        rows = forms.log_int(rng, 17, most)
        n = min(most, 2 ** 37 // rows)
        for r, m in ((rows, n), (max(17, n), min(rows, 2 ** 37 // max(17, n)))):
            if m >= 1:
                assert _items(ga.plan_mxfp4_product(r, m, 4096)) < 2 ** 32, (r, m)
