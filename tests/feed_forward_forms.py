"""Which forms the planner of the feed-forward products can choose, as cells: an
epilogue or the layout of the operands, a tile, whether k is cut and, where it is
not, whether its steps are odd or even (the loops take two at a time).  A product
of fewer than LEAST steps (a slice) is in no cell: it never gets to the middle of
its pipeline."""
import math

import gated_activation_amd as ga

LEAST = {16: 3, 4: 5}   # steps; in 4 bits past two windows of scales

# rows, H, d, activation, live: 16 bits, forward and backward.
LAYERS = [
    (17, 152, 8, "silu", None), (18, 1040, 8, "gelu_tanh", None), (17, 136, 160, "squared_relu", 16),
    (20, 216, 208, "gelu", None), (138, 136, 160, "squared_relu", None), (1, 280, 11688, "silu", None),
    (961, 8, 504, "gelu_tanh", 855), (19, 200, 1176, "squared_relu", None), (1, 6368, 904, "squared_relu", None),
    (218, 152, 248, "gelu", None), (145, 216, 976, "silu", 129), (963, 240, 136, "squared_relu", None),
    (840, 5960, 8, "gelu_tanh", None), (914, 5600, 8, "gelu", None), (1603, 3232, 8, "squared_relu", 1425),
    (74, 208, 8512, "silu", None), (23, 7384, 896, "squared_relu", None), (71, 200, 16688, "gelu_tanh", None),
    (107, 136, 16728, "gelu", 96), (10666, 136, 168, "silu", None), (199, 152, 8608, "squared_relu", None),
    (305, 6944, 168, "gelu_tanh", None), (326, 5608, 224, "gelu", 250), (150, 136, 22496, "silu", None),
    (13254, 136, 264, "squared_relu", None), (142, 7000, 560, "gelu_tanh", None), (6916, 1168, 72, "gelu", 6148),
    (204, 184, 16520, "silu", None), (11121, 200, 304, "squared_relu", None),
    (221, 152, 20240, "squared_relu", None), (10964, 456, 152, "squared_relu", 9746),
    (11442, 672, 104, "gelu_tanh", None), (243, 224, 17280, "gelu", None), (903, 136, 8368, "silu", None),
    (12459, 200, 432, "squared_relu", 11075), (10093, 536, 208, "squared_relu", None),
    (514, 6536, 344, "gelu_tanh", None), (11455, 616, 176, "gelu", None), (426, 136, 23656, "squared_relu", 379),
    (532, 208, 13952, "silu", None), (12348, 968, 136, "gelu_tanh", None), (397, 208, 25640, "squared_relu", None),
    (14213, 784, 200, "gelu", 12634),
]
# rows, H, d, activation, live: in 4 bits.
LAYERS4 = [
    (1, 8, 32, "silu", None), (1, 8, 32, "squared_relu", None), (17, 1304, 32, "squared_relu", 16),
    (18, 4032, 32, "gelu_tanh", None), (70, 8, 4800, "gelu", None), (17, 5744, 32, "squared_relu", None),
    (70, 1464, 32, "squared_relu", 63), (87, 1288, 32, "silu", None), (71, 3928, 32, "squared_relu", None),
    (65, 4328, 32, "gelu_tanh", None), (17, 1136, 1184, "squared_relu", 16), (25, 1144, 1312, "gelu", None),
    (65, 1088, 1088, "squared_relu", None), (18, 1360, 3872, "silu", None), (76, 1240, 1440, "gelu_tanh", 68),
    (68, 1224, 8416, "gelu", None), (73, 1384, 9408, "silu", None), (85, 1288, 16736, "squared_relu", None),
    (80, 1456, 17216, "gelu_tanh", 72), (1874, 1208, 1088, "squared_relu", None), (1794, 1064, 1536, "gelu", None),
    (11346, 1424, 288, "squared_relu", None), (181, 1440, 17920, "silu", 161),
    (3786, 1152, 1184, "squared_relu", None), (3605, 1040, 1504, "gelu_tanh", None),
    (385, 1064, 17088, "squared_relu", None), (13660, 520, 1088, "gelu", 12143),
    (385, 1288, 17088, "squared_relu", None), (13660, 520, 1312, "silu", None),
]
# rows, n, k
PRODUCTS4 = [
    (1, 1, 1), (20, 1, 1027), (21, 1, 1394), (18, 1, 4403), (69, 1, 1316), (68, 1, 1566), (70, 1, 4011),
    (8309, 136, 1160), (67, 19408, 1413), (210, 17274, 1100), (149, 22029, 1451), (4714, 1674, 1096),
    (412, 21649, 1290),
]


def _cell(p, kind, k, bits):
    if p.features == 0:
        return bits, kind, "stream"
    steps = p.k_slice // p.k_step if p.splits > 1 else -(-k // p.k_step)
    if steps < LEAST[bits]:
        return None
    return bits, kind, p.features, p.tokens, p.stages, "cut" if p.splits > 1 else ("even", "odd")[steps % 2]


def layer(rows, H, d, act, live=None):
    """The cells of a layer's forward and backward pass in 16 bits."""
    live = rows if live is None else live
    zd = d if act == "squared_relu" else 2 * d
    single = " of one half" if act == "squared_relu" else ""
    plans = [ga.plan_feed_forward(rows, H, d, act, i) for i in range(6)]
    names = ["hidden" + single, "out", "dhidden" + single, "dx", "dw", "dw"]
    if plans[3].joint:
        both = f" joint, x {'cut' if plans[3].splits > 1 else 'whole'}, w {'cut' if plans[4].splits > 1 else 'whole'}"
        names[3:] = [n + both for n in names[3:]]
    cells = {_cell(p, n, k, 16) for p, n, k in zip(plans, names, (H, d, H, zd, live, live))}
    return cells - {None}


def layer4(rows, H, d, act):
    single = " of one half" if act == "squared_relu" else ""
    plans = [ga.plan_feed_forward(rows, H, d, act, i, bits=4) for i in (ga.GA_PRODUCT_HIDDEN, ga.GA_PRODUCT_OUT)]
    return {_cell(plans[0], "hidden" + single, H, 4), _cell(plans[1], "out", d, 4)} - {None}


def product4(rows, n, k):
    return {_cell(ga.plan_mxfp4_product(rows, n, k), "product", k, 4)} - {None}


def log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def drawn(rng):
    """A layer or product of any size that the planner meets: (kind, arguments)."""
    rows, act = log_int(rng, 1, 16384), rng.choice(["silu", "squared_relu"])
    kind = rng.choice(["layer", "layer", "layer4", "product4"])
    if kind == "layer":
        return kind, (rows, 8 * log_int(rng, 1, 1024), 8 * log_int(rng, 1, 4096), act)
    if kind == "layer4":
        return kind, (rows, 8 * log_int(rng, 1, 1024), 32 * log_int(rng, 1, 1024), act)
    return kind, (rows, log_int(rng, 1, 32768), log_int(rng, 1, 32768))


CELLS = {"layer": layer, "layer4": layer4, "product4": product4}
