"""The widest 4-bit product that a launch holds (needs an MI355X)."""
import numpy as np
import pytest
import torch

import feed_forward_ref as ff
import gated_activation_amd as ga
from train_gpu import close, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 16])
def test_widest_product_of_few_rows(rows):
    """A weight whose rows repeat: so must the outputs, up to the last."""
    n, k, block = 2 ** 27 - 16, 32, 752
    a = ga.mxfp4_quantize(values(np.random.default_rng(1), (rows, k), "bf16")[0].cuda())
    part = ga.mxfp4_quantize(values(np.random.default_rng(2), (block, k), "bf16")[0].cuda())
    assert n % block == 0
    w = ga.Mxfp4(part.codes.repeat(n // block, 1), part.scales.repeat(n // block, 1), k)
    print(f"product {rows}x{n}x{k}", flush=True)
    out = ga.mxfp4_product(a, w, torch.bfloat16).view(rows, -1, block)
    want, bound = ff.product4(*(ga.mxfp4_dequantize(q, torch.float32).double().cpu().numpy() for q in (a, part)), "bf16")
    close(out[:, 0].contiguous(), want, bound, "product")
    assert bool((out == out[:, :1]).all())
    del out, w
    torch.cuda.empty_cache()
