"""The feed-forward products in every form that the planner has for them, several
steps of k in each (needs an MI355X).  That the cases take them all is tested on the
host; bounds: feed_forward_ref."""
import pytest

import feed_forward_forms as forms
from test_gpu_feed_forward import check
from test_gpu_mxfp4 import _layer
from test_gpu_mxfp4 import test_product as check_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,H,d,act,live", forms.LAYERS)
def test_layer(rows, H, d, act, live, dtype):
    print(f"feed forward {act} {dtype} {rows}x{H}x{d} live {live}", flush=True)
    check(rows, H, d, act, dtype, live)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,H,d,act,live", forms.LAYERS4)
def test_4_bit_layer(rows, H, d, act, live, dtype):
    print(f"4-bit layer {act} {dtype} {rows}x{H}x{d} live {live}", flush=True)
    _layer(act, rows, H, d, live, dtype)


@pytest.mark.parametrize("rows,n,k", forms.PRODUCTS4)
def test_4_bit_product(rows, n, k):
    check_product(rows, n, k)
