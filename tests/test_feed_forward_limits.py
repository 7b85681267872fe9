"""How large the feed-forward products get, on the host: with no rows every call ends
after its checks."""
import pytest

import gated_activation_amd as ga
from test_feed_forward_abi import EUNSUP, OK, P, backward, forward, forward4, product


def test_widest_product_of_few_rows():
    """16 features a workgroup of 512 work-items, of which a launch has fewer than 2^32."""
    for n in (4096, 70_000_000, 2 ** 27 - 17, 2 ** 27 - 16):
        assert product(rows=0, n=n, d=32) == OK, n
    for n in (2 ** 27 - 15, 2 ** 27, 2 ** 31 - 1025):
        assert product(rows=0, n=n, d=32) == EUNSUP, n
        assert b"work-items" in ga.lib.ga_last_error(), n
    assert product(rows=0, n=2 ** 31 - 1024, d=32) == EUNSUP


@pytest.mark.parametrize("call,kwargs", [(forward, {}), (backward, {}), (forward4, dict(d=32)), (product, dict(n=8, d=32))])
def test_most_rows(call, kwargs):
    """Rows are counted a few tiles past their end."""
    apart = {k: P(16 * i) for i, k in enumerate({
        forward: ("x", "w_in", "w_down", "y", "kept", "ws"),
        backward: ("dy", "x", "kept", "w_in", "w_down", "dx", "dw_in", "dw_down", "ws"),
        forward4: ("x", "w_in", "w_in_s", "w_down", "w_down_s", "y", "ws"),
        product: ("a", "a_s", "w", "w_s", "out", "ws")}[call])}
    if call is not product:
        kwargs = dict(kwargs, H=8, **({} if "d" in kwargs else {"d": 8}))
    assert call(rows=2 ** 31 - 1024, ws_bytes=1 << 42, **kwargs, **apart) == EUNSUP
    assert b"rows" in ga.lib.ga_last_error()
