"""The range of the attention's scale, as the C entry checks it."""
import math

import pytest

from test_paged_cpu import _attend


@pytest.fixture(scope="module")
def G():
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import gbnorm
    return gbnorm


def test_scale_times_log2_e_is_finite(G):
    largest = 3.4028234663852886e38
    for bad in (largest, 3.0e38, largest / math.log2(math.e) * 1.00001):
        assert _attend(G, scale=bad) == G.GBN_ERR_SHAPE, bad
    for fine in (largest / math.log2(math.e) * 0.99999, 1.0, 1e-45):
        assert _attend(G, scale=fine) == G.GBN_ERR_NULL, fine   # the next check
