"""The "yarn" frequencies where even the slowest pair turns often."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import ops as o
    return o


@pytest.mark.parametrize("dim,base,factor,length", [(128, 10000.0, 4.0, 131072), (128, 10000.0, 4.0, 65536),
                                                    (64, 10000.0, 8.0, 65536), (128, 500000.0, 8.0, 8192),
                                                    (64, 10000.0, 4.0, 4096), (8, 100.0, 2.0, 10 ** 7)])
def test_yarn_ramp_ends_beyond_the_last_pair(ops, dim, base, factor, length):
    """The ramp over the pair's index from the one that turns 32 times within the length (rounded
    down) to the one that turns once (rounded up), the latter bounded by the number of elements:
    a pair that turns oftener than once is not divided by the whole factor."""
    got = ops.rope_frequencies(dim, base, scaling="yarn", factor=factor, original_length=length,
                               device="cpu")

    def index(turns):
        return dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(32)), 0), min(math.ceil(index(1)), dim - 1)
    for i in range(dim // 2):
        plain = base ** (-2.0 * i / dim)
        ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        want = plain * (1 - ramp) + plain / factor * ramp
        # (two fp64 evaluations: a power and five roundings, 2^-53 each)
        assert abs(float(got[i]) - want) <= 16 * 2.0 ** -53 * plain, i
        if length * plain / (2 * math.pi) > 1.5:
            assert float(got[i]) > plain / factor
    assert got.dtype == torch.float64


def test_yarn_of_the_slowest_pair(ops):
    f = ops.rope_frequencies(128, scaling="yarn", factor=4.0, original_length=131072, device="cpu")
    plain = ops.rope_frequencies(128, device="cpu")
    # It turns 2.4 times; from index 45 (32 turns) to 70 (one) the ramp is 18 / 25 at 63.
    assert abs(float(f[63] / plain[63]) - (7 / 25 + 18 / 25 / 4)) < 1e-12
