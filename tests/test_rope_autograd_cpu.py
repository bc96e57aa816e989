"""What the rotation's autograd function has a gradient for, with a stand-in for the
library."""
import pytest
import torch


@pytest.fixture
def rope(monkeypatch):
    """(autograd.rope, the calls its library gets: backward, q given, k given)."""
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    calls = []

    class Fake:
        def rope_fwd(self, q, k, f, pos, *, layout, mscale):
            calls.append((False, q is not None, k is not None))
            return tuple(None if t is None else t * 2 for t in (q, k))

        def rope_bwd(self, q, k, f, pos, *, layout, mscale):
            calls.append((True, q is not None, k is not None))
            return tuple(None if t is None else t * 2 for t in (q, k))

    monkeypatch.setattr(A, "ops", Fake())
    return A.rope, calls


def test_frequencies_that_require_a_gradient_are_refused(rope):
    f = torch.ones(4, dtype=torch.float64)
    q, k = torch.randn(1, 2, 3, 8, requires_grad=True), torch.randn(1, 2, 1, 8)
    with pytest.raises(ValueError, match="inv_freq"):
        rope[0](q, k, f.clone().requires_grad_())
    assert rope[1] == []
    with torch.no_grad():   # nothing is asked of them
        rope[0](q, k, f.clone().requires_grad_())
    assert rope[0](q, k, f)[0].requires_grad
