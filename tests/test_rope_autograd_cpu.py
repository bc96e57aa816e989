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


@pytest.mark.parametrize("need", [(True, False), (False, True), (True, True)])
def test_only_the_gradients_that_are_needed_are_rotated(rope, need):
    f = torch.ones(4, dtype=torch.float64)
    q = torch.randn(1, 2, 3, 8).requires_grad_(need[0])
    k = torch.randn(1, 2, 1, 8).requires_grad_(need[1])
    a, b = rope[0](q, k, f)
    (a.sum() + b.sum()).backward()
    assert rope[1] == [(False, True, True), (True, *need)]
    assert (q.grad is not None, k.grad is not None) == need
