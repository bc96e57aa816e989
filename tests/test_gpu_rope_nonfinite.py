"""Frequencies that are not numbers."""
import pytest
import torch

from paged_cases import Batch, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_frequencies_that_are_no_numbers_show(gpu, bad):
    """The pair that has such a frequency comes out as NaN, the others as they were."""
    d = 16
    g = torch.Generator().manual_seed(6)
    q = torch.randn(2, 5, 3, d, generator=g).cuda()
    f = gpu.rope_frequencies(d)
    want, _ = gpu.rope_fwd(q, None, f)
    f[3] = bad
    for fn in (gpu.rope_fwd, gpu.rope_bwd):
        got, _ = fn(q, None, f, layout="half")
        hit = torch.zeros(d, dtype=torch.bool)
        hit[[3, 3 + d // 2]] = True
        assert torch.isnan(got[..., hit]).all() and torch.isfinite(got[..., ~hit]).all()
    got, _ = gpu.rope_fwd(q, None, f)
    assert torch.equal(got[..., ~hit], want[..., ~hit])
    c = Batch((2, 3), (20, 40), dim=d)
    s = make(c)
    qo = gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                          s["table"], q=s["q"], inv_freq=f)
    assert torch.isnan(qo[..., hit]).all() and torch.isfinite(qo[..., ~hit]).all()
