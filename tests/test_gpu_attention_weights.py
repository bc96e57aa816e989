"""Paged attention where weights are far apart: many keys far below the row's
largest score, whose share of the result is small but not nothing.

Tolerance: that of test_gpu_paged's header.  It counts the rounding of a
probability to f16 as 2^-11 of it, which holds while what is rounded is normal:
at most 29 powers of two (20 nats) below the row's largest in the kernel for few
rows, 23 (15.9 nats) in the one for many, whose gaps below are chosen within."""
import numpy as np
import pytest
import torch

from paged_cases import Batch
from test_gpu_paged import attend, check_attention

pytestmark = pytest.mark.gpu


def sink(q_lens, kv_lens, gap, **kw):
    """Batches whose first key scores 0 and holds zeros, every other -gap nats (scale 1), their
    values 1 +- a little."""
    from paged_cases import make
    c = Batch(tuple(q_lens), tuple(kv_lens), **kw)
    s = make(c)
    cpu = s["cpu"]
    g = torch.Generator().manual_seed(7)
    k = torch.zeros(s["k_cache"].shape)
    k[..., 0] = -16.0
    v = 1.0 + 0.25 * torch.randn(k.shape, generator=g)
    for b in range(len(kv_lens)):
        k[cpu["table"][b][0], 0] = 0.0
        v[cpu["table"][b][0], 0] = 0.0
    q = torch.zeros(s["q"].shape)
    q[..., 0] = gap / 16.0
    for name, x in (("k_cache", k), ("v_cache", v), ("q", q)):
        s[name].copy_(x.to(s[name].dtype))
        cpu[name] = s[name].double().cpu().numpy()
    if c.fp8:
        s["scale_inv"] = torch.ones(1, device="cuda")
        cpu["inv"] = 1.0
    return c, s


SHAPES = {
    "one": ([1], [250]),
    "one-split": ([1], [20000]),
    "few": ([3, 5], [200, 3000]),
    "many": ([140, 60], [250, 3000]),
    "prompt": ([700], [700]),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,gap", [(n, g) for n in SHAPES
                                       for g in (8, 13, 15 if n in ("many", "prompt") else 17)])
def test_keys_far_below_the_largest_keep_their_share(gpu, shape, gap, dtype, fp8):
    c, s = sink(*SHAPES[shape], gap, heads=4, kv_heads=1, dim=64, dtype=dtype, fp8=fp8)
    out, lse = attend(gpu, c, s, scale=1.0)
    check_attention(c, s, out, lse, 1.0)
    n = s["cpu"]["cu"][-1]
    if gap >= 15 and shape != "prompt":
        assert (out[:n].float() > 0).all()


@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("gap", [17, 20])
def test_the_few_rows_kernel_at_its_limit(gpu, gap, dim):
    c, s = sink([2], [256], gap, heads=2, kv_heads=1, dim=dim, dtype="f16")
    out, lse = attend(gpu, c, s, scale=1.0)
    check_attention(c, s, out, lse, 1.0)


@pytest.mark.parametrize("shape", ["one", "few", "many"])
@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
def test_maxima_that_grow_from_tile_to_tile(gpu, shape, fp8):
    """Scores that rise along the keys, by more than a reference maximum may lag
    behind: every tile moves it."""
    c, s = sink(*SHAPES[shape], 1.0, heads=4, kv_heads=1, dim=64, dtype="f16", fp8=fp8)
    cpu = s["cpu"]
    k = s["k_cache"].float().cpu()
    for b, kv in enumerate(c.kv_lens):
        for t in range(kv):
            k[cpu["table"][b][t // c.page], t % c.page, :, 0] = float(min(t // 4, 400))
    s["k_cache"].copy_(k.to(s["k_cache"].dtype))
    cpu["k_cache"] = s["k_cache"].double().cpu().numpy()
    out, lse = attend(gpu, c, s, scale=1.0)
    check_attention(c, s, out, lse, 1.0)
    assert np.isfinite(lse.double().cpu().numpy()[:cpu["cu"][-1]]).all()
