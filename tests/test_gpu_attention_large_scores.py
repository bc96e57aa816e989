"""Paged attention with scores so large that their own rounding exceeds one: the
largest key takes the whole weight, and the row is that key's values.

Every score is exact in fp32 and the second largest at least 2^18 below the
largest, so the weights are 1 and 0 and the result is the value itself: within the
stored rounding, that of the probability (eps / 2 each, the latter of the values'
type) and 24 of fp32.  Rows of zeros among them keep every key alike: the mean of
their values, within the same and 2^-23 for each of n / 16 steps, relative to the mean
of |v|."""
import numpy as np
import pytest
import torch

from paged_cases import Batch, DT, make
from test_gpu_paged import attend

pytestmark = pytest.mark.gpu


def batch(order, q_lens, kv_lens, fp8, dtype):
    """(case, tensors, the call's scales, each row's largest key and how often its size occurs)."""
    c = Batch(tuple(q_lens), tuple(kv_lens), heads=4, kv_heads=1, dim=64, dtype=dtype, fp8=fp8)
    s = make(c)
    cpu = s["cpu"]
    g = torch.Generator().manual_seed(11)
    # Eight elements of a key hold its size: whole multiples of a step of the type, all distinct.
    if fp8:
        codes = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        sizes = codes[codes >= 2.0 ** -3]              # 95 of them: more keys repeat the smallest
    elif dtype == "f16":
        sizes = 2.0 ** 14 - 8.0 * torch.arange(1000)
    else:
        sizes = torch.outer(2.0 ** torch.arange(7, 15), 1 + torch.arange(128) / 128.0).flatten()
    sizes = sizes.sort(descending=True).values
    k = torch.zeros(s["k_cache"].shape)
    best = []
    for b, kv in enumerate(c.kv_lens):
        mine = sizes[torch.arange(kv).clamp(max=len(sizes) - 1)]
        mine = mine.flip(0) if order == "rising" else mine[torch.randperm(kv, generator=g)]
        for t in range(kv):
            k[cpu["table"][b][t // c.page], t % c.page, 0, :8] = mine[t]
        best.append([(int(mine[:n].argmax()), int((mine[:n] == mine[:n].max()).sum()))
                     for n in range(1, kv + 1)])
    q = torch.zeros(s["q"].shape)
    large = 2.0 ** 15 if dtype == "f16" else 2.0 ** 21
    q[:, ::2, :8] = large                              # heads 0 and 2; 1 and 3 are zeros
    for name, x in (("k_cache", k), ("q", q)):
        s[name].copy_(x.to(s[name].dtype))
    one = torch.ones(1, device="cuda")
    kw = dict(k_scale_inv=one * 2.0 ** 8, v_scale_inv=one) if fp8 else {}
    return c, s, kw, best


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3], [90, 100]), ([1], [300]), ([80, 100], [90, 100]),
                                            ([200], [700])], ids=["few", "one", "many", "chunk"])
@pytest.mark.parametrize("order", ["mixed", "rising"])
def test_the_largest_score_takes_all(gpu, order, q_lens, kv_lens, fp8, dtype):
    c, s, kw, best = batch(order, q_lens, kv_lens, fp8, dtype)
    cpu = s["cpu"]
    out, lse = attend(gpu, c, s, scale=1.0, **kw)
    o = out.cpu()
    v = s["v_cache"].float().cpu()
    eps = torch.finfo(DT[dtype]).eps / 2                               # of what is stored
    half = torch.finfo(torch.float16 if fp8 else DT[dtype]).eps / 2   # of a probability
    row, seen = 0, 0
    for b, (n, kv) in enumerate(zip(c.q_lens, c.kv_lens)):
        vals = torch.stack([v[cpu["table"][b][t // c.page], t % c.page, 0] for t in range(kv)])
        for i in range(n):
            keys = kv - n + i + 1
            at, times = best[b][keys - 1]
            if times == 1:   # (rows whose largest repeats are left out)
                seen += 1
                near = vals[at].double().abs() * ((eps + half) * (1 + eps) + 24 * 2.0 ** -23) + 2.0 ** -25
                for h in (0, 2):
                    assert ((o[row, h].double() - vals[at].double()).abs() <= near).all(), (b, i, h)
            mean, size = vals[:keys].double().mean(0), vals[:keys].double().abs().mean(0)
            inner = size * (half + (keys / 16 + 24) * 2.0 ** -23)
            lim = eps * (mean.abs() + inner) + inner + 2.0 ** -25
            for h in (1, 3):
                assert ((o[row, h].double() - mean).abs() <= lim).all(), (b, i, h)
            row += 1
    assert seen > 0 and np.isfinite(lse.cpu().numpy()).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([4, 3], [90, 100]), ([16], [300]), ([80, 100], [90, 100]),
                                            ([200], [700])], ids=["few", "more", "many", "chunk"])
def test_next_to_a_bad_value_that_the_row_drops(gpu, q_lens, kv_lens, fp8, dtype):
    """The last key's values are NaN: rows before it are what they were."""
    c, s, kw, best = batch("mixed", q_lens, kv_lens, fp8, dtype)
    cpu = s["cpu"]
    clean, _ = attend(gpu, c, s, scale=1.0, **kw)
    v = s["v_cache"].float().cpu()
    for b, kv in enumerate(c.kv_lens):
        v[cpu["table"][b][(kv - 1) // c.page], (kv - 1) % c.page] = float("nan")
    s["v_cache"].copy_(v.to(s["v_cache"].dtype))
    out, _ = attend(gpu, c, s, scale=1.0, **kw)
    eps = torch.finfo(DT[dtype]).eps
    row, seen = 0, 0
    for b, (n, kv) in enumerate(zip(c.q_lens, c.kv_lens)):
        for i in range(n - 1):
            if best[b][kv - n + i][1] == 1:
                seen += 1
                # (both within the first test's distance of the exact value)
                a, e = out[row + i, ::2].double(), clean[row + i, ::2].double()
                assert ((a - e).abs() <= 2 * (e.abs() * 2.1 * eps + 2.0 ** -25)).all(), (b, i)
            assert torch.isfinite(out[row + i]).all()
        row += n
    assert seen > 0
