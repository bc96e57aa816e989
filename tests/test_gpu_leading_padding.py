"""Rows before the first sequence (cu_seqlens[0] > 0) are padding like those behind
the last: no error flag, nothing written, the sequences' own results as without
them."""
import pytest
import torch

from paged_cases import DT, Batch, make
from test_gpu_paged import attend, check_append, check_attention, device_flags

pytestmark = pytest.mark.gpu

LEAD = 5


def shifted(c):
    """make(c), and the same with LEAD rows in front."""
    s = make(c)
    t = {**s, "cu": s["cu"] + LEAD}
    for n in ("q", "k", "v"):
        t[n] = torch.cat([torch.full_like(s[n][:1], float("nan")).expand(LEAD, *s[n].shape[1:]), s[n]])
    return s, t


@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
@pytest.mark.parametrize("n", [3, 31, 32, 70])
def test_append(gpu, n, fp8):
    q_lens = [1 + i % 4 for i in range(n)]
    c = Batch(tuple(q_lens), tuple(a + 9 * (i % 3) for i, a in enumerate(q_lens)), fp8=fp8, pad=2)
    s, t = shifted(c)
    before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
    f = gpu.rope_frequencies(c.dim)
    q_out = torch.full_like(t["q"], 7.0)
    device_flags()
    gpu.paged_append(t["k"], t["v"], t["k_cache"], t["v_cache"], t["cu"], t["kv_lens"], t["table"],
                     q=t["q"], inv_freq=f, k_scale=t["scale"], v_scale=t["scale"], q_out=q_out)
    torch.cuda.synchronize()
    assert device_flags() == 0
    end = LEAD + s["cpu"]["cu"][-1]
    assert torch.all(q_out[:LEAD] == 7) and torch.all(q_out[end:] == 7)
    check_append(c, {**t, "k": s["k"], "v": s["v"]}, before, q_out[LEAD:], f.cpu().numpy(), "half", 1.0)


@pytest.mark.parametrize("c", [Batch((1, 2), (300, 40), dim=128), Batch((1, 1), (9000, 7000)),
                               Batch((90, 40), (300, 40)), Batch((40, 90), (300, 2000), fp8=True)],
                         ids=str)
def test_attention(gpu, c):
    s, t = shifted(c)
    out = torch.full_like(t["q"], 7.0)
    lse = torch.full(t["q"].shape[:2], 7.0, device="cuda")
    device_flags()
    attend(gpu, c, t, out=out, lse=lse)
    torch.cuda.synchronize()
    assert device_flags() == 0
    assert torch.all(out[:LEAD] == 7) and torch.all(lse[:LEAD] == 7)
    check_attention(c, s, out[LEAD:], lse[LEAD:])
    assert out.dtype is DT[c.dtype]
