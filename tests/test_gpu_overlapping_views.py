"""Queries whose elements share memory (sliding and repeated views): the outputs the
wrappers allocate hold the elements of a head side by side all the same."""
import pytest
import torch

from paged_cases import Batch, make
from test_gpu_paged import attend

pytestmark = pytest.mark.gpu


def views(shape, dtype):
    """Sliding windows over one vector along the second to last dimension, and one head
    repeated."""
    *lead, h, d = shape
    n = 1
    for x in lead:
        n *= x
    flat = torch.randn(n * 8 + 8 * (h + d), device="cuda").to(dtype)
    strides = [8] * len(lead)
    for i in range(len(lead) - 2, -1, -1):
        strides[i] = strides[i + 1] * lead[i + 1]
    yield flat.as_strided(shape, (*strides, 1, 1))
    yield flat.as_strided(shape, (*strides, 8, 1))
    yield torch.randn(*lead, 1, d, device="cuda").to(dtype).expand(shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope(gpu, dtype):
    f, pos = gpu.rope_frequencies(16), torch.arange(10, device="cuda").view(2, 5)
    for q in views((2, 5, 3, 16), dtype):
        for k in views((2, 5, 2, 16), dtype):
            got = gpu.rope_fwd(q, k, f, pos), gpu.rope_fwd(q, k, f, pos, layout="half", q_out=None,
                                                           stream=torch.cuda.current_stream())
            want = gpu.rope_fwd(q.contiguous(), k.contiguous(), f, pos)
            torch.cuda.synchronize()
            for a in got:
                for x, y in zip(a, want):
                    assert x.stride(-1) == 1 and torch.equal(x, y)
            one, _ = gpu.rope_bwd(q, None, f, pos)
            assert one.stride(-1) == 1
            assert torch.equal(one, gpu.rope_bwd(q.contiguous(), None, f, pos)[0])


def test_append_and_attention(gpu):
    c = Batch((2, 3), (20, 40), heads=4, kv_heads=2, dim=32)
    f = gpu.rope_frequencies(32)
    for q in views((5, 4, 32), torch.bfloat16):
        s = make(c)
        args = (s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"], s["table"])
        a = gpu.paged_append(*args, q=q, inv_freq=f)
        b = gpu.paged_append(*args, q=q.contiguous(), inv_freq=f)
        assert a.stride(-1) == 1 and torch.equal(a, b)
        if q.stride(1) % 8 == 0 and q.data_ptr() % 16 == 0:   # (else the attention refuses it)
            x, lx = attend(gpu, c, {**s, "q": q})
            y, ly = attend(gpu, c, {**s, "q": q.contiguous()})
            assert x.stride(-1) == 1 and torch.equal(x, y) and torch.equal(lx, ly)
